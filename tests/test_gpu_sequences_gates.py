"""Prompts whose log gates change sign within a chunk, on a GPU against the fp64 oracle.

The chunked form scales what it computes from products of gates; the rule only ever multiplies those of consecutive tokens.
Tolerances as for values of changing size in test_gpu_sequences_calls.py: outputs within 2e-5 of the largest one of their
head and chunk of 64 tokens, states within 1e-5 of themselves in the 2-norm (tens of roundings of 2^-23 to 2^-22; a growth
by 2^4 between the tokens of a chunk costs the fp32 triangular system four bits of its own, 2^-24 2^4 = 1e-6)."""
import numpy as np
import pytest
import torch

from test_gpu_sequences import Case, built, f64  # noqa: F401

pytestmark = pytest.mark.gpu

SIGN = (-1.0) ** np.arange(150)


def run_and_check(c, log_g, beta=None):
    """log_g, beta: [tokens] or [tokens, Hv], put into the case."""
    n, Hv = c.beta.shape
    c.log_g = torch.from_numpy(np.broadcast_to(np.asarray(log_g, dtype=np.float32).reshape(n, -1), (n, Hv)).copy()).to(c.dtype).cuda()
    if beta is not None:
        c.beta = torch.from_numpy(np.broadcast_to(np.asarray(beta, dtype=np.float32).reshape(n, -1), (n, Hv)).copy()).to(c.dtype).cuda()
    state, conv = c.state.clone(), c.conv.clone()
    r = c.runner()
    r.prefill(c.lens, *c.inputs(), state, conv, c.out, layer=c.layer)
    r.check_error()
    o, T, _ = c.reference()
    got, at = f64(c.out), 0
    for b, rows in enumerate(c.lens):
        for h in range(Hv):
            for a in range(at, at + rows, 64):
                want = o[a:min(a + 64, at + rows), h]
                err = np.abs(got[a:a + len(want), h] - want).max() / np.abs(want).max()
                assert err <= 2e-5, (b, h, a - at, err)
            s, t = f64(state[b, c.layer, h]), T[b, h]
            assert np.linalg.norm(s - t) <= 1e-5 * np.linalg.norm(t), (b, h, np.linalg.norm(s - t) / np.linalg.norm(t))
        at += rows


@pytest.mark.parametrize("size", [0.5, 1.0, 2.0, 4.0])
@pytest.mark.parametrize("heads,dtype", [("qwen", "f32"), ("d64", "bf16")])
def test_gates_that_alternate(size, heads, dtype):
    """e^size and e^-size in turn: no product of gates is above e^size, though those above 1 alone come to e^(32 size)."""
    run_and_check(Case(40, heads, [150], dtype), size * SIGN)


@pytest.mark.parametrize("size", [0.25, 0.5, 1.0])
def test_gates_of_random_sign(size):
    c = Case(41, "qwen", [150, 70], "f32")
    run_and_check(c, size * c.rng.standard_normal((220, c.d.Hv)))
