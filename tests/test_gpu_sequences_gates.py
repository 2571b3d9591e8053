"""Prompts whose log gates change sign within a chunk, on a GPU against the fp64 oracle.

The chunked form scales what it computes from products of gates; the rule only ever multiplies those of consecutive tokens.
Tolerances as for values of changing size in test_gpu_sequences_calls.py: outputs within 2e-5 of the largest one of their
head and chunk of 64 tokens, states within 1e-5 of themselves in the 2-norm (tens of roundings of 2^-23 to 2^-22; a growth
by 2^4 between the tokens of a chunk costs the fp32 triangular system four bits of its own, 2^-24 2^4 = 1e-6)."""
import numpy as np
import pytest
import torch

from oracle import gdn_oracle as O
from test_gpu_sequences import Case, built, f64  # noqa: F401

pytestmark = pytest.mark.gpu

# The states are fp32, which the caller's gates must keep them in (as the header says): a head is compared until one of its
# entries is above this, so that the rule's sums of 128 products with a state's entries and unit keys do not overflow either
# (|T^T k| <= 128^(1/2) max T).
FP32_MOST = 3.4e38 / 16
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
    x, beta, gates, w = f64(c.x), f64(c.beta), f64(c.log_g), f64(c.w[c.layer]) if c.d.conv_mode else None
    got, at = f64(c.out), 0
    for b, rows in enumerate(c.lens):
        T, W = f64(c.state[b, c.layer]), f64(c.conv[b, c.layer])
        o, left = np.zeros((rows, Hv, c.d.dv)), np.full(Hv, rows)   # left: the token at which a head's state leaves fp32
        for t in range(rows):
            T, W, o[t], _, _ = O.token_step(T, W, x[at + t], beta[at + t], gates[at + t], w, c.d)
            over = np.abs(T).max((1, 2)) > FP32_MOST
            left[over] = np.minimum(left[over], t)
        for h in range(Hv):
            for a in range(0, rows, 64):
                want = o[a:a + 64, h]
                if a + len(want) <= left[h]:
                    err = np.abs(got[at + a:at + a + len(want), h] - want).max() / np.abs(want).max()
                    assert err <= 2e-5, (b, h, a, err)
            if left[h] == rows:
                s = f64(state[b, c.layer, h])
                assert np.linalg.norm(s - T[h]) <= 1e-5 * np.linalg.norm(T[h]), (b, h, np.linalg.norm(s - T[h]) / np.linalg.norm(T[h]))
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


@pytest.mark.parametrize("size", [2.0, 4.0])
@pytest.mark.parametrize("heads", ["qwen", "d64"])
def test_gates_of_random_sign_and_any_size(size, heads):
    c = Case(42, heads, [150, 70], "f32")
    run_and_check(c, size * c.rng.standard_normal((220, c.d.Hv)))


@pytest.mark.parametrize("size", [0.25, 1.0, 2.0])
@pytest.mark.parametrize("first", [1, -1])
def test_states_that_grow_and_shrink_within_a_chunk(size, first):
    """Half a chunk of growing gates and half of shrinking ones, either first: by e^64 and back at the largest."""
    run_and_check(Case(43, "qwen", [150], "f32"), first * size * np.where(np.arange(150) % 64 < 32, 1.0, -1.0))


@pytest.mark.parametrize("alternate", [3.0, 8.0, 30.0])
def test_gates_that_alternate_far(alternate):
    """The state grows by e^alternate and comes back, token by token."""
    run_and_check(Case(44, "qwen", [100], "f32"), alternate * SIGN[:100])


@pytest.mark.parametrize("beta", [3.0, 5.0, -2.0])
@pytest.mark.parametrize("heads", ["qwen", "d64"])
def test_beta_that_grows_states_which_are_then_forgotten(beta, heads):
    """1 - beta k k^T grows what lies along keys that are alike, before gates of e^-3 forget it: later tokens' updates are small
    beside the early ones."""
    c = Case(45, heads, [150], "f32", act=0, conv=0)
    nq = c.d.Hk * c.d.dk
    c.x[:, nq:2 * nq] += 3.0 * c.x[:1, nq:2 * nq]
    at = np.arange(150) % 64
    run_and_check(c, np.where((at >= 24) & (at < 34), -3.0, -0.05), np.where(at < 24, beta, 0.7))


@pytest.mark.parametrize("lens", [[17], [64], [65], [128], [193, 40]])
def test_growing_chunks_first_last_and_alone(lens):
    """The chunk that is taken again is a call's first, last or only one, or every one."""
    n = sum(lens)
    for a, b in ((0, n), (0, 20), (n - 12, n)):
        c = Case(46, "qwen", lens, "f32", slow=True)
        g = f64(c.log_g)
        g[a:b] += 1.5
        run_and_check(c, g)


def test_growing_chunks_of_one_head():
    """Only one head's chunks are taken again; the others' results are those of a call without it, bit for bit."""
    c = Case(47, "qwen", [200], "f32")
    state, conv = c.state.clone(), c.conv.clone()
    r = c.runner()
    r.prefill(c.lens, *c.inputs(), state, conv, c.out, layer=1)
    c.log_g[:, 2] = torch.from_numpy(2.0 * SIGN).float().repeat(2)[:200].cuda() + 0.1
    s2, w2, out = c.state.clone(), c.conv.clone(), torch.empty_like(c.out)
    r.prefill(c.lens, *c.inputs(), s2, w2, out, layer=1)
    r.check_error()
    keep = [h for h in range(c.d.Hv) if h != 2]
    assert torch.equal(out[:, keep], c.out[:, keep]) and torch.equal(s2[:, 1, keep], state[:, 1, keep])
    o, T, _ = c.reference()
    assert np.abs(f64(out[:, 2]) - o[:, 2]).max() <= 2e-5 * np.abs(o[:, 2]).max()
    assert np.linalg.norm(f64(s2[0, 1, 2]) - T[0, 2]) <= 1e-5 * np.linalg.norm(T[0, 2])


@pytest.mark.parametrize("at", [1590, 1600, 3190])
def test_growing_chunks_at_the_ends_of_a_long_prompt_s_parts(at):
    """3200 tokens are 50 chunks, taken in two halves: the chunk that is taken again is the last of the first (before token 1600),
    the first of the second, or the last of all."""
    c = Case(48, (1, 2, 128, 128), [3200], "f32", slow=True)
    g = f64(c.log_g)
    g[at:at + 10] += 1.5
    run_and_check(c, g)
