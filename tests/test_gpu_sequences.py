"""Prompts and single tokens through GDN layers, and log-probabilities, on a GPU against the fp64 oracles.

Tolerances.  All arithmetic is fp32 or keeps 22 bits (fp16 in two terms), and the rule contracts: the state's error is
decayed by the gates and by 1 - beta k k^T, so it holds that of the last tokens, tens of roundings of 2^-23 to 2^-22 of a
head's largest value: 2e-5 of it bounds outputs (5e-6 expected), 1e-5 of a head's state in the 2-norm, as everywhere in
these tests.  bf16 outputs add their rounding, 2^-8 of the value at most.
"""
import numpy as np
import pytest
import torch

import synthetic as S
from oracle import gdn_oracle as O
from oracle import seq_oracle as Q

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HEADS = {"qwen": (2, 6, 128, 128), "d32": (4, 4, 32, 32), "d64": (2, 4, 64, 64), "wide_k": (1, 2, 128, 32),
         "wide_v": (3, 3, 32, 128), "d64x128": (1, 3, 64, 128), "d128x64": (2, 2, 128, 64), "shared9": (1, 9, 64, 32)}


def f64(t):
    return t.double().cpu().numpy()


class Case:
    """One layer's inputs of a ragged batch: device tensors and their fp64 values."""

    def __init__(self, seed, heads, lens, dtype="bf16", out="f32", K=4, conv=1, act=1, q_scale=0.25, layers=2, layer=1,
                 edge="", slow=False):
        self.rng = rng = np.random.default_rng(seed)
        Hk, Hv, dk, dv = HEADS[heads] if isinstance(heads, str) else heads
        self.d = O.Dims(Hk, Hv, dk, dv, K, conv, act, q_scale, 1e-6)
        self.lens, self.B, self.layers, self.layer = list(lens), len(lens), layers, layer
        self.dtype, self.out_dtype = DT[dtype], DT[out]
        rows, C = sum(lens), self.d.C
        x = rng.standard_normal((rows, C)).astype(np.float32)
        beta = 1 / (1 + np.exp(-rng.standard_normal((rows, Hv)).astype(np.float32)))
        log_g = -np.logaddexp(0, rng.standard_normal((rows, Hv))).astype(np.float32)
        if slow:
            log_g *= np.geomspace(0.003, 1, Hv).astype(np.float32)
        if edge:
            w = S.workload(2).replace(Hk=Hk, Hv=Hv, dk=dk, dv=dv, edge=edge)
            x, beta, log_g = S.apply_edges(w, x, beta, log_g)
        cuda = lambda a, t: torch.from_numpy(np.ascontiguousarray(a)).to(t).cuda()  # noqa: E731
        self.x, self.beta, self.log_g = cuda(x, self.dtype), cuda(beta, self.dtype), cuda(log_g, self.dtype)
        self.w = cuda((rng.standard_normal((layers, C, K)) * K ** -0.5).astype(np.float32), torch.float32)
        self.state = cuda((0.3 * rng.standard_normal((self.B, layers, Hv, dk, dv))).astype(np.float32), torch.float32)
        self.conv = cuda(rng.standard_normal((self.B, layers, K - 1, C)).astype(np.float32), torch.float32)
        self.out = torch.full((rows, Hv, dv), 7.0, dtype=self.out_dtype, device="cuda")

    def runner(self, verifier=None):
        from gated_deltanet_tree_gb300 import _native as N
        from gated_deltanet_tree_gb300 import runtime as R
        d = self.d
        code = N.GDN_DTYPE_BF16 if self.dtype == torch.bfloat16 else N.GDN_DTYPE_F32
        dims = R.make_dims(d.Hk, d.Hv, d.dk, d.dv, d.K, d.conv_mode, d.act, code, d.q_scale, d.l2_eps)
        return R.SequenceRunner(dims, self.B, self.layers, verifier=verifier)

    def inputs(self):
        return self.x, (self.w if self.d.conv_mode else None), self.beta, self.log_g

    def reference(self, state=None, conv=None, zero=False):
        l = self.layer
        T = f64(self.state[:, l] if state is None else state)
        W = f64(self.conv[:, l] if conv is None else conv)
        if zero:
            T, W = np.zeros_like(T), np.zeros_like(W)
        w = f64(self.w[l]) if self.d.conv_mode else None
        return Q.run_batch(self.lens, T, W, f64(self.x), f64(self.beta), f64(self.log_g), w, self.d)


def check(case, ref, out, state, conv, where=""):
    """Outputs, states and windows (one layer's) against the reference's."""
    o, T, W = ref
    bf16 = out.dtype == torch.bfloat16
    got, at = f64(out), 0
    for b, n in enumerate(case.lens):
        for h in range(case.d.Hv):
            r, g = o[at:at + n, h], got[at:at + n, h]
            if n:
                tol = 2e-5 * np.abs(r).max() + (2.0 ** -8 * np.abs(r) if bf16 else 0.0) + 1e-30
                err = np.abs(g - r)
                assert (err <= tol).all(), (where, b, h, float((err - tol).max()), np.argwhere(err > tol)[:4].tolist())
            s, t = f64(state[b, h]), T[b, h]
            assert np.linalg.norm(s - t) <= 1e-5 * np.linalg.norm(t) + 1e-30, (where, b, h, "state", np.linalg.norm(s - t) / np.linalg.norm(t))
        at += n
        if case.d.conv_mode:
            assert np.array_equal(f64(conv[b]), W[b]), (where, b, "window")


def others_unchanged(case, before, after):
    keep = [i for i in range(case.layers) if i != case.layer]
    assert torch.equal(before[:, keep], after[:, keep])


# ---- prompts --------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("heads", list(HEADS))
@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("f32", "f32"), ("bf16", "bf16")])
def test_prefill_heads_and_types(heads, dtype, out):
    c = Case(1, heads, [70, 0, 1, 129], dtype, out)
    state, conv = c.state.clone(), c.conv.clone()
    r = c.runner()
    r.prefill(c.lens, *c.inputs(), state, conv, c.out, layer=1)
    r.check_error()
    check(c, c.reference(), c.out, state[:, 1], conv[:, 1])
    others_unchanged(c, c.state, state)
    others_unchanged(c, c.conv, conv)


@pytest.mark.parametrize("heads", ["qwen", "d64"])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 130, 191, 192, 193, 321])
def test_prefill_lengths(heads, n):
    c = Case(2, heads, [n], "bf16", slow=True)
    state, conv = c.state.clone(), c.conv.clone()
    r = c.runner()
    r.prefill([n], *c.inputs(), state, conv, c.out, layer=1)
    r.check_error()
    check(c, c.reference(), c.out, state[:, 1], conv[:, 1], n)


@pytest.mark.parametrize("K,conv,act", [(1, 1, 1), (2, 1, 1), (3, 1, 0), (5, 1, 1), (8, 1, 1), (4, 0, 0), (4, 0, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_taps_and_modes(K, conv, act, dtype):
    c = Case(3, "qwen", [2, 75, 5], dtype, K=K, conv=conv, act=act)
    state, window = c.state.clone(), c.conv.clone()
    r = c.runner()
    r.prefill(c.lens, *c.inputs(), state, window, c.out, layer=1)
    r.check_error()
    check(c, c.reference(), c.out, state[:, 1], window[:, 1])


@pytest.mark.parametrize("edge", ["gate_zero", "gate_floor", "beta01", "zero_rows", "gate_zero+beta01+zero_rows"])
@pytest.mark.parametrize("heads,lens", [("qwen", [150, 20]), ("d32", [70, 3])])
def test_prefill_degenerate_values(edge, heads, lens):
    c = Case(4, heads, lens, "bf16", edge=edge)
    state, conv = c.state.clone(), c.conv.clone()
    r = c.runner()
    r.prefill(c.lens, *c.inputs(), state, conv, c.out, layer=1)
    r.check_error()
    check(c, c.reference(), c.out, state[:, 1], conv[:, 1])


@pytest.mark.parametrize("scale", [1e-12, 1e-4, 1e5, 1e12])
def test_prefill_magnitudes(scale):
    """States and values far from 1, alone and together: v and the state enter linearly, so outputs scale with them.
    (A bf16 v keeps its bits at any scale; q and k are normalised.)"""
    c = Case(5, "qwen", [200], "f32", slow=True, act=0, conv=0)
    nq = 2 * c.d.Hk * c.d.dk
    c.x[:, nq:] *= scale
    for factor in (1.0, scale):
        state = (c.state * factor).contiguous()
        ref = c.reference(state=state[:, 1])
        r = c.runner()
        r.prefill(c.lens, *c.inputs(), state, None, c.out, layer=1)
        r.check_error()
        check(c, ref, c.out, state[:, 1], c.conv[:, 1], (scale, factor))


def test_prefill_sudden_growth():
    """Values that grow by 2^40 within a chunk, and shrink again."""
    c = Case(6, "qwen", [260], "f32", slow=True, act=0, conv=0)
    nq = 2 * c.d.Hk * c.d.dk
    for at, e in ((10, 20), (40, 40), (70, -40), (100, 0), (130, 30)):
        c.x[at:at + 30, nq:] *= 2.0 ** e
    state = c.state.clone()
    ref = c.reference()
    r = c.runner()
    r.prefill(c.lens, *c.inputs(), state, None, c.out, layer=1)
    r.check_error()
    check(c, ref, c.out, state[:, 1], c.conv[:, 1])


def test_prefill_repeated_keys():
    """One key throughout, beta 1, no decay: each token replaces the value before; the triangular system is all ones."""
    c = Case(7, "qwen", [200], "f32", act=0, conv=0)
    nq = c.d.Hk * c.d.dk
    c.x[:, nq:2 * nq] = c.x[:1, nq:2 * nq]
    c.beta.fill_(1.0)
    c.log_g.zero_()
    state = c.state.clone()
    ref = c.reference()
    r = c.runner()
    r.prefill(c.lens, *c.inputs(), state, None, c.out, layer=1)
    r.check_error()
    check(c, ref, c.out, state[:, 1], c.conv[:, 1])


@pytest.mark.parametrize("heads", ["qwen", "d32"])
def test_prefill_in_parts_steps_and_out_of_place(heads):
    """A prompt whole, in parts, and token by token gives the same; a kept prefix is not written; rows of wider ones."""
    c = Case(8, heads, [150, 90, 33], "bf16", slow=True)
    ref = c.reference()
    starts = np.cumsum([0] + c.lens)
    r = c.runner()
    state, conv = c.state.clone(), c.conv.clone()
    cuts = [[70, 64, 0], [79, 1, 20], [1, 25, 13]]
    done = [0, 0, 0]
    out = torch.empty_like(c.out)
    wide = torch.full((sum(c.lens), c.d.C + 64), 9.0, dtype=c.dtype, device="cuda")
    for part in cuts:
        at = torch.cat([torch.arange(starts[b] + done[b], starts[b] + done[b] + n) for b, n in enumerate(part)]).cuda()
        x = wide[:len(at)]
        x[:, 32:32 + c.d.C] = c.x[at]
        gates = torch.stack([c.beta[at], c.log_g[at]], 1).contiguous()         # [n, 2, Hv]
        o = torch.empty(len(at), c.d.Hv, c.d.dv, device="cuda")
        before, window = state.clone(), conv.clone()
        s2, w2 = torch.full_like(state, 5.0), torch.full_like(conv, 5.0)
        r.prefill(part, x[:, 32:32 + c.d.C], c.w, gates[:, 0], gates[:, 1], state, conv, o, layer=1, state_out=s2,
                  conv_out=w2)
        assert torch.equal(state, before) and torch.equal(conv, window)
        for b, n in enumerate(part):
            if n:
                state[b, 1], conv[b, 1] = s2[b, 1], w2[b, 1]
            else:
                assert (s2[b, 1] == 5.0).all() and (w2[b, 1] == 5.0).all()
            done[b] += n
        assert (s2[:, 0] == 5.0).all() and (w2[:, 0] == 5.0).all()
        out[at] = o
    r.check_error()
    assert done == c.lens
    check(c, ref, out, state[:, 1], conv[:, 1], "parts")
    # token by token, with requests ending one after another
    state, conv = c.state.clone(), c.conv.clone()
    for t in range(max(c.lens)):
        live = torch.tensor([int(t < n) for n in c.lens], dtype=torch.int32, device="cuda")
        at = torch.tensor([min(starts[b] + t, sum(c.lens) - 1) for b in range(c.B)], device="cuda")
        o = torch.full((c.B, c.d.Hv, c.d.dv), 3.0, device="cuda")
        r.step(c.x[at], c.w, c.beta[at], c.log_g[at], state, conv, o, layer=1, live=live)
        for b in range(c.B):
            if t < c.lens[b]:
                out[at[b]] = o[b]
            else:
                assert (o[b] == 3.0).all()
    r.check_error()
    check(c, ref, out, state[:, 1], conv[:, 1], "steps")
    others_unchanged(c, c.state, state)


@pytest.mark.parametrize("heads,lens", [("qwen", [100, 7]), ("d64", [3, 64])])
def test_prefill_from_nothing(heads, lens):
    c = Case(9, heads, lens, "bf16")
    state, conv = torch.full_like(c.state, float("nan")), torch.full_like(c.conv, float("nan"))
    r = c.runner()
    r.prefill(c.lens, *c.inputs(), None, None, c.out, layer=1, state_out=state, conv_out=conv)
    r.check_error()
    check(c, c.reference(zero=True), c.out, state[:, 1], conv[:, 1])


def test_prefill_many_requests():
    """More requests than a launch takes, of all lengths up to 80, a fifth of them empty."""
    rng = np.random.default_rng(10)
    lens = [0 if i % 5 == 3 else int(n) for i, n in enumerate(rng.integers(1, 81, 300))]
    c = Case(10, (1, 2, 32, 32), lens, "bf16", layers=1, layer=0)
    state, conv = c.state.clone(), c.conv.clone()
    r = c.runner()
    r.prefill(c.lens, *c.inputs(), state, conv, c.out)
    r.check_error()
    check(c, c.reference(), c.out, state[:, 0], conv[:, 0])


@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("heads", ["qwen", "d32"])
def test_prefill_values_that_are_not_finite_stay_in_their_column(value, heads):
    """Columns of v do not touch each other: an infinity or a NaN in one, of a row or of a state, leaves the others' outputs and
    states within the tolerances, and its own from there on without a finite value."""
    c = Case(12, heads, [150, 40], "f32")
    d = c.d
    head, col, at = d.Hv - 1, 5, 70
    c.x[at, 2 * d.Hk * d.dk + head * d.dv + col] = value
    c.state[0, 1, 0, 3, 7] = value
    with np.errstate(invalid="ignore", over="ignore"):
        o, T, W = c.reference()
    state, conv = c.state.clone(), c.conv.clone()
    r = c.runner()
    r.prefill(c.lens, *c.inputs(), state, conv, c.out, layer=1)
    r.check_error()
    got, S1 = f64(c.out), f64(state[:, 1])
    for a, s in ((o, T), (got, S1)):
        assert not np.isfinite(a[at:150, head, col]).any() and not np.isfinite(a[:150, 0, 7]).any()
        assert not np.isfinite(s[0, head, :, col]).any() and not np.isfinite(s[0, 0, :, 7]).any()
        a[64:150, head, col] = a[:150, 0, 7] = s[0, head, :, col] = s[0, 0, :, 7] = 0   # (a chunk's outputs are one product)
    assert np.array_equal(f64(conv[:, 1]), W, equal_nan=True)
    for b, rows in enumerate((slice(0, 150), slice(150, 190))):
        for h in range(d.Hv):
            assert np.abs(got[rows, h] - o[rows, h]).max() <= 2e-5 * np.abs(o[rows, h]).max(), (b, h)
            assert np.linalg.norm(S1[b, h] - T[b, h]) <= 1e-5 * np.linalg.norm(T[b, h]), (b, h)


def test_prefill_does_not_mix_requests():
    """A request with NaN everywhere leaves the others' results as they were, bit for bit."""
    c = Case(11, "qwen", [90, 100, 64, 5], "bf16")
    state, conv = c.state.clone(), c.conv.clone()
    r = c.runner()
    r.prefill(c.lens, *c.inputs(), state, conv, c.out, layer=1)
    c.x[90:190] = float("nan")
    bad = c.state.clone()
    bad[1] = float("nan")
    window, out = c.conv.clone(), torch.empty_like(c.out)
    r.prefill(c.lens, *c.inputs(), bad, window, out, layer=1)
    r.check_error()
    keep = torch.ones(len(out), dtype=torch.bool)
    keep[90:190] = False
    assert torch.equal(out[keep.cuda()], c.out[keep.cuda()]) and torch.isnan(out[90:190]).all()
    for b in (0, 2, 3):
        assert torch.equal(bad[b], state[b])


# ---- single tokens --------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("heads", list(HEADS))
@pytest.mark.parametrize("dtype,out", [("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("B", [1, 80])
def test_step(heads, dtype, out, B):
    c = Case(20, heads, [1] * B, dtype, out)
    ref = c.reference()
    state, conv = c.state.clone(), c.conv.clone()
    r = c.runner()
    r.step(*c.inputs(), state, conv, c.out, layer=1)
    r.check_error()
    check(c, ref, c.out, state[:, 1], conv[:, 1])
    others_unchanged(c, c.state, state)
    s2, w2, o2 = torch.zeros_like(state), torch.zeros_like(conv), torch.zeros_like(c.out)
    r.step(*c.inputs(), c.state, c.conv, o2, layer=1, state_out=s2, conv_out=w2)
    assert torch.equal(o2, c.out) and torch.equal(s2[:, 1], state[:, 1]) and torch.equal(w2[:, 1], conv[:, 1])
    assert not s2[:, 0].any() and not w2[:, 0].any()


@pytest.mark.parametrize("heads", ["qwen", "d64", "d64x128", "d128x64", "one_head"])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("K,conv", [(4, 1), (1, 1), (3, 1), (4, 0)])
def test_step_of_many(heads, dtype, out, K, conv):
    """Batches large enough for the stream of tiles: in place, to other buffers, and with requests that take no part (runs of
    them at the front, in the middle and at the end)."""
    B = {"qwen": 170, "d64": 190, "d64x128": 320, "d128x64": 155, "one_head": 460}[heads]
    shape = (1, 1, 128, 128) if heads == "one_head" else heads
    c = Case(22, shape, [1] * B, dtype, out, K=K, conv=conv, layers=1, layer=0)
    ref = c.reference()
    state, window = c.state.clone(), c.conv.clone()
    r = c.runner()
    r.step(*c.inputs(), state, window, c.out)
    r.check_error()
    check(c, ref, c.out, state[:, 0], window[:, 0])
    live = torch.ones(B, dtype=torch.int32, device="cuda")
    live[:7], live[60:75], live[B - 9:], live[::11] = 0, 0, 0, 0
    on = live.bool()
    s2, w2, o2 = torch.full_like(state, 5.0), torch.full_like(window, 5.0), torch.full_like(c.out, 5.0)
    r.step(*c.inputs(), c.state, c.conv, o2, state_out=s2, conv_out=w2, live=live)
    r.check_error()
    assert torch.equal(s2[on], state[on]) and torch.equal(o2[on], c.out[on])
    assert (s2[~on] == 5.0).all() and (o2[~on] == 5.0).all() and (w2[~on] == 5.0).all()
    if conv:
        assert torch.equal(w2[on], window[on])
    live.zero_()
    r.step(*c.inputs(), s2, w2, o2, live=live)
    r.check_error()
    assert torch.equal(s2[on], state[on]) and torch.equal(o2[on], c.out[on])


@pytest.mark.parametrize("K,conv,act", [(1, 1, 1), (2, 1, 0), (6, 1, 1), (8, 1, 1), (4, 0, 1)])
def test_step_taps_and_modes(K, conv, act):
    c = Case(21, "qwen", [1, 1, 1], "bf16", K=K, conv=conv, act=act)
    ref = c.reference()
    state, window = c.state.clone(), c.conv.clone()
    r = c.runner()
    r.step(*c.inputs(), state, window, c.out, layer=1)
    r.check_error()
    check(c, ref, c.out, state[:, 1], window[:, 1])


# ---- log-probabilities ----------------------------------------------------------------------------------------------

def rows_of(rng, n, V, kind, dtype):
    z = 2.0 * rng.standard_normal((n, V))
    if kind == "ties":
        z = np.round(z)
    elif kind == "constant":
        z[:] = 1.5
    elif kind == "rising":
        z = np.sort(z, axis=1)
    elif kind == "falling":
        z = -np.sort(-z, axis=1)
    elif kind == "masked":
        z[:, rng.random(V) < 0.7] = -np.inf
        z[:, V // 2] = 0.25
    elif kind == "nearly_all_masked":
        z[:] = -np.inf
        z[:, V - 1], z[:, V // 3] = 3.0, 2.0
    elif kind == "large":
        z *= 1e4
    elif kind == "sure":
        z[:, V // 2] += 200.0
    return torch.from_numpy(z.astype(np.float32)).to(DT[dtype]).cuda()


def check_scores(z, top_k, got, tokens=None):
    """fp32 sums of V terms in some order: 2^-24 V^(1/2) is far below 1e-6; a logarithm of 1 + 1e-6 and differences of
    logits of size m round by 2^-23 m.  The entropy's terms are of the size of the logits' spread."""
    top, best, given, entropy = got
    z64 = f64(z)
    for r in range(z.shape[0]):
        row = z64[r]
        logp = Q.log_probabilities(row)
        order = Q.best_tokens(row, top_k)
        assert best[r].tolist() == order, (r, best[r].tolist(), order)
        size = np.abs(row[np.isfinite(row)]).max() - row.max() + np.abs(row.max()) + 2.0
        tol = 1e-6 + 2.0 ** -22 * size
        for have, want in zip(f64(top[r]), logp[order]):
            assert have == want or abs(have - want) <= tol + 2.0 ** -23 * abs(want), (r, have, want)
        if tokens is not None:
            want, have = logp[int(tokens[r])], float(given[r])
            assert have == want or abs(have - want) <= tol + 2.0 ** -23 * abs(want), (r, have, want)
        assert abs(float(entropy[r]) - Q.entropy(row)) <= 4 * tol, (r, float(entropy[r]), Q.entropy(row))


@pytest.mark.parametrize("V,top_k,n", [(1, 1, 3), (7, 7, 2), (31, 20, 5), (257, 32, 4), (1000, 20, 3), (4099, 8, 9),
                                       (8192, 1, 2), (8193, 32, 3), (16385, 8, 2), (50001, 4, 5), (70000, 32, 2), (131072, 8, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["normal", "ties", "constant", "rising", "masked"])
def test_logprobs(V, top_k, n, dtype, kind):
    from gated_deltanet_tree_gb300.runtime import TokenScorer
    rng = np.random.default_rng(V + top_k)
    z = rows_of(rng, n, V, kind, dtype)
    tokens = torch.from_numpy(rng.integers(0, V, n).astype(np.int32)).cuda()
    s = TokenScorer(n + 2, V, top_k)
    got = s.score(z, tokens)
    s.check_error()
    check_scores(z, top_k, got, tokens)
    assert (s.tokens[n:] == -1).all() and not s.top[n:].any() and not s.given[n:].any()


@pytest.mark.parametrize("kind", ["falling", "nearly_all_masked", "large", "sure"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n", [2, 400])
def test_logprobs_values(kind, dtype, n):
    from gated_deltanet_tree_gb300.runtime import TokenScorer
    rng = np.random.default_rng(30)
    z = rows_of(rng, n, 20003, kind, dtype)
    s = TokenScorer(n, 20003, 20)
    top, best, given, entropy = s.score(z)
    assert given is None
    s.check_error()
    at = [0, 1, n - 1]
    check_scores(z[at], 20, (top[at], best[at], None, entropy[at]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logprobs_rows_of_wider_ones(dtype):
    """Rows at every alignment, and neighbours that must not be seen."""
    from gated_deltanet_tree_gb300.runtime import TokenScorer
    rng = np.random.default_rng(31)
    V, n = 9001, 9
    wide = torch.full((n, V + 14), float("nan"), dtype=DT[dtype], device="cuda")
    wide[:, 8:8 + V] = rows_of(rng, n, V, "normal", dtype)
    z = wide[:, 8:8 + V]
    tokens = torch.from_numpy(rng.integers(0, V, n).astype(np.int32)).cuda()
    s = TokenScorer(n, V, 5)
    got = s.score(z, tokens)
    s.check_error()
    check_scores(z, 5, got, tokens)


def test_logprobs_rows_without_a_distribution():
    from gated_deltanet_tree_gb300 import _native as N
    from gated_deltanet_tree_gb300.runtime import TokenScorer
    rng = np.random.default_rng(32)
    z = rows_of(rng, 5, 40000, "normal", "f32")
    z[1, 39999] = float("nan")
    z[2, 17] = float("inf")
    z[3] = -float("inf")
    s = TokenScorer(5, 40000, 4)
    tokens = torch.tensor([3, 3, 3, 3, 40000], dtype=torch.int32, device="cuda")
    top, best, given, entropy = s.score(z, tokens)
    with pytest.raises(N.GdnError) as e:
        s.check_error()
    assert e.value.status == N.GDN_ERR_LOGITS
    for r in (1, 2, 3):
        assert torch.isnan(top[r]).all() and (best[r] == -1).all() and torch.isnan(given[r]) and torch.isnan(entropy[r])
    assert torch.isnan(given[4]) and torch.isfinite(top[4]).all() and torch.isfinite(given[0])
    check_scores(z[[0, 4]], 4, (top[[0, 4]], best[[0, 4]], None, entropy[[0, 4]]))
    s.check_error()
