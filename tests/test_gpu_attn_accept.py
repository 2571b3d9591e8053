"""GPU parity of the 4-bit cache (append, read, attention) and of the acceptance walk against their fp64 oracles.

Tolerances, from the arithmetic:
- cache contents: exact (a group's scale and codes follow from exactly rounded operations);
- fp32 attention: scores of magnitude S carry an error of a few S 2^-24, so weights are off by about S 1e-6 relative;
  with S <= 30 here, |o - o_ref| <= 3e-5 max|v|;
- bf16 attention: the output's own rounding is 2^-9 |o| at most, the weights' rounding to fp16 adds at most
  2^-11 max|v|; twice that is allowed: |o - o_ref| <= 2^-8 |o_ref| + 2^-10 max|v|.
- acceptance: integers, equal.
"""
import numpy as np
import pytest
import torch

import synthetic as S
from oracle import accept_oracle as A
from oracle import kv4_oracle as K

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def built():
    from gated_deltanet_tree_gb300.build import build
    build()


def rows(rng, *shape, dtype):
    x = torch.from_numpy(rng.standard_normal(shape).astype(np.float32))
    x[..., rng.integers(0, shape[-1], 2)] *= 5.0
    return x.to(DT[dtype]).cuda()


def f64(t):
    return t.double().cpu().numpy()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def oracle_rows(x):
    """Quantised values of rows [..., D]."""
    x = np.asarray(x, dtype=np.float64)
    return np.stack([K.quantise_row(r) for r in x.reshape(-1, x.shape[-1])]).reshape(x.shape)


def make_cache(Hq, Hkv, D, B, layers, pages_max, dtype, shuffle=None, extra=3):
    from gated_deltanet_tree_gb300 import runtime as R
    dims = R.make_attn_dims(Hq, Hkv, D, dtype=DT[dtype])
    n_pages = B * pages_max + extra
    order = np.random.default_rng(0 if shuffle is None else shuffle).permutation(n_pages)[:B * pages_max]
    # pages start as garbage, every bit set: scales read as NaN until written
    pool = torch.full((layers, n_pages, Hkv, 72 * D), 255, dtype=torch.uint8, device="cuda")
    return R.KV4Cache(dims, pool, i32(order.reshape(B, pages_max)), i32(np.zeros(B)))


def cache_rows(c, b, l, h, L, D):
    k, v = np.zeros((L, D)), np.zeros((L, D))
    pool, table = c.pool.cpu().numpy(), c.page_table.cpu().numpy()
    for p in range(-(-L // 64)):
        bk, bv = K.block_rows(pool[l, table[b, p], h], D)
        m = min(64, L - 64 * p)
        k[64 * p:64 * p + m], v[64 * p:64 * p + m] = bk[:m], bv[:m]
    return k, v


# ---- append and read ------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_append_in_pieces_is_exact(D, dtype):
    """Rows appended in ragged pieces that end inside words and pages, compared bit by bit with the oracle's groups;
    the pages are read by the oracle's own reading of the format and by gdn_kv4_read."""
    rng = np.random.default_rng(D)
    B, L, Hkv = 3, 2, 2
    c = make_cache(4, Hkv, D, B, L, 3, dtype)
    have = [[] for _ in range(B)]
    for counts in ([1, 0, 5], [6, 9, 3], [64, 50, 63], [1, 64, 2], [0, 1, 60]):
        n = 64
        k, v = rows(rng, B, L, n, Hkv, D, dtype=dtype), rows(rng, B, L, n, Hkv, D, dtype=dtype)
        c.append(k, v, i32(counts))
        for b, m in enumerate(counts):
            have[b].append((f64(k[b, :, :m]), f64(v[b, :, :m])))
    c.check_error()
    lens = [sum(p[0].shape[1] for p in h) for h in have]
    assert c.seq_len.tolist() == lens and not c.ticket.any()
    kr, vr = c.read(None, 150)
    for b in range(B):
        ko = oracle_rows(np.concatenate([p[0] for p in have[b]], 1))
        vo = oracle_rows(np.concatenate([p[1] for p in have[b]], 1))
        for l in range(L):
            for h in range(Hkv):
                kk, vv = cache_rows(c, b, l, h, lens[b], D)
                assert np.array_equal(kk, ko[l, :, h]) and np.array_equal(vv, vo[l, :, h])
        assert np.array_equal(f64(kr[b])[:, :lens[b]], ko) and np.array_equal(f64(vr[b])[:, :lens[b]], vo)
        assert not kr[b, :, lens[b]:].any() and not vr[b, :, lens[b]:].any()
    # a range that starts inside a page, in bf16
    k2, v2 = c.read(i32([70, 3, 100]), 21, dtype=torch.bfloat16)
    for b, t in enumerate([70, 3, 100]):
        m = max(0, min(21, lens[b] - t))
        assert torch.equal(k2[b, :, :m], kr[b, :, t:t + m].bfloat16()) and not k2[b, :, m:].any()
        assert torch.equal(v2[b, :, :m], vr[b, :, t:t + m].bfloat16()) and not v2[b, :, m:].any()
    c.check_error()


def test_append_takes_paths_strides_and_special_groups():
    rng = np.random.default_rng(1)
    B, L, Hkv, D, n = 2, 1, 2, 128, 9
    c = make_cache(4, Hkv, D, B, L, 2, "bf16")
    wide = rows(rng, B, L, n, 4 * Hkv + 4, D, dtype="bf16")       # a fused projection's rows
    k, v = wide[..., 2:2 + Hkv, :], wide[..., 6:6 + Hkv, :]
    wide[0, 0, 4, 2, 5] = float("nan")          # key group 0 of node 4, head 0
    wide[0, 0, 4, 6, 40] = float("-inf")        # value group 1
    wide[0, 0, 7, 3, 32:64] = 0.0
    wide[1, 0, 0, 2, 0] = 3.0e38
    wide[1, 0, 0, 7, :32] = 1.0e-6              # a scale among fp16's subnormals
    path = i32([[0, 4, 7, 8, 0, 0, 0, 0, 0], [0, 1, 0, 0, 0, 0, 0, 0, 0]])
    c.append(k, v, i32([4, 2]), path=path)
    c.check_error()
    for b, p in enumerate(([0, 4, 7, 8], [0, 1])):
        ko, vo = oracle_rows(f64(k[b, 0])[p]), oracle_rows(f64(v[b, 0])[p])
        for h in range(Hkv):
            kk, vv = cache_rows(c, b, 0, h, len(p), D)
            assert np.array_equal(kk, ko[:, h], equal_nan=True) and np.array_equal(vv, vo[:, h], equal_nan=True)
    kk, _ = cache_rows(c, 0, 0, 0, 4, D)
    assert np.isnan(kk[1, :32]).all() and not np.isnan(kk[1, 32:]).any() and not np.isnan(np.delete(kk, 1, 0)).any()


def test_append_refuses_what_does_not_fit():
    from gated_deltanet_tree_gb300 import _native as N
    rng = np.random.default_rng(2)
    c = make_cache(2, 1, 64, 3, 1, 2, "bf16")
    k, v = rows(rng, 3, 1, 100, 1, 64, dtype="bf16"), rows(rng, 3, 1, 100, 1, 64, dtype="bf16")

    def refused(count, path=None, keep=(0, 1, 2)):
        before, lens = c.pool.clone(), c.seq_len.clone()
        c.append(k, v, i32(count), path=path)
        with pytest.raises(N.GdnError) as e:
            c.check_error()
        assert e.value.status == N.GDN_ERR_CACHE
        c.check_error()
        for b in keep:
            assert int(c.seq_len[b]) == int(lens[b])
            for pg in c.page_table[b].tolist():
                if 0 <= pg < c.pool.shape[1]:
                    assert torch.equal(c.pool[:, pg], before[:, pg])
        assert not c.ticket.any()

    c.append(k, v, i32([100, 100, 10]))
    c.check_error()
    refused([29, 28, 100], keep=[0])                    # request 0 would pass its 128 tokens
    assert c.seq_len.tolist() == [100, 128, 110]
    refused([-1, 0, 0])
    refused([101, 0, 0])
    path = i32(np.zeros((3, 100)))
    path[0, 3] = 100
    refused([5, 0, 0], path=path)
    c.page_table[0, 1] = c.pool.shape[1]
    refused([1, 0, 0])
    c.page_table[0, 1] = -1
    refused([1, 0, 0])
    c.seq_len[0] = 129
    refused([0, 0, 0])


# ---- attention ------------------------------------------------------------------------------------------------------

def filled(rng, Hq, Hkv, D, lens, layers, dtype, slack=0):
    B = len(lens)
    c = make_cache(Hq, Hkv, D, B, layers, max(1, -(-max(lens) // 64)) + slack, dtype)
    n = max(max(lens), 1)
    k, v = rows(rng, B, layers, n, Hkv, D, dtype=dtype), rows(rng, B, layers, n, Hkv, D, dtype=dtype)
    c.append(k, v, i32(lens))
    kr, vr = c.read(None, n)
    c.check_error()
    return c, f64(kr), f64(vr)


def check(out, ref, vmax, dtype, what):
    out, ref = np.asarray(out), np.asarray(ref)
    if dtype == "f32":
        tol = np.full(ref.shape, 3e-5 * vmax)
    else:
        tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * vmax
    assert np.array_equal(np.isnan(out), np.isnan(ref)), what
    ok = np.isnan(ref) | (np.abs(out - ref) <= tol)
    assert ok.all(), (what, float(np.nanmax(np.abs(out - ref))), vmax, np.argwhere(~ok)[:4].tolist())


def run_case(rng, Hq, Hkv, D, lens, trees, dtype, layers=1, new=True, max_len=None, qgain=1.5, poison=()):
    """One call against the oracle, every element.  poison: (request, node) whose new rows are NaN or infinite."""
    B = len(lens)
    c, kr, vr = filled(rng, Hq, Hkv, D, lens, layers, dtype)
    n = 1 if trees is None else max(len(t) for t in trees)
    q = (qgain * rows(rng, B, layers, n, Hq, D, dtype="f32")).to(DT[dtype])
    kn, vn = rows(rng, B, layers, n, Hkv, D, dtype=dtype), rows(rng, B, layers, n, Hkv, D, dtype=dtype)
    vmax = max(float(vn.abs().max()), float(np.abs(vr).max()) if vr.size else 0.0)
    for i, (b, node) in enumerate(poison):
        kn[b, :, node] = float("nan") if i % 2 else float("inf")
        vn[b, :, node] = float("-inf") if i % 2 else float("nan")
    from gated_deltanet_tree_gb300.runtime import DeviceSchedule
    sched = None if trees is None else DeviceSchedule(trees, n, "cuda")
    out = torch.full((B, layers, n, Hq, D), 7.0, dtype=DT[dtype], device="cuda")
    for _ in range(2):       # the second call finds the workspace as the first left it
        c.attention(q, kn if new else None, vn if new else None, out, sched=sched,
                    max_len=max(lens) if max_len is None else max_len)
    c.check_error()
    assert not c.workspace[:65536].any()
    for b in range(B):
        tree = np.array([-1]) if trees is None else trees[b]
        m = len(tree)
        for l in range(layers):
            with np.errstate(invalid="ignore"):
                ref = K.tree_attention(f64(q[b, l, :m]), kr[b, l, :lens[b]], vr[b, l, :lens[b]],
                                       f64(kn[b, l, :m]) if new else None, f64(vn[b, l, :m]) if new else None, tree,
                                       c.dims.scale)
            check(f64(out[b, l, :m]), ref, vmax, dtype, (Hq, Hkv, D, b, l))
        assert (out[b, :, m:] == 7.0).all()
    return out


HEADS = [(24, 4, 256), (8, 1, 256), (32, 8, 128), (5, 5, 128), (14, 2, 128), (8, 4, 64), (3, 1, 64)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_attention_trees(Hq, Hkv, D, dtype):
    """Ragged trees (one node to many) over lengths around words, pages and tiles; zero and one token."""
    rng = np.random.default_rng(Hq + D)
    lens = [0, 1, 63, 64, 65, 129, 200]
    trees = [S.random_tree(m, rng) for m in (1, 2, 3, 11, 7, 22, 5)]
    run_case(rng, Hq, Hkv, D, lens, trees, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
def test_attention_single_tokens(Hq, Hkv, D, dtype):
    rng = np.random.default_rng(Hq + D + 1)
    run_case(rng, Hq, Hkv, D, [0, 1, 7, 64, 100, 191, 333], None, dtype)
    run_case(rng, Hq, Hkv, D, [0, 1, 7, 64, 100, 191, 333], None, dtype, new=False)


@pytest.mark.parametrize("Hq,Hkv,D", [(24, 4, 256), (32, 8, 128), (8, 4, 64)])
@pytest.mark.parametrize("shape", ["chain64", "wide64", "star", "tree33"])
def test_attention_large_trees(Hq, Hkv, D, shape):
    rng = np.random.default_rng(D)
    tree = {"chain64": S.chain_tree(64), "wide64": S.ddtree(64, 8, 16, rng), "tree33": S.random_tree(33, rng),
            "star": np.array([-1] + [0] * 63)}[shape]
    run_case(rng, Hq, Hkv, D, [300, 1], [tree, tree[:max(1, len(tree) // 2)]], "bf16")


@pytest.mark.parametrize("trees", [True, False])
def test_attention_long_and_split(trees):
    """Enough pages that the work is split along the tokens; sharp and flat rows; several layers."""
    rng = np.random.default_rng(8)
    t = [S.random_tree(6, rng), S.random_tree(9, rng)] if trees else None
    run_case(rng, 6, 1, 256, [4000, 1537], t, "bf16")
    run_case(rng, 6, 1, 256, [1990, 77], t, "bf16", layers=3, qgain=6.0)
    run_case(rng, 8, 2, 128, [5000, 65], t, "bf16", qgain=0.01)
    run_case(rng, 8, 2, 64, [1500, 0], t, "f32", layers=2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_ignores_a_wrong_length_hint(dtype):
    rng = np.random.default_rng(9)
    t = [S.random_tree(5, rng), S.random_tree(4, rng)]
    for hint in (0, 1, 64, 700, 100000):
        run_case(rng, 8, 2, 128, [700, 130], t, dtype, max_len=hint)
        run_case(rng, 8, 2, 128, [700, 130], None, dtype, max_len=hint)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv,D", [(24, 4, 256), (8, 2, 128), (4, 2, 64)])
def test_attention_unseen_rows_do_not_reach_a_node(Hq, Hkv, D, dtype):
    """NaN and infinities in drafted rows: only their descendants (and themselves) see them."""
    rng = np.random.default_rng(10)
    trees = [np.array([-1, 0, 0, 1, 2, 2, 0, 6]), S.random_tree(40, rng)]
    run_case(rng, Hq, Hkv, D, [70, 10], trees, dtype, poison=[(0, 2), (0, 6), (1, 39), (1, 20)])


def test_attention_poisoned_cache_rows_reach_their_request_only():
    rng = np.random.default_rng(11)
    c, _, _ = filled(rng, 8, 2, 128, [130, 70], 1, "bf16")
    bad = rows(rng, 2, 1, 1, 2, 128, dtype="bf16")
    bad[0, 0, 0, 1, 3] = float("inf")
    c.append(bad, bad, i32([1, 1]))
    q = rows(rng, 2, 1, 1, 8, 128, dtype="bf16")
    out = torch.zeros_like(q)
    c.attention(q, None, None, out)
    assert torch.isnan(out[0, 0, 0, 4:]).all()
    assert not torch.isnan(out[0, 0, 0, :4]).any() and not torch.isnan(out[1]).any()


def test_attention_large_scores_and_scales():
    """Scores far apart, and rows whose size is at fp16's and bf16's limits."""
    rng = np.random.default_rng(12)
    B, Hq, Hkv, D = 2, 6, 1, 128
    for gain, kgain in ((200.0, 1.0), (1e-4, 1e3), (3e4, 1e-4), (1e-12, 1.0), (1e12, 1e-3)):
        c = make_cache(Hq, Hkv, D, B, 1, 5, "bf16")
        k = (rows(rng, B, 1, 300, Hkv, D, dtype="f32") * kgain).bfloat16()
        v = rows(rng, B, 1, 300, Hkv, D, dtype="bf16")
        c.append(k, v, i32([300, 90]))
        kr, vr = c.read(None, 300)
        for n, tree in ((1, None), (12, S.chain_tree(12))):
            from gated_deltanet_tree_gb300.runtime import DeviceSchedule
            q = (rows(rng, B, 1, n, Hq, D, dtype="f32") * gain).bfloat16()
            out = torch.zeros_like(q)
            sched = None if tree is None else DeviceSchedule([tree] * B, n, "cuda")
            c.attention(q, None, None, out, sched=sched, max_len=300)
            c.check_error()
            # scores grow with the gain: their rounding (S 2^-22) widens the weights' error
            top = float((q.float().norm(dim=-1).max() * kr.norm(dim=-1).max()) * c.dims.scale)
            vmax = float(vr.abs().max())
            for b, L in enumerate((300, 90)):
                ref = K.tree_attention(f64(q[b, 0]), f64(kr[b, 0, :L]), f64(vr[b, 0, :L]), None, None,
                                       [-1] * n, c.dims.scale)
                tol = 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + min(2.0, top * 2.0 ** -20)) * vmax
                assert (np.abs(f64(out[b, 0]) - ref) <= tol).all(), (gain, kgain, n)


def test_attention_strided_rows_and_another_stream():
    rng = np.random.default_rng(13)
    B, Hq, Hkv, D, n = 2, 8, 2, 128, 5
    tree = S.random_tree(n, rng)
    c, kr, vr = filled(rng, Hq, Hkv, D, [90, 10], 1, "bf16")
    wide = rows(rng, B, 1, n, Hq + 2 * Hkv, D, dtype="bf16")
    q, kn, vn = wide[..., :Hq, :], wide[..., Hq:Hq + Hkv, :], wide[..., Hq + Hkv:, :]
    from gated_deltanet_tree_gb300.runtime import DeviceSchedule
    sched = DeviceSchedule([tree] * B, n, "cuda")
    out = torch.zeros(B, 1, n, Hq, D, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.attention(q, kn, vn, out, sched=sched, stream=side)
    side.synchronize()
    vmax = float(wide.abs().max())
    for b, L in enumerate((90, 10)):
        ref = K.tree_attention(f64(q[b, 0]), kr[b, 0, :L], vr[b, 0, :L], f64(kn[b, 0]), f64(vn[b, 0]), tree,
                               c.dims.scale)
        check(f64(out[b, 0]), ref, vmax, "bf16", b)


def test_attention_device_errors():
    from gated_deltanet_tree_gb300 import _native as N
    rng = np.random.default_rng(14)
    for n in (1, 8, 40):
        c, _, _ = filled(rng, 6, 1, 128, [70, 70], 1, "bf16")
        from gated_deltanet_tree_gb300.runtime import DeviceSchedule
        sched = DeviceSchedule([S.chain_tree(n)] * 2, n, "cuda")
        q = rows(rng, 2, 1, n, 6, 128, dtype="bf16")
        kn = rows(rng, 2, 1, n, 1, 128, dtype="bf16")
        good = torch.zeros_like(q)
        c.attention(q, kn, kn, good, sched=sched)
        c.check_error()

        def refused(status):
            out = torch.full_like(q, 3.0)
            c.attention(q, kn, kn, out, sched=sched)
            with pytest.raises(N.GdnError) as e:
                c.check_error()
            assert e.value.status == status
            assert torch.equal(out[1], good[1])          # the other request is served

        keep = c.seq_len.clone()
        for bad in (-1, 64 * c.pages_max + 1):
            c.seq_len[0] = bad
            refused(N.GDN_ERR_CACHE)
        c.seq_len.copy_(keep)
        keep = c.page_table.clone()
        for bad in (-1, c.pool.shape[1]):
            c.page_table[0, 0] = bad
            refused(N.GDN_ERR_CACHE)
        c.page_table.copy_(keep)
        words = sched.words.clone()
        sched.words[0, 0] = n + 1
        refused(N.GDN_ERR_SCHEDULE)
        sched.words.copy_(words)
        if n > 1:
            sched.words[0, 5 + 1] = 1                    # a node that is its own parent
            out = torch.zeros_like(q)
            c.attention(q, kn, kn, out, sched=sched)
            with pytest.raises(N.GdnError) as e:
                c.check_error()
            assert e.value.status == N.GDN_ERR_SCHEDULE


# ---- acceptance -----------------------------------------------------------------------------------------------------

def accept_case(rng, B, n, V, dtype, temps, draft=None, trees=None, tokens=None, logits=None, pad=0):
    from gated_deltanet_tree_gb300 import runtime as R
    trees = trees or [S.random_tree(int(rng.integers(1, n + 1)), rng) for _ in range(B)]
    z = torch.from_numpy((rng.standard_normal((B, n, V + pad)) * 2).astype(np.float32))
    q = None
    if tokens is None:
        tokens = rng.integers(0, V, (B, n))
        for b in range(B):
            for i in range(1, len(trees[b])):      # likely tokens, boosted in their parent's row
                if rng.random() < 0.8:
                    z[b, trees[b][i], tokens[b, i]] += np.log(V) + 1.5
    if logits is not None:
        z = logits
    z = z.to(DT[dtype]).cuda()
    if draft is not None:
        q = torch.softmax(z.float()[..., :V] + 0.7 * torch.randn(B, n, V, device="cuda"), -1)
        if pad:
            q = torch.nn.functional.pad(q, (0, pad))
        q = q.to(DT[draft])
        for b in range(B):
            for i in range(1, len(trees[b])):
                pq = f64(q[b, trees[b][i], :V])
                tokens[b, i] = rng.choice(V, p=pq / pq.sum())
    u = torch.from_numpy(rng.random((B, n)).astype(np.float32)).cuda()
    g = torch.from_numpy(-np.log(-np.log(rng.random((B, V)))).astype(np.float32)).cuda()
    t = torch.tensor(temps, dtype=torch.float32, device="cuda")
    acc = R.TreeAcceptor(B, n, V)
    path, length, nxt = acc.accept(R.DeviceSchedule(trees, n, "cuda"), z[..., :V], i32(tokens), u, g, t,
                                   draft_probs=None if q is None else q[..., :V])
    taken = 0
    for b in range(B):
        m = len(trees[b])
        want, token = A.accept(trees[b].tolist(), tokens[b].tolist(), f64(z[b, :m, :V]), f64(u[b]), f64(g[b]),
                               float(t[b]), None if q is None else f64(q[b, :m, :V]))
        L = int(length[b])
        assert path[b, :L].tolist() == want and int(nxt[b]) == token, b
        assert (path[b, L:] == -1).all()
        taken += L
    return acc, taken


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V", [1, 7, 257, 1000, 4099, 20001])
def test_accept_chosen_drafts(V, dtype):
    rng = np.random.default_rng(V)
    B = 24
    temps = [0.0 if b % 4 == 3 else 0.5 + 0.1 * b for b in range(B)]
    acc, taken = accept_case(rng, B, 22, V, dtype, temps)
    acc.check_error()
    assert V < 100 or taken > B + 8


@pytest.mark.parametrize("draft", ["bf16", "f32"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,pad", [(64, 0), (1001, 0), (1001, 7), (9001, 0)])
def test_accept_sampled_drafts(V, pad, dtype, draft):
    """Chains and trees with sampled siblings (several rejections at a node)."""
    rng = np.random.default_rng(V + pad)
    B = 24
    trees = [S.chain_tree(int(rng.integers(1, 10))) if b % 2 else S.random_tree(9, rng) for b in range(B)]
    trees[0] = np.array([-1] + [0] * 8)
    trees[2] = np.array([-1] + [0] * 8)
    temps = [1.0 if b % 5 else 0.0 for b in range(B)]
    acc, _ = accept_case(rng, B, 9, V, dtype, temps, draft=draft, trees=trees, pad=pad)
    acc.check_error()


@pytest.mark.parametrize("B,n,V", [(1, 22, 131072), (3, 64, 50001), (70, 22, 32000), (1, 1, 150001)])
def test_accept_large(B, n, V):
    rng = np.random.default_rng(B + n)
    acc, _ = accept_case(rng, B, n, V, "bf16", [0.9] * B)
    acc.check_error()
    acc, _ = accept_case(rng, B, n, V, "bf16", [0.0] * B)
    acc.check_error()


def test_accept_ties_duplicates_and_masks():
    rng = np.random.default_rng(20)
    B, n, V = 8, 6, 300
    z = torch.zeros(B, n, V)
    z[:, :, 17] = z[:, :, 5] = z[:, :, 250] = 4.0          # equal largest: the lowest index
    z[:, 0, 100:] = -float("inf")                          # masked tokens are never drawn
    star = np.array([-1, 0, 0, 0, 0, 0])
    tokens = np.tile([0, 17, 17, 120, 5, 5], (B, 1))       # a repeat, a masked one
    acc, _ = accept_case(rng, B, n, V, "f32", [0.0, 0.0] + [1.0] * 6, trees=[star] * B, tokens=tokens, logits=z)
    acc.check_error()
    assert acc.path[0].tolist()[:2] == [0, 4]
    tokens[:, 1], tokens[:, 2] = -1, V                      # out of range: never accepted
    acc, _ = accept_case(rng, B, n, V, "f32", [0.0, 0.0] + [1.0] * 6, trees=[star] * B, tokens=tokens, logits=z)
    acc.check_error()


def test_accept_reports_rows_without_a_distribution():
    from gated_deltanet_tree_gb300 import _native as N
    rng = np.random.default_rng(21)
    n, V = 5, 500
    for temp in (0.0, 1.0):
        for bad in (float("nan"), float("inf"), "none"):
            z = torch.from_numpy(rng.standard_normal((2, n, V)).astype(np.float32))
            tokens = np.tile([0, 3, 4, 5, 6], (2, 1))
            for i in range(n - 1):
                z[:, i, tokens[0, i + 1]] = 60.0
            if bad == "none":
                z[0, 2] = -float("inf")
            else:
                z[0, 2, 499] = bad
            acc, _ = accept_case(rng, 2, n, V, "f32", [temp] * 2, trees=[S.chain_tree(n)] * 2, tokens=tokens, logits=z)
            with pytest.raises(N.GdnError) as e:
                acc.check_error()
            assert e.value.status == N.GDN_ERR_LOGITS
            assert acc.len.tolist() == [3, 5] and int(acc.next[0]) == -1
    from gated_deltanet_tree_gb300 import runtime as R
    for temp in (-1.0, float("nan"), float("inf")):
        acc = R.TreeAcceptor(1, n, V)
        u, g = torch.zeros(1, n, device="cuda"), torch.zeros(1, V, device="cuda")
        acc.accept(R.DeviceSchedule([S.chain_tree(n)], n, "cuda"), z[:1].cuda(), i32(tokens[:1]), u, g,
                   torch.tensor([temp], device="cuda"))
        with pytest.raises(N.GdnError) as e:
            acc.check_error()
        assert e.value.status == N.GDN_ERR_LOGITS and int(acc.next[0]) == -1 and int(acc.len[0]) == 1


def test_accept_greedy_needs_no_numbers_and_feeds_the_commit():
    """path and len go into gdn_commit_fold and the cache append as they are."""
    from gated_deltanet_tree_gb300 import runtime as R
    from harness import GpuSession, WorkloadPlan
    w = S.workload(1).replace(steps=1)
    plan = WorkloadPlan(w)
    gs = GpuSession(w, plan)
    gs.verify(0)
    rng = np.random.default_rng(22)
    V, B, n = 100, w.B, w.n_max
    tokens = np.tile(np.arange(n), (B, 1))
    z = torch.from_numpy(rng.standard_normal((B, n, V)).astype(np.float32)).cuda()
    for b in range(B):
        for i, p in enumerate(plan.trees[0][b]):
            if p >= 0:
                z[b, p, i] = 50.0 - i                       # the lowest child wins
    acc = R.TreeAcceptor(B, n, V)
    path, length, _ = acc.accept(gs.schedule(0), z, i32(tokens))
    assert (length > 1).all()
    gs.ver.commit(gs.schedule(0), path, length)
    c = make_cache(4, 2, 64, B, 1, 1, "bf16")
    k = rows(rng, B, 1, n, 2, 64, dtype="bf16")
    c.append(k, k, length, path=path)
    gs.finish()
    gs.ver.check_error()
    acc.check_error()
    c.check_error()
    assert torch.equal(c.seq_len, length)


# ---- refusals before anything is launched ---------------------------------------------------------------------------

def test_wrapper_refusals():
    from gated_deltanet_tree_gb300 import runtime as R
    rng = np.random.default_rng(23)
    c = make_cache(4, 2, 64, 2, 1, 2, "bf16")
    k = rows(rng, 2, 1, 3, 2, 64, dtype="bf16")
    q = rows(rng, 2, 1, 1, 4, 64, dtype="bf16")
    out = torch.zeros_like(q)
    for bad in (lambda: c.append(k.float(), k, i32([1, 1])), lambda: c.append(k, k[:, :, :2], i32([1, 1])),
                lambda: c.append(k, k, i32([1])), lambda: c.append(k, k, i32([1, 1]), path=i32([0, 1])),
                lambda: c.append(k.transpose(3, 4), k, i32([1, 1])), lambda: c.attention(q, k, None, out),
                lambda: c.attention(q, k, k, out), lambda: c.attention(q.half(), None, None, out),
                lambda: c.attention(q, None, None, out[..., :32]),
                lambda: R.KV4Cache(c.dims, c.pool[..., :64], c.page_table, c.seq_len),
                lambda: R.KV4Cache(c.dims, c.pool, c.page_table.long(), c.seq_len),
                lambda: R.make_attn_dims(4, 2, 64, dtype=torch.float16)):
        with pytest.raises((ValueError, TypeError)):
            bad()


@pytest.mark.parametrize("Hq,Hkv,D,n", [(4, 4, 256, 8), (2, 1, 256, 4), (8, 8, 128, 7), (8, 2, 128, 2), (2, 2, 64, 8),
                                        (8, 4, 64, 4)])
def test_attention_small_trees(Hq, Hkv, D, n):
    """Trees of at most eight rows a kv head, some of them long enough to be split, with unseen NaN and infinite rows."""
    rng = np.random.default_rng(Hq + D + n)
    trees = [S.random_tree(m, rng) for m in (n, 1, max(1, n // 2), n, n)]
    run_case(rng, Hq, Hkv, D, [0, 1, 65, 130, 3000], trees, "bf16")
    run_case(rng, Hq, Hkv, D, [40, 64, 2300], [np.array([-1] + [0] * (n - 1))] * 3, "bf16", layers=2,
             poison=[(0, n - 1), (2, 1)])
    run_case(rng, Hq, Hkv, D, [0, 600], [S.chain_tree(n)] * 2, "bf16", new=False)


def test_attention_many_heads_and_layers():
    """More items a request than the 128-row kernel has records for: tiles of eight rows take the call."""
    rng = np.random.default_rng(30)
    B, layers, Hq, Hkv, D, n = 1, 70, 256, 64, 64, 6
    c = make_cache(Hq, Hkv, D, B, layers, 2, "bf16")
    k = rows(rng, B, layers, 70, Hkv, D, dtype="bf16")
    c.append(k, k, i32([70]))
    kr, vr = c.read(None, 70)
    tree = S.random_tree(n, rng)
    from gated_deltanet_tree_gb300.runtime import DeviceSchedule
    q, kn = rows(rng, B, layers, n, Hq, D, dtype="bf16"), rows(rng, B, layers, n, Hkv, D, dtype="bf16")
    out = torch.zeros_like(q)
    c.attention(q, kn, kn, out, sched=DeviceSchedule([tree], n, "cuda"), max_len=70)
    c.check_error()
    vmax = max(float(kn.abs().max()), float(vr.abs().max()))
    for l, h in ((0, 0), (31, 40), (69, 63)):
        G = Hq // Hkv
        ref = K.tree_attention(f64(q[0, l, :, h * G:(h + 1) * G]), f64(kr[0, l, :, h:h + 1]), f64(vr[0, l, :, h:h + 1]),
                               f64(kn[0, l, :, h:h + 1]), f64(kn[0, l, :, h:h + 1]), tree, c.dims.scale)
        check(f64(out[0, l, :, h * G:(h + 1) * G]), ref, vmax, "bf16", (l, h))


def test_example_runs_the_operators_together():
    """The example's steps, and its last step's attention and acceptance against the oracles."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import hybrid_step
    lines = []
    model = hybrid_step.main(steps=3, show=lines.append)
    assert len(lines) == 4 and torch.isfinite(model.state).all()
    for b in range(model.B):
        L = int(model.acceptor.len[b])
        path = model.acceptor.path[b]
        assert 1 <= L <= model.n_max and int(path[0]) == 0 and (path[L:] == -1).all()
        assert 0 <= int(model.acceptor.next[b]) < model.V


@pytest.mark.parametrize("Hq,Hkv,D", [(24, 4, 256), (32, 8, 128), (32, 8, 64), (42, 7, 128)])
def test_attention_many_items_shared_between_ctas(Hq, Hkv, D):
    """More items than a quarter of the CTAs, most of them split: odd numbers of pages, ends inside a page, unseen NaN
    and infinite rows in split items, tiles that a request does not fill, no new rows."""
    rng = np.random.default_rng(Hq + Hkv + D)
    lens = [700, 65, 1, 0, 330, 129, 512, 640, 200, 64, 450, 1090]
    trees = [S.random_tree(m, rng) for m in (22, 30, 5, 64, 22, 1, 21, 33, 8, 12, 43, 22)]
    run_case(rng, Hq, Hkv, D, lens, trees, "bf16")
    run_case(rng, Hq, Hkv, D, lens, trees, "bf16", poison=[(0, 21), (7, 30), (11, 1)])
    run_case(rng, Hq, Hkv, D, lens[:8], trees[:8], "bf16", new=False, max_len=0)


def quantised(x):
    """Values of rows [..., D] after the cache, by the formula in 64 bits."""
    g = x.double().reshape(*x.shape[:-1], -1, 32)
    a = g.abs()
    first = torch.where(a == a.amax(-1, keepdim=True), torch.arange(32, device=x.device), 99).amin(-1, keepdim=True)
    m = g.gather(-1, first)
    d = (m * -0.125).float().bfloat16().float().clamp(-2720, 2720).half().double()
    n = torch.where(d == 0, 0.0, torch.clamp(torch.round(g / torch.where(d == 0, 1.0, d)), -8, 7))
    return (n * d).reshape(x.shape).float()


@pytest.mark.parametrize("D", [64, 256])
def test_append_bf16_codes_are_the_quotients(D):
    """bf16 rows of any bits over 40 exponents, and rows of a few values of both signs (ties of the largest magnitude and
    of the rounding; zeros of both signs): every value exact."""
    g = torch.Generator(device="cuda").manual_seed(D)
    L = 64 * 512

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=torch.int32)

    top = ints(100, 140, L, D // 32, 1).expand(L, D // 32, 32).reshape(L, D)
    bits = (ints(0, 65536, L, D) & 0x807F) | ((top - ints(0, 5, L, D)) << 7)
    some = torch.tensor([0.0, -0.0, 0.5, -0.5, 1.5, -1.5, 3.5, -3.5, 7.0, 7.5, -7.5, 8.0, -8.0], device="cuda")
    for x in ((bits << 16).view(torch.float32).bfloat16(), some[ints(0, 13, L, D).long()].bfloat16(),
              some[ints(0, 2, L, D).long()].bfloat16()):
        c = make_cache(1, 1, D, 1, 1, L // 64, "bf16")
        c.append(x.view(1, 1, L, 1, D), -x.view(1, 1, L, 1, D), i32([L]))
        k, v = c.read(None, L)
        c.check_error()
        assert torch.equal(k.view(L, D), quantised(x))
        assert torch.equal(v.view(L, D), quantised(-x))


@pytest.mark.parametrize("n", [1, 22])
def test_cache_pages_beyond_four_gigabytes(n):
    """The same call over pages at the end of a pool of 5 GB and over a small pool: equal to the last bit."""
    from gated_deltanet_tree_gb300 import runtime as R
    rng = np.random.default_rng(n)
    Hq, Hkv, D, L = 24, 4, 256, 150
    k, v = rows(rng, 1, 1, L, Hkv, D, dtype="bf16"), rows(rng, 1, 1, L, Hkv, D, dtype="bf16")
    q, kn = rows(rng, 1, 1, n, Hq, D, dtype="bf16"), rows(rng, 1, 1, n, Hkv, D, dtype="bf16")
    tree = S.random_tree(n, rng)
    results = []
    for pages in (3, 70000):
        dims = R.make_attn_dims(Hq, Hkv, D)
        pool = torch.zeros(1, pages, Hkv, 72 * D, dtype=torch.uint8, device="cuda")
        c = R.KV4Cache(dims, pool, i32([[pages - 1, pages - 3, pages - 2]]), i32([0]))
        c.append(k, v, i32([L]))
        out = torch.zeros_like(q)
        c.attention(q, kn, kn, out, sched=None if n == 1 else R.DeviceSchedule([tree], n, "cuda"), max_len=L)
        c.check_error()
        results.append((out, *c.read(None, L), pool[0, -3:].clone()))
        assert not pool[0, :-3].any()
    for a, b in zip(*results):
        assert torch.equal(a, b)
