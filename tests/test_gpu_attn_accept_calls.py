"""The cache and acceptance calls as programs make them on a GPU: streams, CUDA graphs, refusals between calls, and the
paths of the kernels that only large batches, many launches or long contexts reach.  Tolerances as in
test_gpu_attn_accept.py unless a test derives its own."""
import numpy as np
import pytest
import torch

import synthetic as S
from oracle import accept_oracle as A
from oracle import kv4_oracle as K
from test_gpu_attn_accept import DT, accept_case, built, check, f64, filled, i32, make_cache, rows, run_case  # noqa: F401

pytestmark = pytest.mark.gpu


def schedule(trees, n):
    from gated_deltanet_tree_gb300.runtime import DeviceSchedule
    return DeviceSchedule(trees, n, "cuda")


def tree_reference(c, q, kr, vr, kn, vn, lens, trees):
    return [K.tree_attention(f64(q[b, 0, :len(t)]), kr[b, 0, :lens[b]], vr[b, 0, :lens[b]], f64(kn[b, 0, :len(t)]),
                             f64(vn[b, 0, :len(t)]), t, c.dims.scale) for b, t in enumerate(trees)]


# ---- streams and graphs ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("n", [1, 6])
def test_first_call_on_a_side_stream_while_the_current_one_is_busy(n):
    """Items shared by several CTAs (their counters and partial results are in the workspace) in a cache's first call,
    on another stream than the one the cache was made on, which is busy all the while."""
    rng = np.random.default_rng(40 + n)
    lens, trees = [3000, 1700], [S.random_tree(n, rng), S.random_tree(n, rng)]
    filled_c, kr, vr = filled(rng, 24, 4, 256, lens, 1, "bf16")
    q, kn, vn = (rows(rng, 2, 1, n, h, 256, dtype="bf16") for h in (24, 4, 4))
    sched = schedule(trees, n)
    ref = tree_reference(filled_c, q, kr, vr, kn, vn, lens, trees)
    vmax = max(float(vn.abs().max()), float(np.abs(vr).max()))
    from gated_deltanet_tree_gb300.runtime import KV4Cache
    out = torch.full_like(q, 7.0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    junk = torch.full((64 << 20,), 0xA5, dtype=torch.uint8, device="cuda")     # what an unfilled workspace would hold
    del junk
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                                              # ends by itself, about 10 ms
    c = KV4Cache(filled_c.dims, filled_c.pool, filled_c.page_table, filled_c.seq_len)
    torch.cuda._sleep(20_000_000)
    c.attention(q, kn, vn, out, sched=sched, max_len=3000, stream=side)
    side.synchronize()
    got = out.clone()
    torch.cuda.synchronize()
    c.check_error()
    assert not c.workspace[:65536].any()
    for b in range(2):
        check(f64(got[b, 0]), ref[b], vmax, "bf16", b)


@pytest.mark.parametrize("n", [1, 22])
def test_captured_steps_replay_after_larger_calls(n):
    """A graph of a step (attention, acceptance, append of what was accepted) holds its buffers: larger calls on the same
    cache in between change neither them nor its results, and a replay follows the cache's lengths."""
    from gated_deltanet_tree_gb300 import runtime as R
    rng = np.random.default_rng(42)
    B, Hq, Hkv, D, V = 2, 6, 2, 128, 20001
    c, _, _ = filled(rng, Hq, Hkv, D, [500, 90], 1, "bf16", slack=2)
    acc = R.TreeAcceptor(B, n, V)
    trees = [S.random_tree(n, rng) for _ in range(B)]
    sched = schedule(trees, n)
    q, k, v = (rows(rng, B, 1, n, h, D, dtype="bf16") for h in (Hq, Hkv, Hkv))
    tokens = rng.integers(0, V, (B, n))

    def logits():
        z = rng.standard_normal((B, n, V)).astype(np.float32)
        for b in range(B):
            for i in range(1, n):
                if rng.random() < 0.5:
                    z[b, trees[b][i], tokens[b, i]] += 20.0
        return torch.from_numpy(z).cuda()

    z, tok, out = logits(), i32(tokens), torch.zeros_like(q)

    def step():
        c.attention(q, k, v, out, sched=sched)
        path, length, _ = acc.accept(sched, z, tok)
        c.append(k, v, length, path=path)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            step()
    torch.cuda.current_stream().wait_stream(side)
    big, kb = rows(rng, B, 1, 64, Hq, D, dtype="bf16"), rows(rng, B, 1, 64, Hkv, D, dtype="bf16")
    bigger = schedule([S.random_tree(64, rng)] * B, 64)
    for i in range(3):
        c.attention(big, kb, kb, torch.zeros_like(big), sched=bigger, max_len=0)
        junk = [torch.full((8 << 20,), 0xA5, dtype=torch.uint8, device="cuda") for _ in range(8)]   # freed memory's next user
        for t in (q, k, v):
            t.copy_(rows(rng, *t.shape, dtype="bf16"))
        z.copy_(logits())
        lens = c.seq_len.tolist()
        kr, vr = (f64(t) for t in c.read(None, max(lens)))
        graph.replay()
        torch.cuda.synchronize()
        assert all(bool((t == 0xA5).all()) for t in junk)
        c.check_error()
        acc.check_error()
        ref = tree_reference(c, q, kr, vr, k, v, lens, trees)
        for b in range(B):
            check(f64(out[b, 0]), ref[b], max(float(v.abs().max()), float(np.abs(vr).max())), "bf16", (i, b))
            path, token = A.accept(trees[b].tolist(), tokens[b].tolist(), f64(z[b]), None, None, 0.0)
            assert acc.path[b, :len(path)].tolist() == path and int(acc.next[b]) == token
            assert int(c.seq_len[b]) == lens[b] + len(path) == lens[b] + int(acc.len[b])


def test_read_on_a_side_stream_keeps_off_the_current_streams_memory():
    """A block that the current stream has still to write to, freed just before the read: its next user is of that stream."""
    rng = np.random.default_rng(44)
    c, kr, vr = filled(rng, 4, 4, 256, [2000, 1500], 2, "bf16")
    side = torch.cuda.Stream()
    for handle in (side, side.cuda_stream):
        torch.cuda.synchronize()
        blocks = [torch.empty(2, 2, 2000, 4, 256, device="cuda") for _ in range(4)]       # of the size of k and of v
        torch.cuda._sleep(40_000_000)                # ends by itself, about 20 ms
        for x in blocks:
            x.fill_(77.0)
        del blocks, x
        k, v = c.read(None, 2000, stream=handle)
        side.synchronize()
        torch.cuda.synchronize()
        assert np.array_equal(f64(k), kr) and np.array_equal(f64(v), vr)
    c.check_error()


# ---- refusals between calls -----------------------------------------------------------------------------------------

def test_a_refused_call_leaves_nothing_behind():
    """Rows of a fused projection whose stride is no multiple of 16 bytes are refused; the calls after that are served."""
    from gated_deltanet_tree_gb300 import _native as N
    rng = np.random.default_rng(43)
    Hq, Hkv, D, n = 8, 2, 64, 5
    c, kr, vr = filled(rng, Hq, Hkv, D, [90], 1, "bf16", slack=1)
    flat = rows(rng, 1, 1, n, (Hq + 2 * Hkv) * D + 4, dtype="bf16")                  # (four gate columns)
    wide = flat[..., :-4].unflatten(-1, (Hq + 2 * Hkv, D))
    q, k, v = wide[..., :Hq, :], wide[..., Hq:Hq + Hkv, :], wide[..., Hq + Hkv:, :]
    tree = S.random_tree(n, rng)
    out, sched, one = torch.zeros(1, 1, n, Hq, D, dtype=torch.bfloat16, device="cuda"), schedule([tree], n), i32([1])
    for bad in (lambda: c.attention(q, k, v, out, sched=sched), lambda: c.attention(q, None, None, out, sched=sched),
                lambda: c.append(k, v, one)):
        with pytest.raises(N.GdnError) as e:
            bad()
        assert e.value.status == N.GDN_ERR_INVALID_ARG
        kc, vc = k.contiguous(), v.contiguous()
        c.attention(q.contiguous(), kc, vc, out, sched=sched)
        ref = tree_reference(c, q, kr, vr, k, v, [90], [tree])
        check(f64(out[0, 0]), ref[0], max(float(v.abs().max()), float(np.abs(vr).max())), "bf16", "after a refusal")
        again = c.read(None, 90)
        assert np.array_equal(f64(again[0]), kr) and np.array_equal(f64(again[1]), vr)
    c.append(kc, vc, one)
    c.check_error()
    assert int(c.seq_len[0]) == 91


@pytest.mark.parametrize("n", [1, 6])
def test_calls_after_a_timeout(n):
    """The counters as a launch leaves them whose later CTAs saw the time-out flag: some have counted, some have not.
    While the flag is set a call does nothing; once it has been reported the next call is right."""
    from gated_deltanet_tree_gb300 import _native as N
    rng = np.random.default_rng(45)
    lens, trees = [3000, 1700], [S.random_tree(n, rng), S.random_tree(n, rng)]
    c, kr, vr = filled(rng, 24, 4, 256, lens, 1, "bf16")
    q, kn, vn = (rows(rng, 2, 1, n, h, 256, dtype="bf16") for h in (24, 4, 4))
    out, sched = torch.full_like(q, 7.0), schedule(trees, n)
    c.workspace[:65536].view(torch.int32)[:64:3] = 1
    c.err[0] = 4                                     # GDN_DEVERR_TIMEOUT
    c.attention(q, kn, vn, out, sched=sched)
    assert (out == 7.0).all()
    with pytest.raises(N.GdnError) as e:
        c.check_error()
    assert e.value.status == N.GDN_ERR_TIMEOUT
    c.attention(q, kn, vn, out, sched=sched)
    c.check_error()
    ref = tree_reference(c, q, kr, vr, kn, vn, lens, trees)
    for b in range(2):
        check(f64(out[b, 0]), ref[b], max(float(vn.abs().max()), float(np.abs(vr).max())), "bf16", b)


# ---- values at fp16's lower end -------------------------------------------------------------------------------------

@pytest.mark.parametrize("Hq,Hkv,D", [(24, 4, 256), (32, 4, 128), (32, 4, 64)])
@pytest.mark.parametrize("size", [1e-4, 1e-6, 1e-9, 1e-30])
def test_small_new_values_keep_their_bits(Hq, Hkv, D, size):
    """Values that are small throughout, with and without cached ones (of the same size, as the cache reads back)."""
    rng = np.random.default_rng(D)
    n, lens = 22, [0, 90, 0]
    c = make_cache(Hq, Hkv, D, 3, 1, 2, "bf16")
    k, v = rows(rng, 3, 1, 90, Hkv, D, dtype="bf16"), rows(rng, 3, 1, 90, Hkv, D, dtype="bf16")
    c.append(k, (size * v.float()).bfloat16(), i32(lens))
    kr, vr = (f64(t) for t in c.read(None, 90))
    trees = [S.random_tree(m, rng) for m in (22, 17, 9)]
    q, kn = rows(rng, 3, 1, n, Hq, D, dtype="bf16"), rows(rng, 3, 1, n, Hkv, D, dtype="bf16")
    vn = (size * rows(rng, 3, 1, n, Hkv, D, dtype="f32")).bfloat16()
    out = torch.zeros_like(q)
    c.attention(q, kn, vn, out, sched=schedule(trees, n))
    c.check_error()
    ref = tree_reference(c, q, kr, vr, kn, vn, lens, trees)
    for b, t in enumerate(trees):
        check(f64(out[b, 0, :len(t)]), ref[b], float(vn.abs().max()), "bf16", b)


@pytest.mark.parametrize("Hq,D,B,dtype", [(24, 256, 152, "bf16"), (24, 128, 152, "bf16"), (32, 64, 152, "bf16"),
                                          (8, 256, 304, "bf16"), (8, 64, 304, "bf16"), (8, 256, 304, "f32"),
                                          (8, 64, 304, "f32")])
@pytest.mark.parametrize("scale", [float(np.log(2.0)), 0.3, 0.0625])
@pytest.mark.parametrize("size", [2.0 ** 22, 2.0 ** 25, 1.5 * 2.0 ** 25, 1.25 * 2.0 ** 26, 2.0 ** 27, 2.0 ** 40])
def test_scores_whose_steps_are_larger_than_one(Hq, D, B, dtype, size, scale):
    """Scores of 2^22 to 2^40 (base 2), one page's a few steps above the others': equal values come out as they are,
    whatever the weights."""
    from gated_deltanet_tree_gb300 import runtime as R
    dims = R.make_attn_dims(Hq, 1, D, dtype=DT[dtype], scale=scale)
    pool = torch.zeros(1, 2, 1, 72 * D, dtype=torch.uint8, device="cuda")
    k = torch.zeros(1, 1, 128, 1, D, device="cuda")
    k[..., 0] = 1.0
    k[0, 0, 64:, 0, 40] = 1.0
    first = R.KV4Cache(dims, pool, i32([[0, 1]]), i32([0]))
    first.append(k.to(DT[dtype]), torch.ones_like(k).to(DT[dtype]), i32([128]))
    table = torch.zeros(B, 26, dtype=torch.int32, device="cuda")
    table[:, [12, 24]] = 1
    c = R.KV4Cache(dims, pool, table, i32([64 * 26] * B))
    q = torch.zeros(B, 1, 1, Hq, D, dtype=DT[dtype], device="cuda")
    for sign in (1.0, -1.0):
        for step in (4.0, 8.0, 16.0):
            q[..., 0], q[..., 40] = sign * size, step
            out = torch.zeros_like(q)
            c.attention(q, None, None, out, max_len=64 * 26)
            c.check_error()
            assert (out == 1.0).all() if dtype == "bf16" else ((out - 1.0).abs() <= 1e-6).all(), (sign, step)


# ---- long contexts --------------------------------------------------------------------------------------------------

def one_and_many(Hq, D, B, T, gap, dtype, dominant, tail):
    """B requests of T tokens: the first with score `gap` (nats), the others with score 0; their values (a number for
    each half of the channels, exact in the cache) -> the output and the definition's, [.., 2 halves].  Every page but
    the first is the same one of the pool."""
    from gated_deltanet_tree_gb300 import runtime as R
    dims = R.make_attn_dims(Hq, 1, D, dtype=DT[dtype], scale=1.0)
    pool = torch.zeros(1, 2, 1, 72 * D, dtype=torch.uint8, device="cuda")
    k = torch.zeros(1, 1, 128, 1, D, device="cuda")
    k[0, 0, 0, 0, 0] = 1.0
    v = torch.empty_like(k)
    for i in range(2):
        v[..., i * D // 2:(i + 1) * D // 2] = tail[i]
        v[0, 0, 0, 0, i * D // 2:(i + 1) * D // 2] = dominant[i]
    first = R.KV4Cache(dims, pool, i32([[0, 1]]), i32([0]))
    first.append(k.to(DT[dtype]), v.to(DT[dtype]), i32([128]))
    kr, vr = first.read(None, 128)
    first.check_error()
    assert torch.equal(kr, k) and torch.equal(vr, v)
    table = torch.ones(B, -(-T // 64), dtype=torch.int32, device="cuda")
    table[:, 0] = 0
    c = R.KV4Cache(dims, pool, table, i32([T] * B))
    q = torch.zeros(B, 1, 1, Hq, D, dtype=DT[dtype], device="cuda")
    q[..., 0] = gap
    assert float(q[0, 0, 0, 0, 0]) == gap
    out = torch.zeros_like(q)
    c.attention(q, None, None, out, max_len=T)
    c.check_error()
    w = (T - 1) * np.exp(-gap)
    return f64(out).reshape(B, Hq, 2, D // 2), (np.array(dominant) + w * np.array(tail))[:, None] / (1.0 + w)


@pytest.mark.parametrize("Hq,D,B", [(24, 256, 152), (24, 128, 152), (32, 64, 152), (8, 256, 304)])
def test_small_weights_of_a_long_tail_add_up(Hq, D, B):
    """A million tokens of weight 2^-27 each behind one of weight 1, every request in one CTA: 0.7% of the output."""
    for gap in (18.75, 15.0):
        out, ref = one_and_many(Hq, D, B, 1 << 20, gap, "bf16", (0.0, 1.0), (1.0, 0.0))
        tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -10
        assert (np.abs(out - ref) <= tol)[..., 0, :].all(), (gap, float(np.abs(out - ref)[..., 0, :].max()))


@pytest.mark.parametrize("Hq,D,B", [(8, 256, 152), (8, 128, 304), (8, 64, 304)])
def test_small_weights_of_a_long_tail_add_up_in_fp32(Hq, D, B):
    """The same in fp32, down to 2^-31 a token, with fp32's tolerance."""
    for gap in (21.75, 18.75, 15.0):
        out, ref = one_and_many(Hq, D, B, 1 << 20, gap, "f32", (0.0, 1.0), (1.0, 0.0))
        assert (np.abs(out - ref) <= 3e-5)[..., 0, :].all(), (gap, float(np.abs(out - ref)[..., 0, :].max()))


@pytest.mark.parametrize("Hq,D,B", [(24, 256, 152), (24, 128, 152), (32, 64, 152), (8, 256, 304)])
def test_a_long_tail_adds_to_a_dominating_value(Hq, D, B):
    """The same with one value everywhere, and with opposite ones: additions to a large sum, a million of them."""
    for gap in (18.75, 15.0):
        out, ref = one_and_many(Hq, D, B, 1 << 20, gap, "bf16", (1.0, 1.0), (1.0, -1.0))
        tol = 2.0 ** -8 * np.abs(ref) + 2.0 ** -10
        assert (np.abs(out - ref) <= tol).all(), (gap, [float(np.abs(out - ref)[..., i, :].max()) for i in range(2)])


LONG = [300001] * 30 + [131072, 131073, 262144, 262145, 270000, 5, 0, 64, 140000, 290017]


@pytest.mark.parametrize("Hq,D,B", [(8, 256, 152), (8, 128, 304), (8, 64, 304)])
def test_a_long_tail_adds_to_a_dominating_value_in_fp32(Hq, D, B):
    for gap in (21.75, 18.75, 15.0):
        out, ref = one_and_many(Hq, D, B, 1 << 20, gap, "f32", (1.0, 1.0), (1.0, -1.0))
        assert (np.abs(out - ref) <= 3e-5).all(), (gap, [float(np.abs(out - ref)[..., i, :].max()) for i in range(2)])


@pytest.mark.parametrize("Hq,Hkv,D,n", [(24, 4, 256, 3), (24, 4, 128, 4), (32, 4, 64, 5), (24, 4, 256, 22)])
def test_attention_runs_of_pages(Hq, Hkv, D, n):
    """Requests so long that a CTA takes thousands of an item's pages, whole items and parts of them, with new rows (some
    not finite) at the end: against the definition in 64 bits.  The pages' numbers repeat, in random order."""
    runs_of_pages(Hq, Hkv, D, n, "bf16", LONG[12:] if n > 16 else LONG)       # (22 nodes: two tiles of rows a head)


@pytest.mark.parametrize("Hq,Hkv,D,n,dtype", [(24, 4, 256, 1, "bf16"), (8, 4, 128, 2, "bf16"), (8, 4, 64, 4, "bf16"),
                                              (24, 4, 256, 2, "f32"), (8, 4, 128, 2, "f32"), (8, 4, 64, 5, "f32")])
def test_attention_runs_of_pages_few_rows(Hq, Hkv, D, n, dtype):
    runs_of_pages(Hq, Hkv, D, n, dtype, [300001] * 40 + LONG)


def runs_of_pages(Hq, Hkv, D, n, dtype, lens):
    from gated_deltanet_tree_gb300 import runtime as R
    rng = np.random.default_rng(D + n)
    pages = 60
    small, kr, vr = filled(rng, Hq, Hkv, D, [64 * pages], 1, dtype)
    B, pages_max = len(lens), -(-max(lens) // 64)
    pick = torch.from_numpy(rng.integers(0, pages, (B, pages_max)).astype(np.int32)).cuda()
    table = small.page_table[0][pick.long()].contiguous()
    c = R.KV4Cache(small.dims, small.pool, table, i32(lens))
    trees = [S.random_tree(n, rng) for _ in range(B)]
    q = (1.5 * rows(rng, B, 1, n, Hq, D, dtype="f32")).to(DT[dtype])
    kn, vn = rows(rng, B, 1, n, Hkv, D, dtype=dtype), rows(rng, B, 1, n, Hkv, D, dtype=dtype)
    vmax = max(float(vn.abs().max()), float(np.abs(vr).max()))
    kn[1, 0, n - 1], vn[4, 0, max(0, n - 2)] = float("nan"), float("inf")
    out = torch.full_like(q, 7.0)
    for _ in range(2):
        c.attention(q, kn, vn, out, sched=schedule(trees, n), max_len=max(lens))
    c.check_error()
    kr, vr = torch.from_numpy(kr[0, 0]).cuda(), torch.from_numpy(vr[0, 0]).cuda()
    G = Hq // Hkv
    for b in (0, 1, 4, B - 10, B - 9, B - 8, B - 7, B - 6, B - 5, B - 4, B - 2, B - 1):
        at = (64 * pick[b].long()[:, None] + torch.arange(64, device="cuda")).flatten()[:lens[b]]
        for h in range(Hkv):
            k, v = kr[at, h], vr[at, h]
            for i in range(n):
                line = K.root_path(trees[b], i)
                qi = q[b, 0, i, h * G:(h + 1) * G].double()
                w = torch.cat([qi @ k.T, qi @ kn[b, 0, line, h].double().T], -1) * c.dims.scale
                w = torch.softmax(w, -1)
                ref = w[:, :lens[b]] @ v + w[:, lens[b]:] @ vn[b, 0, line, h].double()
                got, ref = f64(out[b, 0, i, h * G:(h + 1) * G]), f64(ref)
                far = np.isinf(ref)
                assert np.array_equal(got[far], ref[far])
                check(np.where(far, 0.0, got), np.where(far, 0.0, ref), vmax, dtype, (b, h, i))


# ---- acceptance along the walk --------------------------------------------------------------------------------------

def at_once(B, n, V, draft):
    return n > 1 and B * n * V <= (2 if draft else 1) << 25


@pytest.mark.parametrize("B,n,V,dtype", [(32, 22, 50001, "bf16"), (40, 22, 40003, "f32"), (9, 64, 65536, "bf16"),
                                         (600, 64, 1001, "bf16"), (5, 64, 131073, "f32")])
def test_accept_chosen_drafts_along_the_walk(B, n, V, dtype):
    """More rows than are reduced at once: descents, rejected siblings and greedy requests through the cluster's own
    reduction."""
    assert not at_once(B, n, V, False)
    rng = np.random.default_rng(B + V)
    trees = [S.chain_tree(n) if b % 3 == 2 else S.random_tree(int(rng.integers(1, n + 1)), rng) for b in range(B)]
    temps = [0.0 if b % 4 == 3 else 0.5 + 0.7 * b / B for b in range(B)]
    acc, taken = accept_case(rng, B, n, V, dtype, temps, trees=trees)
    acc.check_error()
    assert taken > B + B // 4


def test_accept_deep_paths_along_the_walk():
    """Chains of 22 nodes accepted to every depth, greedy and sampled: 22 cluster joins one after another."""
    rng = np.random.default_rng(51)
    B, n, V = 33, 22, 60001
    assert not at_once(B, n, V, False)
    tokens = rng.integers(0, V, (B, n))
    z = torch.from_numpy(rng.standard_normal((B, n, V)).astype(np.float32))
    for b in range(B):
        for i in range(1, n):
            if i != b % n:                       # request b stops above node b % n
                z[b, i - 1, tokens[b, i]] += 40.0
    for dtype in ("bf16", "f32"):
        acc, _ = accept_case(rng, B, n, V, dtype, [0.0 if b % 2 else 0.9 for b in range(B)], trees=[S.chain_tree(n)] * B,
                             tokens=tokens, logits=z)
        acc.check_error()
        assert acc.len.tolist() == [b % n or n for b in range(B)]


@pytest.mark.parametrize("B,n,V,dtype,draft", [(70, 16, 65537, "bf16", "f32"), (48, 22, 70000, "f32", "bf16")])
def test_accept_sampled_drafts_along_the_walk(B, n, V, dtype, draft):
    assert not at_once(B, n, V, True)
    rng = np.random.default_rng(B + V)
    trees = [S.chain_tree(n) if b % 2 else S.random_tree(n, rng) for b in range(B)]
    trees[0] = np.array([-1] + [0] * (n - 1))
    temps = [1.0 if b % 5 else 0.0 for b in range(B)]
    acc, taken = accept_case(rng, B, n, V, dtype, temps, draft=draft, trees=trees)
    acc.check_error()
    assert taken > B


@pytest.mark.parametrize("draft", [False, True])
def test_accept_is_the_same_both_ways(draft):
    """One batch along the walk, and its requests a few at a time with all rows at once."""
    from gated_deltanet_tree_gb300 import runtime as R
    B, n, V, few = (64, 22, 48000, 4) if draft else (64, 22, 24000, 4)
    assert not at_once(B, n, V, draft) and at_once(few, n, V, draft)
    rng = np.random.default_rng(50)
    g = torch.Generator(device="cuda").manual_seed(50)
    trees = [S.random_tree(n, rng) for _ in range(B)]
    par = torch.from_numpy(np.stack([np.maximum(t, 0) for t in trees])).cuda()
    z = 2.0 * torch.randn(B, n, V, generator=g, device="cuda")
    tok = torch.randint(0, V, (B, n), generator=g, device="cuda")
    z.view(B, -1).scatter_add_(1, par * V + tok, torch.full((B, n), float(np.log(V)) + 2.5, device="cuda"))
    q = torch.softmax(z + 0.5 * torch.randn(B, n, V, generator=g, device="cuda"), -1) if draft else None
    u = torch.rand(B, n, generator=g, device="cuda")
    noise = -torch.log(-torch.log(torch.rand(B, V, generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)))
    t = 0.6 + 0.6 * torch.rand(B, generator=g, device="cuda")
    t[::5] = 0.0
    z, tok = z.bfloat16(), tok.int()
    whole = R.TreeAcceptor(B, n, V)
    whole.accept(schedule(trees, n), z, tok, u, noise, t, draft_probs=q)
    whole.check_error()
    part = R.TreeAcceptor(few, n, V)
    for b in range(0, B, few):
        s = slice(b, b + few)
        path, length, token = part.accept(schedule(trees[s], n), z[s], tok[s].clone(), u[s].clone(), noise[s], t[s].clone(),
                                          draft_probs=None if q is None else q[s])
        part.check_error()
        assert torch.equal(path, whole.path[s]) and torch.equal(length, whole.len[s])
        assert torch.equal(token, whole.next[s])
    assert int(whole.len.max()) >= 4


@pytest.mark.parametrize("B,n,V", [(13, 6, 3001), (13, 22, 140001), (13, 64, 90001)])
@pytest.mark.parametrize("draft", [None, "f32"])
def test_accept_at_small_temperatures(B, n, V, draft):
    """Down to the smallest fp32 number: z / T passes 2^24 (where its rounding passes 1) and fp32's largest number."""
    assert at_once(B, n, V, draft) == (n == 6 or (n == 22 and draft is not None))
    rng = np.random.default_rng(52)
    temps = [1e-2, 1e-4, 1e-6, 1e-7, 1e-8, 1e-9, 1e-12, 1e-20, 1e-30, 1e-36, 1e-38, 1e-41, 1.4e-45]
    for shift in (0.0, 30.0, -200.0):
        trees = [S.chain_tree(n) if b % 2 else S.random_tree(n, rng) for b in range(B)]
        tokens = rng.integers(0, V, (B, n))
        z = torch.from_numpy((shift + 2 * rng.standard_normal((B, n, V))).astype(np.float32))
        for b in range(B):
            for i in range(1, n):
                if rng.random() < 0.8:
                    z[b, trees[b][i], tokens[b, i]] += 20.0
        acc, _ = accept_case(rng, B, n, V, "f32", temps, draft=draft, trees=trees, tokens=None if draft else tokens,
                             logits=z)
        acc.check_error()


@pytest.mark.parametrize("V", [3001, 140001])
def test_accept_draws_among_equal_logits_at_small_temperatures(V):
    """Equal largest logits share the probability whatever the temperature: the Gumbel numbers decide."""
    from gated_deltanet_tree_gb300 import runtime as R
    rng = np.random.default_rng(53)
    temps = [1.0, 1e-3, 1e-5, 1e-6, 1e-7, 1e-8, 1e-12, 1e-30, 1e-38, 1.4e-45]
    B = 10 * len(temps)
    z = torch.from_numpy(rng.standard_normal((B, 1, V)).astype(np.float32)).cuda()
    ties = np.stack([np.sort(rng.choice(V, 5, replace=False)) for _ in range(B)])
    z.view(B, V).scatter_(1, torch.from_numpy(ties).cuda(), 47.3)
    g = torch.from_numpy(-np.log(-np.log(rng.random((B, V)))).astype(np.float32)).cuda()
    acc = R.TreeAcceptor(B, 1, V)
    acc.accept(schedule([np.array([-1])] * B, 1), z, i32(np.zeros((B, 1))), torch.zeros(B, 1, device="cuda"), g,
               torch.tensor(temps * 10, device="cuda"))
    acc.check_error()
    best = np.take_along_axis(g.cpu().numpy(), ties, 1).argmax(1)
    assert acc.next.tolist() == ties[np.arange(B), best].tolist()


def test_accept_rejections_that_leave_nothing():
    """Drafts whose probabilities are the target's own, exactly, with tokens that cannot have been drawn (outside the
    vocabulary): the rejection leaves nothing, and later siblings are tried against the distribution as it was."""
    rng = np.random.default_rng(54)
    B, n = 16, 9
    star = np.array([-1] + [0] * (n - 1))
    for V, keep in ((1, 1), (2, 2), (16, 16), (16, 4), (8192, 8192)):
        z = torch.zeros(B, n, V)
        z[..., keep:] = -float("inf")
        tokens = rng.integers(-1, keep + 1, (B, n))
        tokens[tokens >= keep] = V + 5
        tokens[:, 1] = V
        q = torch.softmax(z, -1).cuda()
        assert torch.equal(q[0, 0, :keep], torch.full((keep,), 1.0 / keep, device="cuda"))
        u = torch.from_numpy(rng.random((B, n)).astype(np.float32))
        noise = torch.from_numpy(-np.log(-np.log(rng.random((B, V)))).astype(np.float32))
        from gated_deltanet_tree_gb300 import runtime as R
        acc = R.TreeAcceptor(B, n, V)
        path, length, token = acc.accept(schedule([star] * B, n), z.cuda(), i32(tokens), u.cuda(), noise.cuda(),
                                         torch.ones(B, device="cuda"), draft_probs=q)
        acc.check_error()
        for b in range(B):
            want, nxt = A.accept(star.tolist(), tokens[b].tolist(), f64(z[b]), f64(u[b]), f64(noise[b]), 1.0, f64(q[b]))
            assert path[b, :int(length[b])].tolist() == want and int(token[b]) == nxt, (V, keep, b)


# ---- large batches and many launches --------------------------------------------------------------------------------

@pytest.mark.parametrize("Hq,Hkv,D,n,dtype", [(6, 1, 256, 1, "bf16"), (4, 1, 64, 2, "f32"), (24, 1, 256, 2, "bf16"),
                                              (8, 1, 128, 4, "bf16")])
def test_attention_many_short_requests(Hq, Hkv, D, n, dtype):
    """More requests than a CTA has threads: their units are summed, and a CTA's place found, in blocks; lengths from 0,
    more requests than CTAs and several requests a CTA."""
    rng = np.random.default_rng(60 + n)
    B = 1300
    lens = rng.integers(0, 140, B)
    lens[[0, 5, 576, 1152, B - 1]] = [0, 128, 0, 64, 131]
    trees = None if n == 1 else [S.random_tree(int(rng.integers(1, n + 1)), rng) for _ in range(B)]
    if trees is not None:
        trees[0] = S.random_tree(n, rng)
    run_case(rng, Hq, Hkv, D, lens.tolist(), trees, dtype)
    # (requests out of range among them: nothing served but the others)
    from gated_deltanet_tree_gb300 import _native as N
    c, kr, vr = filled(rng, Hq, Hkv, D, lens.tolist(), 1, dtype)
    q = rows(rng, B, 1, 1, Hq, D, dtype=dtype)
    good, out = torch.zeros_like(q), torch.full_like(q, 7.0)
    c.attention(q, None, None, good)
    c.check_error()
    bad = [1, 255, 256, 700, B - 2]
    c.seq_len[bad] = -1
    c.attention(q, None, None, out)
    with pytest.raises(N.GdnError) as e:
        c.check_error()
    assert e.value.status == N.GDN_ERR_CACHE
    assert (out[bad] == 7.0).all()
    kept = np.setdiff1d(np.arange(B), bad)
    vmax = max(1.0, float(np.abs(vr).max()))
    check(f64(out[kept]), f64(good[kept]), vmax, dtype, "others")       # (split elsewhere: other roundings)


@pytest.mark.parametrize("Hq,Hkv,D,n,layers,B", [(24, 4, 64, 2, 32, 66), (24, 4, 256, 4, 16, 66), (8, 8, 64, 1, 32, 66),
                                                 (512, 64, 64, 1, 8, 40)])
def test_attention_in_several_launches(Hq, Hkv, D, n, layers, B):
    """More items than a launch has counters or records for: requests of later launches, whose counters are the first
    ones' again."""
    some = n * (Hq // Hkv)
    few = some <= {256: 16, 128: 20, 64: 28}[D]
    assert (16384 if few else 4096) // (layers * Hkv * -(-some // (8 if few else 128))) < B
    rng = np.random.default_rng(70 + n)
    lens = rng.integers(0, 100, B)
    lens[[0, 1, B - 1]] = [1, 99, 400]
    trees = None if n == 1 else [S.random_tree(int(rng.integers(1, n + 1)), rng) for _ in range(B)]
    if trees is not None:
        trees[0] = S.random_tree(n, rng)
    c = make_cache(Hq, Hkv, D, B, layers, 7, "bf16")
    k, v = rows(rng, B, layers, 400, Hkv, D, dtype="bf16"), rows(rng, B, layers, 400, Hkv, D, dtype="bf16")
    c.append(k, v, i32(lens))
    kr, vr = c.read(None, 400)
    q, kn, vn = (rows(rng, B, layers, n, h, D, dtype="bf16") for h in (Hq, Hkv, Hkv))
    out = torch.full_like(q, 7.0)
    for _ in range(2):
        c.attention(q, kn, vn, out, sched=None if trees is None else schedule(trees, n), max_len=400)
    c.check_error()
    assert not c.workspace[:65536].any()
    G, vmax = Hq // Hkv, max(float(vn.abs().max()), float(vr.abs().max()))
    # every request's every layer and head in fp64, batched: an additive mask for what a row does not see
    L = int(lens.max())
    see = torch.zeros(B, n, L + n, dtype=torch.bool, device="cuda")
    see[:, :, :L] = (torch.arange(L, device="cuda") < i32(lens)[:, None])[:, None]
    for b in range(B):
        t = np.array([-1]) if trees is None else trees[b]
        for i in range(len(t)):
            see[b, i, [L + j for j in K.root_path(t, i)]] = True
    for l in range(layers):
        kk = torch.cat([kr[:, l, :L], kn[:, l].float()], 1).double()                   # [B, L + n, Hkv, D]
        vv = torch.cat([vr[:, l, :L], vn[:, l].float()], 1).double()
        qq = q[:, l].double().unflatten(2, (Hkv, G))                                   # [B, n, Hkv, G, D]
        a = torch.einsum("bnhgd,bthd->bnhgt", qq, kk) * c.dims.scale
        a = a.masked_fill(~see[:, :, None, None], -float("inf"))
        ref = torch.einsum("bnhgt,bthd->bnhgd", torch.softmax(a, -1), vv).flatten(2, 3)
        for b in range(B):
            m = 1 if trees is None else len(trees[b])
            check(f64(out[b, l, :m]), f64(ref[b, :m]), vmax, "bf16", (b, l))
            assert (out[b, l, m:] == 7.0).all()


# ---- the example ----------------------------------------------------------------------------------------------------

def test_example_step_against_the_oracles():
    """The example's last step: its attention's output from the cache as it was before the step, its acceptance from the
    logits and numbers it drew, and the rows its append left in the cache."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import hybrid_step
    seen = {}

    class Watched(hybrid_step.HybridStack):
        def step(self, *args):
            before = tuple(f64(t) for t in self.cache.read(None, 64 * self.cache.pages_max)) + (self.cache.seq_len.tolist(),)
            attention, accept = self.cache.attention, self.acceptor.accept

            def look_attention(q, k, v, out, sched):
                attention(q, k, v, out, sched=sched)
                seen["attention"] = (before, q.clone(), k.clone(), v.clone(), out.clone(), sched)

            def look_accept(sched, z, tokens, u, g, t):
                got = accept(sched, z, tokens, u, g, t)
                seen["accept"] = (z.clone(), tokens.clone(), u.clone(), g.clone(), t.clone(), [x.clone() for x in got])
                return got

            self.cache.attention, self.acceptor.accept = look_attention, look_accept
            got = super().step(*args)
            del self.cache.attention, self.acceptor.accept
            return got

    whole, hybrid_step.HybridStack = hybrid_step.HybridStack, Watched
    try:
        model = hybrid_step.main(steps=3, show=lambda line: None)
    finally:
        hybrid_step.HybridStack = whole
    (kr, vr, lens), q, k, v, out, sched = seen["attention"]
    z, tokens, u, g, t, (path, length, token) = seen["accept"]
    after = [f64(x) for x in model.cache.read(None, 64 * model.cache.pages_max)]
    for b in range(model.B):
        m = int(sched.n[b])
        tree = sched.parents[b, :m]
        ref = K.tree_attention(f64(q[b, 0, :m]), kr[b, 0, :lens[b]], vr[b, 0, :lens[b]], f64(k[b, 0, :m]), f64(v[b, 0, :m]),
                               tree, model.cache.dims.scale)
        check(f64(out[b, 0, :m]), ref, max(float(v.abs().max()), float(np.abs(vr).max())), "bf16", b)
        want, nxt = A.accept(tree.tolist(), tokens[b].tolist(), f64(z[b, :m]), f64(u[b]), f64(g[b]), float(t[b]))
        L = int(length[b])
        assert path[b, :L].tolist() == want and int(token[b]) == nxt
        for x, new in zip(after, (k, v)):
            rows64 = np.stack([[K.quantise_row(r) for r in f64(new[b, 0, i])] for i in want])
            assert np.array_equal(x[b, 0, lens[b]:lens[b] + L], rows64)
        assert int(model.cache.seq_len[b]) == lens[b] + L
