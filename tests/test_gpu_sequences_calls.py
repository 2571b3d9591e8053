"""Prompt, single-token and log-probability calls as programs make them on a GPU: streams, CUDA graphs, calls between tree
verifies, values that change their size within a chunk, and sizes beyond 32-bit offsets.  Tolerances as in
test_gpu_sequences.py unless a test derives its own."""
import threading

import numpy as np
import pytest
import torch

import synthetic as S
from oracle import gdn_oracle as O
from oracle import seq_oracle as Q
from test_gpu_sequences import DT, Case, built, check, check_scores, f64, rows_of  # noqa: F401

pytestmark = pytest.mark.gpu


# ---- with tree verifies ---------------------------------------------------------------------------------------------

def test_prompt_trees_and_tokens_of_one_request():
    """A request's whole life: prompt, a tree, its accepted path, a token, more prompt -- against the replay of all rows."""
    from gated_deltanet_tree_gb300 import _native as N
    from gated_deltanet_tree_gb300 import runtime as R
    rng = np.random.default_rng(1)
    B, layers, n_max = 2, 2, 12
    c = Case(1, "qwen", [100, 40], "bf16", layers=layers)
    d = c.d
    dims = R.make_dims(d.Hk, d.Hv, d.dk, d.dv, d.K, 1, 1, N.GDN_DTYPE_BF16, d.q_scale, d.l2_eps)
    ver = R.TreeVerifier(dims, B, layers, n_max)
    run = R.SequenceRunner(dims, B, layers, verifier=ver)
    state, conv = c.state.clone(), c.conv.clone()
    T, W = f64(c.state), f64(c.conv)
    w64 = f64(c.w)
    for layer in range(layers):
        run.prefill(c.lens, *c.inputs(), state, conv, c.out, layer=layer)
        _, T[:, layer], W[:, layer] = Q.run_batch(c.lens, T[:, layer], W[:, layer], f64(c.x), f64(c.beta), f64(c.log_g), w64[layer], d)
    trees = [S.random_tree(n_max, rng), S.random_tree(9, rng)]
    sched = ver.schedule(trees)
    t = Case(2, "qwen", [B * layers * n_max], "bf16", layers=layers)
    x, beta, log_g = (a.view(B, layers, n_max, -1) for a in (t.x, t.beta, t.log_g))
    o = torch.zeros(B, layers, n_max, d.Hv, d.dv, device="cuda")
    boundary = torch.zeros(B, layers, max(1, sched.nb_max), d.Hv, d.dk, d.dv, device="cuda")
    ver.verify(sched, x, c.w, beta, log_g, state, conv, o, boundary)
    one = Case(3, "qwen", [1, 1], "bf16", layers=layers)
    for call in (lambda: run.step(*one.inputs(), state, conv, one.out), lambda: run.prefill([1, 1], *one.inputs(), state, conv, one.out)):
        with pytest.raises(N.GdnError) as e:
            call()
        assert e.value.status == N.GDN_ERR_STATE
    paths = [O.root_path(p.tolist(), len(p) - 1) for p in trees]
    ver.commit(sched, *R.paths_tensor(paths, n_max, "cuda"))
    with pytest.raises(N.GdnError) as e:                       # committed, but not in the states yet
        run.step(*one.inputs(), state, conv, one.out)
    assert e.value.status == N.GDN_ERR_STATE
    ver.finish(state, conv)
    for b in range(B):
        for layer in range(layers):
            rows = [a[b, layer, paths[b]] for a in (x, beta, log_g)]
            want, T[b, layer], W[b, layer] = Q.run_sequence(T[b, layer], W[b, layer], *(f64(a) for a in rows), w64[layer], d)
            got = f64(o[b, layer, paths[b]])
            assert np.abs(got - want).max() <= 2e-5 * np.abs(want).max()
    more = Case(4, "qwen", [70, 0], "bf16", layers=layers)
    for layer in range(layers):
        run.step(*one.inputs(), state, conv, one.out, layer=layer)
        w1, T[:, layer], W[:, layer] = Q.run_batch([1, 1], T[:, layer], W[:, layer], f64(one.x), f64(one.beta), f64(one.log_g), f64(one.w[layer]), d)
        assert np.abs(f64(one.out) - w1).max() <= 2e-5 * np.abs(w1).max()
        run.prefill(more.lens, *more.inputs(), state, conv, more.out, layer=layer)
        w2, T[:, layer], W[:, layer] = Q.run_batch(more.lens, T[:, layer], W[:, layer], f64(more.x), f64(more.beta), f64(more.log_g), f64(more.w[layer]), d)
        assert np.abs(f64(more.out) - w2).max() <= 2e-5 * np.abs(w2).max()
    run.check_error()
    assert np.array_equal(f64(conv), W)
    for b in range(B):
        for layer in range(layers):
            for h in range(d.Hv):
                assert np.linalg.norm(f64(state[b, layer, h]) - T[b, layer, h]) <= 1e-5 * np.linalg.norm(T[b, layer, h])


def test_calls_after_a_time_out_do_nothing_until_it_is_read():
    from gated_deltanet_tree_gb300 import _native as N
    from gated_deltanet_tree_gb300 import runtime as R
    for lens, heads, B in (([90, 3], "qwen", 2), ([1] * 160, "qwen", 160)):
        c = Case(5, heads, lens, "bf16", layers=1, layer=0)
        run = c.runner()
        run.err[0] = 4                                         # what a kernel that gave up on a wait reports
        state, conv = c.state.clone(), c.conv.clone()
        if B == 2:
            run.prefill(lens, *c.inputs(), state, conv, c.out)
        run.step(c.x[:B], c.w, c.beta[:B], c.log_g[:B], state, conv, c.out[:B])
        torch.cuda.synchronize()
        assert torch.equal(state, c.state) and torch.equal(conv, c.conv) and (c.out == 7.0).all()
        with pytest.raises(N.GdnError) as e:
            run.check_error()
        assert e.value.status == N.GDN_ERR_TIMEOUT
        run.prefill(lens, *c.inputs(), state, conv, c.out)
        run.check_error()
        check(c, c.reference(), c.out, state[:, 0], conv[:, 0])


# ---- streams and graphs ---------------------------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["prefill", "step", "score"])
def test_first_call_on_a_side_stream_while_the_current_one_is_busy(kind):
    from gated_deltanet_tree_gb300 import runtime as R
    side = torch.cuda.Stream()
    c = Case(6, "qwen", [130, 20] if kind == "prefill" else [1, 1], "bf16", layers=1, layer=0)
    z = rows_of(np.random.default_rng(6), 3, 50000, "normal", "bf16")
    state, conv = c.state.clone(), c.conv.clone()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                              # ends by itself, about 10 ms
    run, scorer = c.runner(), R.TokenScorer(3, 50000, 8)
    torch.cuda._sleep(20_000_000)
    if kind == "prefill":
        run.prefill(c.lens, *c.inputs(), state, conv, c.out, stream=side)
    elif kind == "step":
        run.step(*c.inputs(), state, conv, c.out, stream=side)
    else:
        got = scorer.score(z, stream=side)
    side.synchronize()
    if kind == "score":
        got = [None if g is None else g.clone() for g in got]
    out, s, w = c.out.clone(), state.clone(), conv.clone()
    torch.cuda.synchronize()
    if kind == "score":
        scorer.check_error()
        check_scores(z, 8, got)
    else:
        run.check_error()
        check(c, c.reference(), out, s[:, 0], w[:, 0])


def test_two_runners_at_once():
    """Two prompts on two streams, each with its own runner, both at work together; and again in the other order."""
    cases = [Case(7 + i, "qwen", [400, 150], "bf16", slow=True, layers=1, layer=0) for i in range(2)]
    runs, streams = [c.runner() for c in cases], [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for order in ((0, 1), (1, 0)):
        states = [(c.state.clone(), c.conv.clone()) for c in cases]
        for c in cases:
            c.out.fill_(7.0)
        torch.cuda.synchronize()
        for i in order:
            c = cases[i]
            runs[i].prefill(c.lens, *c.inputs(), *states[i], c.out, stream=streams[i])
        torch.cuda.synchronize()
        for i in order:
            runs[i].check_error()
            check(cases[i], cases[i].reference(), cases[i].out, states[i][0][:, 0], states[i][1][:, 0], (order, i))


def test_long_prompts_on_two_busy_streams_and_captured():
    """Prompts long enough to be prepared beside their chains (on a stream of the library's own): two at once on busy streams
    whose next work overwrites the inputs, again, and captured into a graph, where all of it stays on the one stream.  The
    four results agree within the tolerance of two calls that round differently, 2e-5 and 1e-5, and with the oracle's last
    tokens, continued from the state before them."""
    n, tail = 3400, 60
    cases = [Case(30 + i, (1, 2, 128, 128), [n, 3300], "bf16", slow=True, layers=1, layer=0) for i in range(2)]
    runs, streams = [c.runner() for c in cases], [torch.cuda.Stream() for _ in cases]
    kept = [[t.clone() for t in (c.x, c.beta, c.log_g, c.state, c.conv)] for c in cases]
    results = []
    torch.cuda.synchronize()
    for again in range(2):
        torch.cuda.synchronize()
        for c, r, st, k in zip(cases, runs, streams, kept):
            with torch.cuda.stream(st):
                torch.cuda._sleep(4_000_000)
                for a, b in zip((c.x, c.beta, c.log_g, c.state, c.conv), k):
                    a.copy_(b)
                r.prefill(c.lens, *c.inputs(), c.state, c.conv, c.out)
                results.append((c.out.clone(), c.state.clone(), c.conv.clone()))
                for t in (c.x, c.beta, c.log_g, c.state, c.conv, c.out):
                    t.fill_(float("nan"))
    torch.cuda.synchronize()
    for r in runs:
        r.check_error()
    assert all(torch.equal(a, b) for i in range(2) for a, b in zip(results[i], results[2 + i]))
    c, r = cases[0], runs[0]
    graph = torch.cuda.CUDAGraph()
    for a, b in zip((c.x, c.beta, c.log_g, c.state, c.conv), kept[0]):
        a.copy_(b)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        r.prefill(c.lens, *c.inputs(), c.state, c.conv, c.out)
    graph.replay()
    torch.cuda.synchronize()
    r.check_error()
    out, state, conv = results[0]
    assert (c.out - out).abs().max() <= 2e-5 * out.abs().max() and torch.equal(c.conv, conv)
    assert (c.state - state).norm() <= 1e-5 * state.norm()
    # the last tokens against the oracle
    for b, at in enumerate((n, n + 3300)):
        s, w = kept[0][3][b:b + 1].clone(), kept[0][4][b:b + 1].clone()
        one = Case(0, (1, 2, 128, 128), [1], "bf16", layers=1, layer=0).runner()
        first, size = (0, n) if b == 0 else (n, 3300)
        rows = slice(first, first + size - tail)
        k = kept[0]
        one.prefill([size - tail], k[0][rows], c.w, k[1][rows], k[2][rows], s, w, torch.empty_like(c.out[rows]))
        rows = slice(at - tail, at)
        o, T, _ = Q.run_sequence(f64(s[0, 0]), f64(w[0, 0]), f64(k[0][rows]), f64(k[1][rows]), f64(k[2][rows]), f64(c.w[0]), c.d)
        assert np.abs(f64(out[rows]) - o).max() <= 4e-5 * np.abs(o).max()
        assert np.linalg.norm(f64(state[b, 0]) - T) <= 2e-5 * np.linalg.norm(T)


def test_first_long_prompt_of_a_thread_while_another_captures():
    """A thread's first long prompt makes the library's stream for that thread: it must end no capture of another one, and give
    the bits of the same call made outside."""
    c = Case(34, (1, 2, 128, 128), [3200], "bf16", slow=True, layers=1, layer=0)
    r, work = c.runner(), torch.cuda.Stream()
    want, out = c.out.clone(), torch.empty_like(c.out)
    state, window = torch.empty_like(c.state), torch.empty_like(c.conv)
    r.prefill(c.lens, *c.inputs(), c.state, c.conv, want, state_out=state, conv_out=window)
    x, y = torch.ones(1000, device="cuda"), torch.zeros(1000, device="cuda")
    torch.cuda.synchronize()
    failed = []

    def call():
        try:
            r.prefill(c.lens, *c.inputs(), c.state, c.conv, out, state_out=state, conv_out=window, stream=work)
        except Exception as e:
            failed.append(e)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y.add_(x)
        thread = threading.Thread(target=call)
        thread.start()
        thread.join()
        y.add_(x)
    graph.replay()
    torch.cuda.synchronize()
    r.check_error()
    assert not failed and torch.equal(out, want) and torch.equal(y, 2 * x)


@pytest.mark.parametrize("B", [2, 160])
def test_captured_calls_replay(B):
    """A graph of a prompt, a token and the tokens' scores follows its buffers; larger calls in between do not change it."""
    from gated_deltanet_tree_gb300 import runtime as R
    lens = [130, 20] if B == 2 else [3] * B
    c, one = Case(9, "qwen", lens, "bf16", layers=1, layer=0), Case(10, "qwen", [1] * B, "bf16", layers=1, layer=0)
    run = c.runner()
    scorer = R.TokenScorer(B, 20001, 4)
    z = rows_of(np.random.default_rng(3), B, 20001, "normal", "bf16")
    state, conv = c.state.clone(), c.conv.clone()
    live = torch.ones(B, dtype=torch.int32, device="cuda")

    def work():
        run.prefill(lens, *c.inputs(), state, conv, c.out)
        run.step(one.x, c.w, one.beta, one.log_g, state, conv, one.out, live=live)
        scorer.score(z)

    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work()
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            work()
    torch.cuda.current_stream().wait_stream(side)
    big = Case(11, "qwen", [500] * B if B == 2 else [70] * B, "bf16", layers=1, layer=0)
    for i in range(2):
        run.prefill(big.lens, *big.inputs(), big.state.clone(), big.conv.clone(), big.out)
        new = Case(20 + i, "qwen", lens, "bf16", layers=1, layer=0)
        for a, b in ((c.x, new.x), (c.beta, new.beta), (c.log_g, new.log_g), (state, new.state), (conv, new.conv)):
            a.copy_(b)
        live.fill_(1)
        live[i::3] = 0
        graph.replay()
        torch.cuda.synchronize()
        run.check_error()
        o, T, W = c.reference(state=new.state[:, 0], conv=new.conv[:, 0])
        bf16 = np.abs(f64(c.out) - o).max() <= 2e-5 * np.abs(o).max()
        assert bf16, np.abs(f64(c.out) - o).max()
        for b in range(B):
            if live[b]:
                y, T[b], W[b] = Q.run_sequence(T[b], W[b], f64(one.x[b:b + 1]), f64(one.beta[b:b + 1]), f64(one.log_g[b:b + 1]),
                                               f64(c.w[0]), c.d)
                assert np.abs(f64(one.out[b]) - y[0]).max() <= 2e-5 * np.abs(y).max()
            assert np.linalg.norm(f64(state[b, 0]) - T[b]) <= 1e-5 * np.linalg.norm(T[b])
            assert np.array_equal(f64(conv[b, 0]), W[b])
    check_scores(z[:3], 4, tuple(None if t is None else t[:3] for t in (scorer.top, scorer.tokens, None, scorer.entropy)))


def test_calls_are_repeatable():
    """The same call gives the same bits: no sum depends on which CTA or warp comes first."""
    c = Case(12, "qwen", [300, 65, 1], "bf16", slow=True, layers=1, layer=0)
    first = None
    for _ in range(4):
        state, conv = c.state.clone(), c.conv.clone()
        run = c.runner()
        run.prefill(c.lens, *c.inputs(), state, conv, c.out)
        got = (c.out.clone(), state)
        first = got if first is None else first
        assert torch.equal(got[0], first[0]) and torch.equal(got[1], first[1])


# ---- values that change their size within a chunk --------------------------------------------------------------------

@pytest.mark.parametrize("pattern", [
    ((0, 64, 30), (64, 128, -30)),             # a large chunk, then a small one
    ((20, 21, 40),),                           # one token far above the rest, forgotten within the chunk
    ((0, 40, 35), (100, 130, 35)),
    ((64, 65, 60), (65, 260, -20)),
    ((0, 10, -60), (10, 20, 20), (20, 260, -40)),
    ((127, 128, 45), (191, 192, 45)),          # a chunk's last token
    ((240, 260, -50),)])
@pytest.mark.parametrize("gates", ["mixed", "fast"])
def test_prefill_values_of_changing_size(pattern, gates):
    """Tokens [a, b) scaled by 2^e.  States and outputs are held to their own size per chunk of 64 tokens, although the
    bounds that the operands are scaled by are then far above them: outputs within 2e-5 of the largest of the chunk, the
    state, after every chunk, within 1e-5 of itself."""
    for n in (64, 128, 192, 260):
        c = Case(13, "qwen", [n], "f32", act=0, conv=0, layers=1, layer=0, slow=gates == "mixed")
        nq = 2 * c.d.Hk * c.d.dk
        for a, b, e in pattern:
            c.x[a:b, nq:] *= 2.0 ** e
        if gates == "fast":
            c.log_g *= 2.0
        state = c.state.clone()
        o, T, W = c.reference()
        run = c.runner()
        run.prefill(c.lens, *c.inputs(), state, None, c.out)
        run.check_error()
        got = f64(c.out)
        for h in range(c.d.Hv):
            for a in range(0, n, 64):
                r = o[a:a + 64, h]
                assert np.abs(got[a:a + 64, h] - r).max() <= 2e-5 * np.abs(r).max(), (n, h, a, np.abs(got[a:a + 64, h] - r).max() / np.abs(r).max())
            s, t = f64(state[0, 0, h]), T[0, h]
            assert np.linalg.norm(s - t) <= 1e-5 * np.linalg.norm(t), (n, h, np.linalg.norm(s - t) / np.linalg.norm(t))


def test_prefill_tokens_without_effect():
    """Huge values with beta 0 and zero states: nothing is written, and nothing of them is in the outputs."""
    c = Case(14, "qwen", [130], "f32", act=0, conv=0, layers=1, layer=0, slow=True)
    nq = 2 * c.d.Hk * c.d.dk
    c.beta[20:100] = 0.0
    c.x[20:100, nq:] = 1e30
    for zero in (False, True):
        state = torch.zeros_like(c.state) if zero else c.state.clone()
        o, T, W = c.reference(state=state[:, 0])
        run = c.runner()
        run.prefill(c.lens, *c.inputs(), state, None, c.out)
        run.check_error()
        for h in range(c.d.Hv):
            for a in range(0, 130, 64):
                r = o[a:a + 64, h]
                assert np.abs(f64(c.out[a:a + 64, h]) - r).max() <= 2e-5 * np.abs(r).max()
            assert np.linalg.norm(f64(state[0, 0, h]) - T[0, h]) <= 1e-5 * np.linalg.norm(T[0, h])


def test_prefill_gates_above_one():
    """log gates above 0 (the state grows): e^10 within a chunk."""
    c = Case(15, "qwen", [150], "f32", layers=1, layer=0, slow=True)
    c.log_g.abs_().mul_(0.2)
    state, conv = c.state.clone(), c.conv.clone()
    run = c.runner()
    run.prefill(c.lens, *c.inputs(), state, conv, c.out)
    run.check_error()
    check(c, c.reference(), c.out, state[:, 0], conv[:, 0])


def test_prefill_long_sequence_of_slow_gates():
    """2000 tokens that hardly forget: the state's error does not grow with the length.  Each token's rounding is kept by
    e^(log gate) and by 1 - beta k k^T, which contracts: 1 of dk directions by about a half a token."""
    c = Case(16, (1, 2, 64, 64), [2000], "f32", layers=1, layer=0)
    c.log_g.mul_(1e-3)
    state, conv = c.state.clone(), c.conv.clone()
    run = c.runner()
    run.prefill(c.lens, *c.inputs(), state, conv, c.out)
    run.check_error()
    check(c, c.reference(), c.out, state[:, 0], conv[:, 0])


# ---- sizes ----------------------------------------------------------------------------------------------------------

def test_prefill_rows_beyond_32_bit_offsets():
    """220000 rows of 10240 channels: the last request's results are those of a call of its own."""
    from gated_deltanet_tree_gb300 import runtime as R
    dims = R.make_dims(16, 48, 128, 128, 4)
    gen = torch.Generator(device="cuda").manual_seed(1)
    lens = [70000, 0, 149870, 130]
    rows = sum(lens)
    x = torch.empty(rows, 10240, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    beta = torch.rand(rows, 48, generator=gen, device="cuda").bfloat16()
    log_g = -torch.rand(rows, 48, generator=gen, device="cuda").bfloat16()
    w = 0.5 * torch.randn(1, 10240, 4, generator=gen, device="cuda")
    out = torch.empty(rows, 48, 128, dtype=torch.bfloat16, device="cuda")
    state, conv = torch.empty(4, 1, 48, 128, 128, device="cuda"), torch.empty(4, 1, 3, 10240, device="cuda")
    run = R.SequenceRunner(dims, 4)
    run.prefill(lens, x, w, beta, log_g, None, None, out, state_out=state, conv_out=conv)
    run.check_error()
    own = R.SequenceRunner(dims, 1)
    o, s, v = torch.empty_like(out[-130:]), torch.empty_like(state[:1]), torch.empty_like(conv[:1])
    own.prefill([130], x[-130:], w, beta[-130:], log_g[-130:], None, None, o, state_out=s, conv_out=v)
    own.check_error()
    assert torch.equal(o, out[-130:]) and torch.equal(s[0], state[3]) and torch.equal(v[0], conv[3])
    # the middle request's last tokens, from the state that a call of its earlier ones leaves
    own.prefill([149000], x[70000:219000], w, beta[70000:219000], log_g[70000:219000], None, None, out[70000:219000], state_out=s,
                conv_out=v)
    o = torch.empty_like(out[:870])
    own.prefill([870], x[219000:219870], w, beta[219000:219870], log_g[219000:219870], s, v, o)
    own.check_error()
    want = out[219000:219870].float()
    assert (o.float() - want).abs().max() <= (2.0 ** -7 + 4e-5) * want.abs().max()
    assert (s[0] - state[2]).norm() <= 2e-5 * state[2].norm() and torch.equal(v[0], conv[2])


def test_logprobs_beyond_32_bit_offsets():
    from gated_deltanet_tree_gb300 import runtime as R
    rows, V = 17000, 131072
    z = torch.zeros(rows, V, dtype=torch.bfloat16, device="cuda")
    few = rows_of(np.random.default_rng(5), 3, V, "normal", "bf16")
    at = [0, 9000, rows - 1]
    z[at] = few
    s = R.TokenScorer(rows, V, 4)
    tokens = torch.full((rows,), V - 1, dtype=torch.int32, device="cuda")
    top, best, given, entropy = s.score(z, tokens)
    s.check_error()
    check_scores(few, 4, (top[at], best[at], given[at], entropy[at]), tokens[at])
    flat = [1, 8999, rows - 2]
    assert (best[flat] == torch.arange(4, device="cuda")).all()
    assert (top[flat] + np.log(V)).abs().max() <= 1e-5 and (entropy[flat] - np.log(V)).abs().max() <= 4e-5


@pytest.mark.parametrize("V", [400000, 1100003])
def test_logprobs_of_large_vocabularies(V):
    """More tiles a CTA than the bound is renewed after, rising rows among them (every tile passes the bound)."""
    from gated_deltanet_tree_gb300 import runtime as R
    rng = np.random.default_rng(V)
    z = rows_of(rng, 2, V, "normal", "f32")
    z[1] = torch.linspace(-3, 3, V, device="cuda")
    s = R.TokenScorer(2, V, 32)
    got = s.score(z)
    s.check_error()
    check_scores(z, 32, got)
    many = z.repeat(160, 1)
    s = R.TokenScorer(320, V, 32)
    top, best, _, entropy = s.score(many)
    s.check_error()
    check_scores(z, 32, (top[318:], best[318:], None, entropy[318:]))


def test_example_with_single_tokens():
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import hybrid_step
    seen = []
    model = hybrid_step.main(steps=2, decode=3, show=seen.append)
    assert len(seen) == 6 and torch.isfinite(model.state).all() and model.state.abs().max() > 0
    assert ((model.last >= 0) & (model.last < model.V)).all()


def test_example_prompt_reaches_the_gdn_states():
    """The example's prompt against the oracle: states and windows of every layer."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import hybrid_step
    model = hybrid_step.HybridStack(B=2)
    rng = np.random.default_rng(2)
    T, W = f64(model.state), f64(model.conv_state)
    tokens = torch.from_numpy(rng.integers(0, model.V, (2, 70))).cuda()
    count = torch.tensor([70, 9], dtype=torch.int32, device="cuda")
    model.prompt(tokens, count)
    g = model.gdn
    d = O.Dims(g.Hk, g.Hv, g.dk, g.dv, g.K, q_scale=g.q_scale, l2_eps=g.l2_eps)
    for b in range(2):
        raw, beta, log_g = model.gdn_inputs(torch.cat([model.embed[tokens[0, :70]], model.embed[tokens[1, :9]]]))
        rows = slice(0, 70) if b == 0 else slice(70, 79)
        for layer in range(model.gdn_layers):
            _, t, w = Q.run_sequence(T[b, layer], W[b, layer], f64(raw[rows]), f64(beta[rows]), f64(log_g[rows]), f64(model.conv_w[layer]), d)
            assert np.linalg.norm(f64(model.state[b, layer]) - t) <= 1e-5 * np.linalg.norm(t)
            assert np.array_equal(f64(model.conv_state[b, layer]), w)
