"""Prompt, single-token and log-probability calls on a GPU, beside test_gpu_sequences.py and test_gpu_sequences_calls.py, whose
tolerances these tests use."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import gdn_oracle as O
from oracle import seq_oracle as Q
from test_gpu_sequences import DT, Case, built, check, check_scores, f64, rows_of  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,n", [(9001, 6), (131, 5), (20003, 400)])
@pytest.mark.parametrize("row,col", [(1, 0), (0, 1), (3, 5), (2, 7)])
def test_logits_that_begin_at_any_element(dtype, V, n, row, col):
    """A slice from an odd row of an odd vocabulary, or from an odd column of wider rows, with neighbours that must not be seen."""
    from gated_deltanet_tree_gb300.runtime import TokenScorer
    rng = np.random.default_rng(V + col)
    wide = torch.full((n + row, V + col), float("nan"), dtype=DT[dtype], device="cuda")
    z = wide[row:, col:]
    z.copy_(rows_of(rng, n, V, "normal", dtype))
    s = TokenScorer(n, V, 5)
    tokens = torch.from_numpy(rng.integers(0, V, n).astype(np.int32)).cuda()
    top, best, given, entropy = s.score(z, tokens)
    s.check_error()
    at = list(range(n)) if n < 10 else [0, 1, 2, 3, n - 1]
    check_scores(z[at], 5, (top[at], best[at], given[at], entropy[at]), tokens[at])


def test_scores_of_a_prompt_s_next_tokens():
    """score(logits[:-1], tokens[1:]) on the current stream, on busy ones given as an object and as a number, and in a graph."""
    from gated_deltanet_tree_gb300.runtime import TokenScorer
    rng = np.random.default_rng(3)
    V, n = 5001, 40
    z = rows_of(rng, n, V, "normal", "f32")
    tokens = torch.from_numpy(rng.integers(0, V, n).astype(np.int32)).cuda()
    s, side = TokenScorer(n, V, 3), torch.cuda.Stream()
    want = s.score(z[:-1], tokens[1:].clone())[2].clone()
    check_scores(z[:-1], 3, s.score(z[:-1], tokens[1:]), tokens[1:])
    late = torch.zeros_like(tokens)
    torch.cuda.synchronize()
    for how in ("object", "number", "current"):
        late.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(4_000_000)                       # ends by itself, about 2 ms
            late.copy_(tokens)
        if how == "current":
            with torch.cuda.stream(side):
                s.score(z[:-1], late[1:])
        else:
            s.score(z[:-1], late[1:], stream=side if how == "object" else side.cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(s.given[:n - 1], want), how
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.score(z[:-1], late[1:])
    late.copy_(torch.flip(tokens, (0,)))
    graph.replay()
    torch.cuda.synchronize()
    s.check_error()
    check_scores(z[:-1], 3, (s.top[:n - 1], s.tokens[:n - 1], s.given[:n - 1], s.entropy[:n - 1]), late[1:])


@pytest.mark.parametrize("Hk,Hv,lens", [(128, 128, [20 + 3 * i for i in range(60)]), (512, 512, [130, 0, 65, 17, 3, 64, 100, 20, 40, 30, 200, 18, 19, 90]),
                                        (1024, 1024, [150, 40, 70]), (16, 48, [590 - 37 * (i % 11) - i for i in range(40)])])
def test_prompts_of_many_heads(Hk, Hv, lens):
    """So many heads that the workspace holds fewer chunks than there are requests, or chunks: 49, 12 and 6; 220 of 16 and 48 heads,
    where forty requests have 270 (no more are begun than fill the GPU and fit in whole, the others in later segments).  Each
    request's results are those of a call of its own: bit for bit where that takes the same chunks at a time (up to 64 rows),
    else within two calls' rounding (2e-5 of a head's largest output, 1e-5 of a state)."""
    from gated_deltanet_tree_gb300 import runtime as R
    dims, gen, B, rows = R.make_dims(Hk, Hv, 128, 128, 4), torch.Generator(device="cuda").manual_seed(2), len(lens), sum(lens)
    C = R.channels(dims)

    def normal(*shape):
        return torch.empty(*shape, device="cuda").normal_(generator=gen)

    x, w = normal(rows, C).bfloat16(), 0.5 * normal(1, C, 4)
    beta, log_g = torch.sigmoid(normal(rows, Hv)).bfloat16(), -normal(rows, Hv).abs().bfloat16()
    state, conv = normal(B, 1, Hv, 128, 128), normal(B, 1, 3, C)
    s2, w2, out = torch.full_like(state, 5.0), torch.full_like(conv, 5.0), torch.empty(rows, Hv, 128, device="cuda")
    R.SequenceRunner(dims, B).prefill(lens, x, w, beta, log_g, state, conv, out, state_out=s2, conv_out=w2)
    own, at = R.SequenceRunner(dims, 1), 0
    for b, n in enumerate(lens):
        r = slice(at, at + n)
        at += n
        if n == 0:
            assert (s2[b] == 5.0).all() and (w2[b] == 5.0).all()
            continue
        s, v, o = torch.empty_like(s2[:1]), torch.empty_like(w2[:1]), torch.empty_like(out[r])
        own.prefill([n], x[r], w, beta[r], log_g[r], state[b:b + 1], conv[b:b + 1], o, state_out=s, conv_out=v)
        own.check_error()
        assert torch.equal(v[0], w2[b])
        if n <= 64:
            assert torch.equal(o, out[r]) and torch.equal(s[0], s2[b]), b
        else:
            assert ((o - out[r]).abs().amax((0, 2)) <= 2e-5 * o.abs().amax((0, 2))).all(), b
            assert ((s[0] - s2[b]).norm(dim=(2, 3)) <= 1e-5 * s[0].norm(dim=(2, 3))).all(), b
    # a head of each request against the oracle
    d = O.Dims(1, 1, 128, 128, 4, 1, 1, dims.q_scale, dims.l2_eps)
    h, at = Hv - 1, 0
    kh = h // (Hv // Hk)
    cols = torch.cat([torch.arange(128) + 128 * i for i in (kh, Hk + kh, 2 * Hk + h)]).cuda()
    for b, n in enumerate(lens[:8]):
        r = slice(at, at + n)
        at += n
        if n:
            o, T, _ = Q.run_sequence(f64(state[b, 0, h:h + 1]), f64(conv[b, 0][:, cols]), f64(x[r][:, cols]), f64(beta[r, h:h + 1]),
                                     f64(log_g[r, h:h + 1]), f64(w[0, cols]), d)
            assert np.abs(f64(out[r, h:h + 1]) - o).max() <= 2e-5 * np.abs(o).max(), b
            assert np.linalg.norm(f64(s2[b, 0, h]) - T[0]) <= 1e-5 * np.linalg.norm(T[0]), b


@pytest.mark.parametrize("what", ["state", "row", "gate", "columns"])
def test_a_request_that_is_not_finite_takes_no_longer(what):
    """A NaN state, or one from a NaN row or gate on, or with finite values in some columns only: no chunk is worth taking again
    (token by token, thirty times as slow), and other requests' results keep their bits."""
    c = Case(50, (1, 2, 128, 128), [2500, 2400], "bf16", slow=True, layers=1, layer=0)
    r, times, results = c.runner(), [], []
    for bad in (False, True):
        if bad and what == "state":
            c.state[0] = float("nan")
        elif bad and what == "columns":
            c.state[0, 0, :, :, :100] = float("nan")
        elif bad:
            (c.x if what == "row" else c.log_g)[70] = float("nan")
        best = float("inf")
        for _ in range(5):
            state, conv = torch.empty_like(c.state), torch.empty_like(c.conv)
            begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            begin.record()
            r.prefill(c.lens, *c.inputs(), c.state, c.conv, c.out, state_out=state, conv_out=conv)
            end.record()
            torch.cuda.synchronize()
            best = min(best, begin.elapsed_time(end))
        r.check_error()
        times.append(best)
        results.append((c.out.clone(), state))
    (out, state), (out2, state2) = results
    assert torch.equal(out[2500:], out2[2500:]) and torch.equal(state[1], state2[1])
    cols = slice(0, 100) if what == "columns" else slice(None)
    assert torch.isnan(out2[128:2500, :, cols]).all() and torch.isnan(state2[0, :, :, :, cols]).all()
    if what == "columns":
        for a, b in ((out[:2500, :, 100:], out2[:2500, :, 100:]), (state[0, ..., 100:], state2[0, ..., 100:])):
            assert (a - b).abs().max() <= 2e-5 * a.abs().max()     # (the largest entry, and with it the scale, may be another one)
    assert times[1] <= 2 * times[0], times


# ---- the library's own streams: programs of their own, which hold few streams -------------------------------------------

PROMPTS = """
import threading
import torch
from gated_deltanet_tree_gb300 import runtime as R
n, made = 3200, []
torch.manual_seed(5)
x = torch.randn(n, 512, device="cuda").bfloat16()
beta, log_g = torch.rand(n, 2, device="cuda").bfloat16(), -torch.rand(n, 2, device="cuda").bfloat16()
w = 0.5 * torch.randn(1, 512, 4, device="cuda")


class Prompt:
    def __init__(self):
        self.run, self.stream = R.SequenceRunner(R.make_dims(1, 2, 128, 128, 4), 1), torch.cuda.Stream()
        self.state, self.conv = torch.empty(1, 1, 2, 128, 128, device="cuda"), torch.empty(1, 1, 3, 512, device="cuda")
        self.out, self.end = torch.empty(n, 2, 128, device="cuda"), torch.cuda.Event()
        torch.cuda.synchronize()

    def call(self, wait=0):
        with torch.cuda.stream(self.stream):
            if wait:
                torch.cuda._sleep(wait)                        # ends by itself
            self.run.prefill([n], x, w, beta, log_g, None, None, self.out, state_out=self.state, conv_out=self.conv)
            self.end.record()

    def results(self):
        return [t.clone() for t in (self.out, self.state, self.conv)]


def same(a, b):
    return all(torch.equal(s, t) for s, t in zip(a, b))

"""


def program(text):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", PROMPTS + text], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_long_prompts_of_one_thread_do_not_wait_for_each_other():
    """A prompt behind work of 0.2 s or more on one stream; another one's on a second stream is done before it."""
    program("""
a, b = Prompt(), Prompt()
a.call()
torch.cuda.synchronize()
want = a.results()
for first, second in ((a, b), (b, a), (a, b)):
    for t in (*first.results(), *second.results()):
        t.zero_()
    first.call(wait=400_000_000)
    second.call()
    second.end.synchronize()
    assert not first.end.query()
    assert same(second.results(), want)
    torch.cuda.synchronize()
    assert same(first.results(), want)
""")


def test_more_long_prompts_at_work_than_the_library_has_streams():
    """Twelve streams' prompts at once, and again from a thread each: those that find none of the library's streams free give
    the same bits."""
    program("""
prompts = [Prompt() for _ in range(12)]
prompts[0].call()
torch.cuda.synchronize()
want = prompts[0].results()
for threads in (False, True, False):
    for p in prompts:
        for t in (p.out, p.state, p.conv):
            t.fill_(7.0)
    torch.cuda.synchronize()
    if threads:
        calls = [threading.Thread(target=p.call, args=(20_000_000,)) for p in prompts]
        for c in calls:
            c.start()
        for c in calls:
            c.join()
    else:
        for p in prompts:
            p.call(20_000_000)
    torch.cuda.synchronize()
    for p in prompts:
        p.run.check_error()
        assert same(p.results(), want)
""")


def test_threads_that_end_leave_nothing_behind():
    """A long prompt each from threads that end: the library's streams are the process's (a stream and its events take half a
    megabyte of device memory)."""
    program("""
p = Prompt()
p.call()
torch.cuda.synchronize()
before = torch.cuda.mem_get_info()[0]
for _ in range(100):
    t = threading.Thread(target=p.call)
    t.start()
    t.join()
torch.cuda.synchronize()
p.run.check_error()
assert before - torch.cuda.mem_get_info()[0] < 16 << 20
""")


def test_scores_on_the_default_stream_given_as_0():
    """Slices of tokens are copied on the stream that the call is given, also where that is the default stream's 0 and another
    one is current."""
    from gated_deltanet_tree_gb300.runtime import TokenScorer
    rng = np.random.default_rng(4)
    V, n = 501, 20
    z = rows_of(rng, n, V, "normal", "f32")
    tokens = torch.from_numpy(rng.integers(0, V, n).astype(np.int32)).cuda()
    s, late, other = TokenScorer(n, V, 3), torch.zeros_like(tokens), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                              # ends by itself, about 10 ms
    late.copy_(tokens)
    with torch.cuda.stream(other):
        s.score(z[:-1], late[1:], stream=0)
    torch.cuda.synchronize()
    s.check_error()
    check_scores(z[:-1], 3, (s.top[:n - 1], s.tokens[:n - 1], s.given[:n - 1], s.entropy[:n - 1]), tokens[1:])
