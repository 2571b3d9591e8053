"""Prompt, single-token and log-probability calls on a GPU, beside test_gpu_sequences.py and test_gpu_sequences_calls.py, whose
tolerances these tests use."""
import numpy as np
import pytest
import torch

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
