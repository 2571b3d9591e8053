"""Pins of the oracles of the 4-bit cache, its attention and the acceptance walk (CPU, no library)."""
import numpy as np
import pytest
import torch

from oracle import accept_oracle as A
from oracle import kv4_oracle as K


# ---- 4-bit groups ---------------------------------------------------------------------------------------------------

def test_bf16_rounding_is_torchs():
    x = np.random.default_rng(0).standard_normal(2000) * 10.0 ** np.random.default_rng(1).integers(-6, 6, 2000)
    want = torch.from_numpy(x.astype(np.float32)).bfloat16().double().numpy()
    assert [K.round_bf16(float(np.float32(v))) for v in x] == want.tolist()


def test_group_extremes_and_errors():
    rng = np.random.default_rng(2)
    for _ in range(200):
        x = torch.from_numpy(rng.standard_normal(32).astype(np.float32)).bfloat16().double().numpy()
        c, d = K.quantise_group(x)
        i = int(np.argmax(np.abs(x)))
        assert c[i] == -8 and c[i] * d == x[i]                    # the largest magnitude is exact
        assert d == -x[i] / 8
        same = np.sign(x) == np.sign(x[i])
        assert np.all(np.abs(c * d - x)[same] <= abs(d) / 2)
        assert np.all(np.abs(c * d - x) <= abs(d))                # the other extreme may need the missing code 8
        assert c.min() >= -8 and c.max() <= 7


def test_group_ties_zero_and_non_finite():
    x = np.zeros(32)
    assert K.quantise_group(x)[1] == 0
    x[3], x[9] = -2.0, 2.0                 # the lower channel decides the sign
    c, d = K.quantise_group(x)
    assert d == 0.25 and c[3] == -8 and c[9] == 7
    x[3], x[9] = 2.0, -2.0
    assert K.quantise_group(x)[1] == -0.25
    for bad in (np.nan, np.inf, -np.inf):
        x[20] = bad
        assert np.isnan(K.quantise_group(x)[1])
    assert abs(K.quantise_group(np.full(32, 1e6))[1]) == 2720.0


def test_block_words_by_hand():
    # one code set at a time: D = 64, token 5 channel 35 (key), token 41 channel 6 (value)
    D = 64
    b = np.zeros(72 * D, dtype=np.uint8)
    b.view("<f2")[16 * D:18 * D] = 1.0
    b.view("<f2")[34 * D:] = 1.0
    w = b.view("<u4")
    w[:8 * D] = 0x88888888
    w[9 * D:17 * D] = 0x88888888
    # token 5: turn (5 >> 2) & 1 = 1, chunk 1 sits at place 0; channel 35 = element 3 of word 0 of the chunk: nibble 5
    w[5 * 8 + 0] = 0x88888888 ^ (0xB << 20)       # 8 ^ 11 = 3: code -5
    # token 41: octet 5 -> half 1, place 1; channel 6: quad 1, second of it; element 1: nibble 4
    w[9 * D + ((1 * 16 + 1) * 4 + 1) * 4 + 2] = 0x88888888 ^ (0x7 << 16)   # 8 ^ 7 = 15: code 7
    k, v = K.block_rows(b, D)
    assert k[5, 35] == -5 and np.count_nonzero(k) == 1
    assert v[41, 6] == 7 and np.count_nonzero(v) == 1


# ---- attention ------------------------------------------------------------------------------------------------------

def test_attention_closed_forms():
    rng = np.random.default_rng(3)
    v = rng.standard_normal((7, 4))
    assert np.allclose(K.attention_row(np.zeros(4), rng.standard_normal((7, 4)), v, 1.0), v.mean(0), atol=1e-15)
    k = np.zeros((7, 4))
    k[5, 0] = 1.0
    assert np.allclose(K.attention_row(np.array([1e4, 0, 0, 0]), k, v, 1.0), v[5], atol=1e-12)
    assert np.all(K.attention_row(np.ones(4), np.zeros((0, 4)), np.zeros((0, 4)), 1.0) == 0)
    q, k = rng.standard_normal(4), rng.standard_normal((7, 4))
    want = torch.softmax(torch.from_numpy(0.3 * (k @ q)), 0).numpy() @ v
    assert np.allclose(K.attention_row(q, k, v, 0.3), want, atol=1e-14)


def test_tree_attention_sees_root_paths_only():
    rng = np.random.default_rng(4)
    parent = [-1, 0, 1, 0, 3, 1]
    q, kn, vn = (rng.standard_normal(s) for s in ((6, 4, 8), (6, 2, 8), (6, 2, 8)))
    k, v = rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    base = K.tree_attention(q, k, v, kn, vn, parent, 0.5)
    for j in range(6):
        kn2, vn2 = kn.copy(), vn.copy()
        kn2[j], vn2[j] = np.nan, np.nan
        with np.errstate(invalid="ignore"):
            got = K.tree_attention(q, k, v, kn2, vn2, parent, 0.5)
        for i in range(6):
            assert (j in K.root_path(parent, i)) == bool(np.isnan(got[i]).any())
            if j not in K.root_path(parent, i):
                assert np.array_equal(got[i], base[i])


# ---- acceptance -----------------------------------------------------------------------------------------------------

def _first_token(path, nxt, tokens):
    return tokens[path[1]] if len(path) > 1 else nxt


@pytest.mark.parametrize("temperature", [1.0, 0.6])
@pytest.mark.parametrize("sampled", [False, True])
def test_walk_samples_the_target(sampled, temperature):
    """Whatever was drafted, the token after the root is distributed as the target's softmax: 4.5 standard deviations
    of a binomial count over 20000 walks (a miss in 20 checks has probability below 2e-4)."""
    rng = np.random.default_rng(5)
    V, N = 5, 20000
    logits = rng.standard_normal((4, V)) * 1.5
    q = np.tile(A.softmax(rng.standard_normal(V)), (4, 1))
    parent = [-1, 0, 0, 0]
    counts = np.zeros(V)
    for _ in range(N):
        tokens = [0] + (rng.choice(V, 3, p=q[0]).tolist() if sampled else [1, 4, 1])
        g = -np.log(-np.log(rng.random(V)))
        path, nxt = A.accept(parent, tokens, logits, rng.random(4), g, temperature, q if sampled else None)
        counts[_first_token(path, nxt, tokens)] += 1
    p = A.softmax(logits[0] / temperature)
    assert np.all(np.abs(counts - N * p) <= 4.5 * np.sqrt(N * p * (1 - p)))


def test_greedy_walk_by_hand():
    logits = np.zeros((5, 6))
    logits[0, 2] = logits[0, 4] = 3.0      # the lowest index of the largest: 2
    logits[2, 5] = 1.0
    logits[4, 1] = 1.0
    parent, tokens = [-1, 0, 0, 1, 2], [0, 4, 2, 5, 5]
    assert A.accept(parent, tokens, logits, None, None, 0.0) == ([0, 2, 4], 1)
    logits[4, 0] = np.nan
    assert A.accept(parent, tokens, logits, None, None, 0.0) == ([0, 2, 4], -1)
    assert A.accept([-1], [0], np.full((1, 3), -np.inf), None, None, 0.0) == ([0], -1)


def test_equal_distributions_accept_everything():
    rng = np.random.default_rng(6)
    z = rng.standard_normal((6, 9))
    q = np.stack([A.softmax(r) for r in z])
    parent = [-1, 0, 1, 2, 3, 4]
    for _ in range(50):
        path, _ = A.accept(parent, rng.integers(0, 9, 6).tolist(), z, rng.random(6) * (1 - 1e-9),
                           -np.log(-np.log(rng.random(9))), 1.0, q)
        assert path == [0, 1, 2, 3, 4, 5]
