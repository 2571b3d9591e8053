"""What KV4Cache and TreeAcceptor pass to the library, and what they refuse (no GPU: the device calls are recorded)."""
import ctypes

import pytest
import torch


class Recorder:
    """The library with its device calls replaced: each records its arguments and returns `status`."""

    def __init__(self, real):
        self.real, self.calls, self.status = real, [], 0

    def __getattr__(self, name):
        if name not in ("gdn_kv4_append", "gdn_kv4_read", "gdn_kv4_attention", "gdn_tree_accept", "gdn_check_error_words"):
            return getattr(self.real, name)

        def call(*args):
            seen = []
            for a in args:
                a = getattr(a, "_obj", a)
                seen.append(type(a).from_buffer_copy(a) if isinstance(a, ctypes.Structure) else a)
            self.calls.append((name, seen))
            return self.status
        return call


@pytest.fixture()
def R(monkeypatch):
    from gated_deltanet_tree_gb300.build import build
    build()
    from gated_deltanet_tree_gb300 import _native as N
    from gated_deltanet_tree_gb300 import runtime
    rec = Recorder(N.lib())
    monkeypatch.setattr(N, "lib", lambda: rec)
    runtime.recorder = rec
    yield runtime
    del runtime.recorder


def make_cache(R, Hq=4, Hkv=2, D=64, B=2, layers=2, dtype=torch.bfloat16):
    return R.KV4Cache.empty(R.make_attn_dims(Hq, Hkv, D, dtype=dtype), B, layers, 2, device="cpu")


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def schedule(R, B, n):
    return R.DeviceSchedule([[-1] + list(range(n - 1))] * B, n, "cpu")


# ---- strides --------------------------------------------------------------------------------------------------------

def spread(shape, strides):
    """A tensor of that shape and those strides without memory behind it (nothing reads it)."""
    return torch.empty_strided(shape, strides, dtype=torch.bfloat16, device="meta")


@pytest.mark.parametrize("B,layers,n", [(2, 2, 3), (2, 1, 1), (1, 2, 1), (1, 1, 3)])
def test_repeated_rows_are_refused(R, B, layers, n):
    """Rows of stride 0 (a broadcast): the calls read a stride of 0 as contiguous rows, past the end of the memory."""
    c = make_cache(R, B=B, layers=layers)
    one = torch.zeros(1, 1, 1, 2, 64, dtype=torch.bfloat16)
    k = one.expand(B, layers, n, 2, 64)
    good = k.contiguous()
    q = torch.zeros(1, 1, 1, 4, 64, dtype=torch.bfloat16).expand(B, layers, n, 4, 64)
    out = torch.zeros(B, layers, n, 4, 64, dtype=torch.bfloat16)
    count, sched = i32(*[1] * B), schedule(R, B, n)
    for bad in (lambda: c.append(k, k, count, stream=0), lambda: c.append(good, k, count, stream=0),
                lambda: c.attention(q, good, good, out, sched=sched, stream=0),
                lambda: c.attention(out, k, k, out, sched=sched, stream=0)):
        with pytest.raises(ValueError, match="broadcast|row strides"):
            bad()
    assert not R.recorder.calls


def test_overlapping_rows_are_refused(R):
    c = make_cache(R, B=1, layers=1)
    flat = torch.zeros(64 * 16, dtype=torch.bfloat16)
    k = flat.as_strided((1, 1, 3, 2, 64), (192, 192, 64, 64, 1))
    with pytest.raises(ValueError):
        c.append(k, k, i32(1), stream=0)
    assert not R.recorder.calls


def test_far_rows_are_refused(R):
    """A stride beyond 32 bits: ctypes would cut it to its low bits."""
    far = (1 << 32) + 128
    assert R._row_stride(spread((2, 1, 1, 2, 64), (640, 640, 640, 64, 1)), "k", (2, 1, 1, 2, 64)) == 640
    with pytest.raises(ValueError):
        R._row_stride(spread((2, 1, 1, 2, 64), (far, far, far, 64, 1)), "k", (2, 1, 1, 2, 64))
    acc = R.TreeAcceptor(2, 1, 100, device="cpu")
    acc._index = spread((1,), (1,)).get_device()
    assert acc._rows(spread((2, 1, 100), (128, 128, 1)), "logits") == 128
    with pytest.raises(ValueError):
        acc._rows(spread((2, 1, 100), (far, far, 1)), "logits")


@pytest.mark.parametrize("B,n", [(2, 3), (1, 3), (2, 1)])
def test_repeated_logits_are_refused(R, B, n):
    acc = R.TreeAcceptor(B, n, 100, device="cpu")
    z = torch.zeros(1, 1, 100).expand(B, n, 100)
    tokens, sched = torch.zeros(B, n, dtype=torch.int32), schedule(R, B, n)
    args = (torch.zeros(B, n), torch.zeros(B, 100), torch.ones(B))
    for bad in (lambda: acc.accept(sched, z, tokens, *args, stream=0),
                lambda: acc.accept(sched, z.contiguous(), tokens, *args, draft_probs=z, stream=0)):
        with pytest.raises(ValueError):
            bad()
    assert not R.recorder.calls
    acc.accept(sched, z.contiguous(), tokens, *args, stream=0)
    assert [name for name, _ in R.recorder.calls] == ["gdn_tree_accept"]


def test_row_strides_are_a_calls_own(R):
    """Rows of a fused projection, then contiguous rows, then no new rows: each call passes its own strides, and neither
    a served nor a refused one leaves any behind."""
    c = make_cache(R, B=1, layers=1)
    wide = torch.zeros(1, 1, 3, 10, 64, dtype=torch.bfloat16)
    q, k, v = wide[..., :4, :], wide[..., 4:6, :], wide[..., 6:8, :]
    out, count, sched = torch.zeros(1, 1, 3, 4, 64, dtype=torch.bfloat16), i32(1), schedule(R, 1, 3)

    def strides(call):
        call()
        d = R.recorder.calls[-1][1][0]
        assert (c.dims.q_row, c.dims.kv_row) == (0, 0)
        return d.q_row or 4 * 64, d.kv_row or 2 * 64

    kc, vc = k.contiguous(), v.contiguous()
    assert strides(lambda: c.attention(q, k, v, out, sched=sched, stream=0)) == (640, 640)
    assert strides(lambda: c.attention(out, k, v, out, sched=sched, stream=0)) == (256, 640)
    assert strides(lambda: c.attention(q, None, None, out, sched=sched, stream=0)) == (640, 128)
    assert strides(lambda: c.attention(out, kc, vc, out, sched=sched, stream=0)) == (256, 128)
    assert strides(lambda: c.append(k, v, count, stream=0)) == (256, 640)
    assert strides(lambda: c.append(kc, vc, count, stream=0)) == (256, 128)
    R.recorder.status = -1                                  # (the library refuses, as it does rows of odd strides)
    for call in (lambda: c.attention(q, k, v, out, sched=sched, stream=0), lambda: c.append(k, v, count, stream=0)):
        with pytest.raises(R.N.GdnError):
            call()
        assert (c.dims.q_row, c.dims.kv_row) == (0, 0)


@pytest.mark.parametrize("status,zeroed", [(-6, True), (-9, False), (-10, False)])
def test_workspace_is_zeroed_after_a_timeout(R, status, zeroed):
    c = make_cache(R)
    c.check_error(stream=0)
    c.workspace[:] = 3
    R.recorder.status = status
    with pytest.raises(R.N.GdnError) as e:
        c.check_error(stream=0)
    assert e.value.status == status and bool((c.workspace == (0 if zeroed else 3)).all())


# ---- sizes ----------------------------------------------------------------------------------------------------------

def test_vocabularies_beyond_the_index_range_are_refused(R):
    """The kernels' 32-bit indices run past V by a cluster's step; at 2^31 - 1 they would turn negative."""
    from gated_deltanet_tree_gb300 import _native as N
    P = 0x10000          # never dereferenced
    lib, sched = R.recorder.real, N.gdn_batch_schedule(B=1, n_max=1, nb_max=0, depth_max=0, words=P)
    for V in ((1 << 30) + 1, (1 << 31) - 1):
        assert N.gdn_accept_workspace_bytes(1, 1, V) == 0
        assert lib.gdn_tree_accept(ctypes.byref(sched), V, 0, 0, P, P, None, 0, P, P, P, P, P, P, P, P, 1 << 40,
                                   0) == N.GDN_ERR_UNSUPPORTED
    assert N.gdn_accept_workspace_bytes(1, 2, 1 << 30) > 0


# ---- workspace ------------------------------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("Hq,Hkv,D", [(24, 4, 256), (8, 2, 128), (4, 2, 64)])
def test_one_workspace_serves_every_call(R, Hq, Hkv, D, dtype):
    """Single tokens, then trees and longer requests: the same memory from the first call on (a kernel in flight or a
    captured graph may hold it), large enough for each, and nothing kept by the lengths that were passed."""
    from gated_deltanet_tree_gb300 import _native as N
    c = make_cache(R, Hq, Hkv, D, dtype=dtype)
    kept = {name: value for name, value in vars(c).items()}
    for n, max_len in ((1, 1), (1, 100), (2, 0), (8, 4096), (22, 0), (64, 1 << 20), (64, 0), (1, 7)):
        q = torch.zeros(2, 2, n, Hq, D, dtype=dtype)
        k = torch.zeros(2, 2, n, Hkv, D, dtype=dtype)
        c.attention(q, k, k, torch.zeros_like(q), sched=None if n == 1 else schedule(R, 2, n), max_len=max_len, stream=0)
        _, args = R.recorder.calls[-1]
        assert args[9:11] == [kept["workspace"].data_ptr(), kept["workspace"].numel()]
        assert args[10] >= N.gdn_kv4_workspace_bytes(c.dims, 2, 2, n, max_len) > 0
    assert vars(c).keys() == kept.keys() and all(vars(c)[x] is kept[x] for x in kept)
    assert not any(isinstance(x, dict) for x in kept.values())


def test_kernel_choice_is_at_the_measured_crossings(R):
    """Few rows a kv head leave partial results of 8 rows, 304 CTAs; more rows of 128 rows, 152 CTAs."""
    from gated_deltanet_tree_gb300 import _native as N
    records = 16384 * 4 + 4096 * 16
    for D, most in ((256, 16), (128, 20), (64, 28)):
        for rows in range(1, 65):
            few = records + 304 * 2 * 8 * (D + 2) * 4
            many = records + 152 * 2 * 128 * (D + 2) * 4
            got = N.gdn_kv4_workspace_bytes(R.make_attn_dims(2, 2, D), 2, 1, rows, 0)
            assert got == (few if rows <= most else many), (D, rows)
            assert N.gdn_kv4_workspace_bytes(R.make_attn_dims(2, 2, D, dtype=torch.float32), 2, 1, rows, 0) == few


def test_acceptance_reduces_all_rows_at_once_while_they_are_few(R):
    """The workspace holds 16 bytes for each slice of 8192 entries, up to 2^26 entries (the limit with draft
    probabilities), and next to nothing beyond that or where there is no child."""
    from gated_deltanet_tree_gb300 import _native as N
    for B, n, V, slices in ((1, 22, 131072, 16), (4, 64, 131072, 16), (64, 16, 65536, 8), (64, 16, 65537, 0), (70000, 2, 100, 0),
                            (5, 1, 1000, 0)):
        need = B * n * slices * 16 + 1
        assert N.gdn_accept_workspace_bytes(B, n, V) == -(-need // 256) * 256
