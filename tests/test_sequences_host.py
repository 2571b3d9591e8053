"""Refusals of the prompt, single-token and log-probability calls, and what their Python side passes on (no GPU)."""
import ctypes

import numpy as np
import pytest
import torch

P = 0x10000          # never dereferenced: 16-byte aligned
BIG = 1 << 40


@pytest.fixture(scope="module")
def N():
    from gated_deltanet_tree_gb300.build import build
    build()
    from gated_deltanet_tree_gb300 import _native
    _native.lib()
    return _native


def dims(N, **kw):
    d = dict(Hk=2, Hv=4, dk=64, dv=64, K=4, conv_mode=1, act=1, in_dtype=N.GDN_DTYPE_BF16, q_scale=1.0, l2_eps=1e-6)
    d.update(kw)
    return N.gdn_dims(**d)


def banks(N, **kw):
    b = N.gdn_banks()
    N.gdn_banks_init(b, 2, 3, 8)
    for k, v in kw.items():
        setattr(b, k, v)
    return b


def status(N, fn):
    with pytest.raises(N.GdnError) as e:
        fn()
    assert str(e.value).split(": ", 1)[1]
    return e.value.status


def both(N, d=None, **kw):
    """The two calls with the same arguments, some of them replaced."""
    d = dims(N) if d is None else d
    a = dict(layers=3, layer=1, lens=[70, 2], B=2, x=P, x_row=0, w=P, beta=P, log_g=P, gate_row=0, state=BIG, conv=2 * BIG,
             state_out=3 * BIG, conv_out=4 * BIG, out=P, out_dtype=0, banks=None, err=P, ws=P, ws_bytes=BIG, live=None)
    a.update(kw)
    shared = (a["x"], a["x_row"], a["w"], a["beta"], a["log_g"], a["gate_row"], a["state"], a["conv"], a["state_out"],
              a["conv_out"], a["out"], a["out_dtype"], a["banks"], a["err"])
    return (lambda: N.gdn_prefill(d, a["layers"], a["layer"], a["lens"], *shared, a["ws"], a["ws_bytes"], 0),
            lambda: N.gdn_step(d, a["layers"], a["layer"], a["B"], a["live"], *shared, 0))


BAD = [(dict(layers=0), -1), (dict(layer=3), -1), (dict(layer=-1), -1), (dict(x=None), -1), (dict(x=P + 8), -1),
       (dict(x_row=504), -1), (dict(x_row=516), -1), (dict(x_row=1 << 31), -1), (dict(w=None), -1), (dict(w=P + 4), -1),
       (dict(beta=None), -1), (dict(log_g=P + 1), -1), (dict(gate_row=3), -1), (dict(state=P + 4), -1), (dict(conv=P + 8), -1),
       (dict(state_out=None), -1), (dict(conv_out=None), -1), (dict(conv_out=P + 8), -1), (dict(out=None), -1),
       (dict(out_dtype=2), -1), (dict(err=None), -1),
       # outputs that overlap what they come from without being it
       (dict(state_out=BIG + 64), -1), (dict(conv_out=2 * BIG + 1024), -1)]


@pytest.mark.parametrize("change,want", BAD)
def test_arguments_refused_by_both_calls(N, change, want):
    for call in both(N, **change):
        assert status(N, call) == want


@pytest.mark.parametrize("change,want", [(dict(Hk=3), -1), (dict(dk=96), -4), (dict(dv=256), -4), (dict(K=9), -4), (dict(K=0), -4),
                                         (dict(conv_mode=2), -1), (dict(act=3), -1), (dict(in_dtype=7), -1),
                                         (dict(q_scale=float("nan")), -1), (dict(l2_eps=-1.0), -1), (dict(Hk=1 << 18, Hv=1 << 18), -4)])
def test_dims_refused(N, change, want):
    for call in both(N, dims(N, **change)):
        assert status(N, call) == want
    if want == -4 and "Hk" not in change:
        assert N.gdn_prefill_workspace_bytes(dims(N, **change)) == 0


def test_lengths_and_workspace_refused(N):
    d = dims(N)
    assert status(N, both(N, lens=[3, -1])[0]) == -1
    assert status(N, both(N, lens=[(1 << 31) - 1, (1 << 31) - 1])[0]) == -4
    assert status(N, both(N, ws=None)[0]) == -1
    need = N.gdn_prefill_workspace_bytes(d)
    assert 0 < need < 1 << 31
    assert status(N, both(N, ws_bytes=need - 1)[0]) == -7
    assert status(N, both(N, lens=[])[0]) == -1
    assert status(N, both(N, B=0)[1]) == -1
    assert status(N, both(N, live=P + 4)[1]) == -1
    assert N._check(N.lib().gdn_prefill(ctypes.byref(d), 3, 0, 2, (ctypes.c_int32 * 2)(0, 0), P, 0, P, P, P, 0, None, None, P, P,
                                        P, 0, None, P, P, need, None)) is None       # nothing to do: nothing is launched


def test_states_that_trees_hold_back_are_refused(N):
    for change, want in [(dict(verified_bank=0), N.GDN_ERR_STATE), (dict(pend_bank=1, write_bank=0), N.GDN_ERR_STATE),
                         (dict(B=3), N.GDN_ERR_CAPACITY), (dict(layers=2), N.GDN_ERR_CAPACITY)]:
        for call in both(N, banks=banks(N, **change)):
            assert status(N, call) == want


@pytest.mark.parametrize("change,want", [
    (dict(rows=0), -1), (dict(V=0), -1), (dict(V=(1 << 30) + 1), -4), (dict(v_stride=999), -1), (dict(dtype=3), -1), (dict(top=0), -1),
    (dict(V=10, v_stride=0, top=11), -1), (dict(top=33), -4), (dict(logits=None), -1), (dict(logits=P + 2), -1), (dict(tokens=None), -1),
    (dict(given=None), -1), (dict(tokens=P + 4), -1), (dict(top_logp=None), -1), (dict(top_token=P + 8), -1), (dict(entropy=P + 4), -1),
    (dict(err=None), -1), (dict(rows=1 << 29), -4), (dict(rows=1 << 20, v_stride=1 << 60), -4)])
def test_log_probability_arguments_refused(N, change, want):
    a = dict(rows=4, V=1000, v_stride=1000, dtype=0, logits=P, tokens=P, top=4, top_logp=P, top_token=P, given=P, entropy=P, err=P)
    a.update(change)
    assert status(N, lambda: N.gdn_top_logprobs(a["rows"], a["V"], a["v_stride"], a["dtype"], a["logits"], a["tokens"], a["top"],
                                                a["top_logp"], a["top_token"], a["given"], a["entropy"], a["err"], 0)) == want


# ---- the Python side ------------------------------------------------------------------------------------------------

class Recorder:
    """The library with its device calls replaced: each records its arguments."""

    def __init__(self, real):
        self.real, self.calls = real, []

    def __getattr__(self, name):
        if name not in ("gdn_prefill", "gdn_step", "gdn_top_logprobs"):
            return getattr(self.real, name)

        def call(*args):
            self.calls.append((name, [list(a[:2]) if isinstance(a, (ctypes._Pointer, ctypes.Array)) else a for a in args]))
            return 0
        return call


@pytest.fixture()
def R(N, monkeypatch):
    from gated_deltanet_tree_gb300 import runtime
    rec = Recorder(N.lib())
    monkeypatch.setattr(N, "lib", lambda: rec)
    runtime.recorder = rec
    yield runtime
    del runtime.recorder


def tensors(rows=5, C=512, Hv=4, B=2, layers=3):
    bf = dict(dtype=torch.bfloat16)
    return dict(x_raw=torch.zeros(rows, C, **bf), conv_w=torch.zeros(layers, C, 4), beta=torch.zeros(rows, Hv, **bf),
                log_g=torch.zeros(rows, Hv, **bf), state=torch.zeros(B, layers, Hv, 64, 64), conv_state=torch.zeros(B, layers, 3, C),
                out=torch.zeros(rows, Hv, 64))


def test_what_the_runner_passes(N, R):
    r = R.SequenceRunner(dims(N), 2, 3, device="cpu")
    t = tensors()
    r.prefill([5, 0], **t, layer=2, stream=7)
    wide = torch.zeros(5, 600, dtype=torch.bfloat16)
    t["x_raw"], gates = wide[:, 16:528], torch.zeros(5, 2, 4, dtype=torch.bfloat16)
    t["beta"], t["log_g"] = gates[:, 0], gates[:, 1]
    s2, c2 = torch.zeros_like(t["state"]), torch.zeros_like(t["conv_state"])
    r.prefill(np.array([2, 3]), **dict(t, out=t["out"].bfloat16()), state_out=s2, conv_out=c2, stream=7)
    (_, a), (_, b) = R.recorder.calls
    assert a[1:5] == [3, 2, 2, [5, 0]] and a[6] == 512 and a[10] == 4 and a[16] == N.GDN_DTYPE_F32 and a[-1] == 7
    assert a[11] == a[13] == t["state"].data_ptr() and a[12] == a[14] == t["conv_state"].data_ptr()
    assert b[4] == [2, 3] and b[6] == 600 and b[10] == 8 and b[13:15] == [s2.data_ptr(), c2.data_ptr()] and b[16] == N.GDN_DTYPE_BF16
    u = tensors(rows=2)
    r.step(**u, live=torch.ones(2, dtype=torch.int32), stream=7)
    r.prefill([0, 0], **tensors(rows=0), stream=7)                     # nothing to do
    assert [c[0] for c in R.recorder.calls] == ["gdn_prefill", "gdn_prefill", "gdn_step"]


def test_what_the_runner_refuses(N, R):
    r = R.SequenceRunner(dims(N), 2, 3, device="cpu")
    t = tensors()
    i32 = dict(dtype=torch.int32)
    bad = [dict(x_raw=t["x_raw"].float()), dict(x_raw=t["x_raw"][:4]), dict(x_raw=torch.zeros(5, 512, 2, dtype=torch.bfloat16)[..., 0]),
           dict(x_raw=torch.zeros(1, 512, dtype=torch.bfloat16).expand(5, -1)), dict(beta=t["beta"][:, :3]), dict(log_g=t["log_g"].float()),
           dict(log_g=torch.zeros(5, 8, dtype=torch.bfloat16)[:, :4]), dict(conv_w=t["conv_w"][:2]), dict(conv_w=t["conv_w"].bfloat16()),
           dict(state=t["state"].bfloat16()), dict(state=t["state"][:1]), dict(state=t["state"].transpose(3, 4)),
           dict(conv_state=t["conv_state"][:, :, :2]), dict(out=t["out"][:4]), dict(out=torch.zeros(5, 64, 4).transpose(1, 2)),
           dict(state=None), dict(conv_state=None)]
    for change in bad:
        with pytest.raises((ValueError, TypeError)):
            r.prefill([5, 0], **dict(t, **change), stream=7)
    for lens in ([5], [4, 0], [1, 2, 2]):
        with pytest.raises(ValueError):
            r.prefill(lens, **t, stream=7)
    with pytest.raises(TypeError):
        r.prefill([5, 0], **dict(t, out=t["out"].half()), stream=7)
    u = tensors(rows=2)
    for live in (torch.ones(3, **i32), torch.ones(2), torch.ones(4, **i32)[::2]):
        with pytest.raises(ValueError):
            r.step(**u, live=live, stream=7)
    with pytest.raises(ValueError):
        R.SequenceRunner(dims(N), 2, 3, device="cpu", prompts=False).prefill([5, 0], **t, stream=7)
    assert not R.recorder.calls


def test_what_the_scorer_passes_and_refuses(N, R):
    s = R.TokenScorer(6, 100, 4, device="cpu")
    z = torch.zeros(6, 100)
    top, best, given, entropy = s.score(z, torch.zeros(6, dtype=torch.int32), stream=7)
    assert top.shape == (6, 4) and best.shape == (6, 4) and given.shape == entropy.shape == (6,)
    top, _, given, _ = s.score(torch.zeros(3, 140).bfloat16()[:, 8:108], stream=7)
    assert top.shape == (3, 4) and given is None
    (_, a), (_, b) = R.recorder.calls
    assert a[:4] == [6, 100, 100, N.GDN_DTYPE_F32] and a[6] == 4 and b[:4] == [3, 100, 140, N.GDN_DTYPE_BF16] and b[5] is None
    for bad in (torch.zeros(7, 100), torch.zeros(0, 100), torch.zeros(6, 99), torch.zeros(100), torch.zeros(1, 100).expand(6, -1),
                torch.zeros(6, 100, 2)[..., 0]):
        with pytest.raises(ValueError):
            s.score(bad, stream=7)
    with pytest.raises(TypeError):
        s.score(z.half(), stream=7)
    for tokens in (torch.zeros(6), torch.zeros(5, dtype=torch.int32), torch.zeros(12, dtype=torch.int32)[::2]):
        with pytest.raises(ValueError):
            s.score(z, tokens, stream=7)
    for args in ((6, 100, 0), (6, 100, 33), (6, 3, 4)):
        with pytest.raises(ValueError):
            R.TokenScorer(*args, device="cpu")
    assert len(R.recorder.calls) == 2
