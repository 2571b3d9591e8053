"""Refusals of the cache, attention and acceptance entry points (no GPU: every call fails a host check first)."""
import ctypes

import pytest

P = 0x10000          # never dereferenced: 16-byte aligned


@pytest.fixture(scope="module")
def N():
    from gated_deltanet_tree_gb300.build import build
    build()
    from gated_deltanet_tree_gb300 import _native
    _native.lib()
    return _native


def dims(N, **kw):
    d = dict(Hq=8, Hkv=2, D=128, dtype=N.GDN_DTYPE_BF16, scale=0.1, q_row=0, kv_row=0)
    d.update(kw)
    return N.gdn_attn_dims(**d)


def cache(N, **kw):
    d = dict(pool=P, page_table=P, seq_len=P, ticket=P, err=P, B=2, layers=1, pages_max=4, n_pages=8)
    d.update(kw)
    return N.gdn_kv4_cache(**d)


def sched(N, **kw):
    d = dict(B=2, n_max=8, nb_max=0, depth_max=0, words=P)
    d.update(kw)
    return N.gdn_batch_schedule(**d)


def status(N, fn, *a, **kw):
    with pytest.raises(N.GdnError) as e:
        fn(*a, **kw)
    assert str(e.value).split(": ", 1)[1]
    return e.value.status


BAD_DIMS = [(dict(Hq=0), -1), (dict(Hkv=0), -1), (dict(Hq=9), -1), (dict(Hq=2048, Hkv=2), -4), (dict(D=96), -4),
            (dict(D=0), -4), (dict(dtype=2), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
            (dict(q_row=1000), -1), (dict(q_row=1025), -1), (dict(kv_row=128), -1), (dict(kv_row=260), -1)]
BAD_CACHE = [(dict(pool=None), -1), (dict(page_table=P + 4), -1), (dict(seq_len=None), -1), (dict(ticket=None), -1),
             (dict(err=None), -1), (dict(B=0), -1), (dict(layers=0), -1), (dict(layers=2), -7), (dict(pages_max=0), -1),
             (dict(n_pages=0), -1), (dict(pages_max=1 << 26), -4), (dict(n_pages=1 << 31), -4)]


def calls(N, d, c, **kw):
    a = dict(layers=1, n=8, k=P, v=P, q=P, out=P, path=P, count=P, s=sched(N), ws=P, ws_bytes=1 << 40, max_len=0)
    a.update(kw)
    return {
        "append": lambda: N.gdn_kv4_append(d, a["layers"], a["n"], a["k"], a["v"], a["path"], a["count"], c, 0),
        "read": lambda: N.gdn_kv4_read(d, a["layers"], a["n"], None, a.get("od", 0), a["k"], a["v"], c, 0),
        "attention": lambda: N.gdn_kv4_attention(d, a["layers"], a["s"], a["q"], a["k"], a["v"], a["out"], c,
                                                 a["max_len"], a["ws"], a["ws_bytes"], 0)}


@pytest.mark.parametrize("name", ["append", "read", "attention"])
def test_bad_dims_and_caches(N, name):
    for kw, want in BAD_DIMS:
        assert status(N, calls(N, dims(N, **kw), cache(N))[name]) == want, kw
    for kw, want in BAD_CACHE:
        assert status(N, calls(N, dims(N), cache(N, **kw))[name]) == want, kw


def test_bad_arguments(N):
    d, c = dims(N), cache(N)
    for name, kw, want in [
            ("append", dict(n=0), -1), ("append", dict(n=(1 << 21) + 1), -1), ("append", dict(k=None), -1),
            ("append", dict(v=P + 8), -1), ("append", dict(count=None), -1), ("append", dict(path=P + 2), -1),
            ("append", dict(layers=0), -7), ("read", dict(n=0), -1), ("read", dict(od=2), -1),
            ("read", dict(k=None), -1), ("read", dict(v=P + 4), -1), ("attention", dict(q=None), -1),
            ("attention", dict(out=P + 8), -1), ("attention", dict(k=None), -1), ("attention", dict(v=None), -1),
            ("attention", dict(max_len=-1), -1), ("attention", dict(ws=None), -1),
            ("attention", dict(ws_bytes=0), -7), ("attention", dict(s=sched(N, B=3)), -7),
            ("attention", dict(s=sched(N, n_max=65)), -4), ("attention", dict(s=sched(N, words=None)), -1)]:
        assert status(N, calls(N, d, c, **kw)[name]) == want, (name, kw)


def test_sizes(N):
    d = dims(N)
    assert N.gdn_kv4_pool_bytes(d, 3, 5) == 3 * 5 * 2 * 72 * 128
    assert N.gdn_kv4_pool_bytes(d, 0, 5) == 0 and N.gdn_kv4_pool_bytes(dims(N, D=32), 1, 1) == 0
    assert N.gdn_kv4_pool_bytes(dims(N, Hq=4, Hkv=4, D=256), 64, 1 << 20) == (1 << 20) * 64 * 4 * 72 * 256
    for dt in (0, 1):
        for n in (1, 22, 64):
            for length in (0, 1, 4096, 1 << 20):
                assert N.gdn_kv4_workspace_bytes(dims(N, dtype=dt), 2, 1, n, length) > 0
    assert N.gdn_kv4_workspace_bytes(d, 0, 1, 1, 1) == 0 and N.gdn_kv4_workspace_bytes(d, 1, 1, 65, 1) == 0
    assert N.gdn_accept_workspace_bytes(1, 22, 100) > 0 and N.gdn_accept_workspace_bytes(1, 65, 100) == 0
    assert ctypes.sizeof(N.gdn_kv4_cache) == 64 and ctypes.sizeof(N.gdn_attn_dims) == 28


def test_accept_refusals(N):
    base = dict(s=sched(N), V=100, stride=0, ld=0, z=P, tok=P, dp=None, dd=0, u=P, g=P, t=P, path=P, len=P, nxt=P,
                err=P, ws=P, ws_bytes=1 << 40)

    def call(**kw):
        a = dict(base, **kw)
        return lambda: N.gdn_tree_accept(a["s"], a["V"], a["stride"], a["ld"], a["z"], a["tok"], a["dp"], a["dd"],
                                         a["u"], a["g"], a["t"], a["path"], a["len"], a["nxt"], a["err"], a["ws"],
                                         a["ws_bytes"], 0)

    for kw, want in [(dict(V=0), -1), (dict(stride=99), -1), (dict(ld=2), -1), (dict(dp=P, dd=5), -1),
                     (dict(z=None), -1), (dict(tok=P + 4), -1), (dict(dp=P + 4), -1), (dict(u=None), -1),
                     (dict(g=None), -1), (dict(t=P + 4), -1), (dict(path=None), -1), (dict(len=None), -1),
                     (dict(nxt=None), -1), (dict(err=None), -1), (dict(ws=None), -1), (dict(ws_bytes=0), -7),
                     (dict(s=sched(N, n_max=0)), -4), (dict(s=sched(N, B=0)), -1)]:
        assert status(N, call(**kw)) == want, kw


def test_error_words_pointer(N):
    assert status(N, N.gdn_check_error_words, None, 0) == -1


def test_attention_with_too_many_items(N):
    d, c = dims(N, Hq=1024, Hkv=512, dtype=N.GDN_DTYPE_F32), cache(N, layers=5)
    assert N.gdn_kv4_workspace_bytes(d, 2, 5, 64, 100) == 0
    assert status(N, calls(N, d, c, layers=5, s=sched(N, n_max=64))["attention"]) == -4
