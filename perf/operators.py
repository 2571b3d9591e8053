"""Timed cases of the operators around a tree verify: 4-bit cache attention, cache append, draft acceptance.

A verify step of a hybrid model runs its drafted nodes through the full-attention layers as well as the Gated
DeltaNet ones, decides which of them are accepted, and commits the accepted rows.  Three operators do that:

- ``attention``: the nodes of each request's tree (or one token a request) attend to the committed tokens, whose
  keys and values are held in 4 bits in pages of 64 tokens, and to their own ancestors among the drafted nodes;
- ``append``: rows of new keys and values (a prompt's, or an accepted path's) are quantised into the pages;
- ``accept``: drafted tokens are checked against the target's logits from given random numbers.

``run`` computes each in its plain form with torch (32 bits) or, where ``own`` is set, through the library.
The page format is the one include/gdn_tree.h documents (gdn_kv4_cache).
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
PAGE = 64
GROUP = 32


# ---- cases ------------------------------------------------------------------------------------------------------

def listed():
    """Heads 24/4 of size 256 are the attention layers of the hybrid models whose GDN layers the library verifies;
    22-node trees of width 4, 64-node trees and chains and 32-request batches are its own workloads."""
    return [
        # one token of one request: plain decoding between drafted steps, where latency counts
        dict(name="attention_one_token", kind="attention", B=1, n=1, Hq=24, Hkv=4, D=256, length=4096, dtype="bf16"),
        # one token of each of 32 requests over long ragged caches: bound by the cache's bytes
        dict(name="attention_tokens_batched", kind="attention", B=32, n=1, Hq=24, Hkv=4, D=256, length=32768,
             dtype="bf16"),
        # the batched workload's trees: 32 requests, up to 22 nodes each
        dict(name="attention_tree22_batched", kind="attention", B=32, n=22, Hq=24, Hkv=4, D=256, length=8192,
             dtype="bf16"),
        # one 22-node tree over a short cache: the ordinary interactive step
        dict(name="attention_tree22_one", kind="attention", B=1, n=22, Hq=24, Hkv=4, D=256, length=5000, dtype="bf16"),
        # the widest trees over very long contexts, two requests
        dict(name="attention_tree64_long", kind="attention", B=2, n=64, Hq=24, Hkv=4, D=256, length=200001,
             dtype="bf16"),
        # another head layout (4 query heads a kv head, size 128), small trees, ragged lengths that end inside a page
        dict(name="attention_tree8_d128", kind="attention", B=16, n=8, Hq=32, Hkv=8, D=128, length=5001, dtype="bf16"),
        # 32-bit sessions (the library's fp32 configuration), small
        dict(name="attention_tree8_f32", kind="attention", B=4, n=8, Hq=8, Hkv=4, D=64, length=2000, dtype="f32"),
        # commit of the accepted paths of the batched workload in all 16 attention layers of a 64-layer hybrid
        dict(name="append_accepted", kind="append", B=32, layers=16, n=22, Hkv=4, D=256, length=8192, path=True,
             dtype="bf16"),
        # a prompt's rows of one layer
        dict(name="append_prompt", kind="append", B=2, layers=1, n=20001, Hkv=4, D=256, length=100, path=False,
             dtype="bf16"),
        # one request's 22-node tree, sampling from a large vocabulary
        dict(name="accept_tree_one", kind="accept", B=1, n=22, V=131072, draft="point", dtype="bf16", zero_t=0),
        # the batched workload's trees; a quarter of the requests are greedy
        dict(name="accept_tree_batched", kind="accept", B=32, n=22, V=131072, draft="point", dtype="bf16", zero_t=4),
        # sampled chain drafts with their draft probabilities, odd vocabulary (rows at every alignment)
        dict(name="accept_chain_batched", kind="accept", B=64, n=9, V=65537, draft="chain", dtype="f32", zero_t=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case from the same ranges: sizes over their logarithm, odd ones among them; no larger than the listed ones."""
    kind = rng.choice(["attention", "attention", "append", "accept"])
    if kind == "attention":
        Hq, Hkv, D = rng.choice([(24, 4, 256), (24, 4, 256), (32, 8, 128), (16, 16, 128), (8, 1, 256), (8, 4, 64)])
        dtype = "f32" if rng.random() < 0.15 else "bf16"
        n = 1 if rng.random() < 0.3 else rng.choice([2, 5, 8, 13, 22, 32, 47, 64])
        B = _log(rng, 1, 48)
        length = _log(rng, 300, 200001)
        most = 3e8 if dtype == "f32" else 2e11     # multiply-adds of the scores: rows x tokens x D
        length = max(1, min(length, int(most / (B * n * Hq * D)), int(1e9 / (B * Hkv * D))))
        return dict(kind=kind, B=B, n=n, Hq=Hq, Hkv=Hkv, D=D, length=length, dtype=dtype)
    if kind == "append":
        Hkv, D = rng.choice([(4, 256), (8, 128), (1, 256), (4, 64)])
        dtype = "f32" if rng.random() < 0.15 else "bf16"
        if rng.random() < 0.5:
            return dict(kind=kind, B=_log(rng, 1, 48), layers=rng.choice([1, 3, 16]), n=rng.choice([1, 9, 22, 64]),
                        Hkv=Hkv, D=D, length=_log(rng, 50, 5000), path=True, dtype=dtype)
        return dict(kind=kind, B=_log(rng, 1, 4), layers=rng.choice([1, 2]), n=_log(rng, 65, 10000), Hkv=Hkv, D=D,
                    length=_log(rng, 1, 300), path=False, dtype=dtype)
    draft = rng.choice(["point", "point", "chain"])
    n = rng.choice([3, 9, 16]) if draft == "chain" else rng.choice([1, 8, 22, 37, 64])
    V = rng.choice([4099, 32000, 50001, 65537, 131072, 150001])
    B = max(1, min(_log(rng, 1, 128), int((4.0e7 if draft == "chain" else 1.0e8) / (n * V))))
    return dict(kind="accept", B=B, n=n, V=V, draft=draft, dtype=rng.choice(["bf16", "bf16", "f32"]),
                zero_t=rng.choice([0, 0, 3, 1]))


def _counts(n, B):
    """Ragged sizes n/2 .. n, evenly spaced over the requests (prepare shuffles them)."""
    return [max(1, n - (n // 2) * i // B) for i in range(B)]


def _size(case):
    return 4 if case["dtype"] == "f32" else 2


# Rows of logits that a walk visits on these inputs, on average (a walk ends at the first node without an accepted
# child): measured on the plain form's outputs, limited by the trees' depth.
VISITED = {"point": 2.5, "chain": 4.0}


def work(case):
    B, n = case["B"], case["n"]
    nodes = sum(_counts(n, B))
    if case["kind"] == "attention":
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        lens = _counts(case["length"], B)
        # the pairing of lengths with node counts is shuffled: the product's mean
        pairs = sum(lens) * nodes / B
        return {"bytes": sum(lens) * Hkv * D * 9 / 8 + nodes * (2 * Hq + 2 * Hkv) * D * _size(case),
                "flops": 4.0 * D * Hq * pairs}
    if case["kind"] == "append":
        rows = (0.5 * nodes if case["path"] else nodes) * case["layers"]
        return {"bytes": rows * case["Hkv"] * D_of(case) * (2 * _size(case) + 9 / 8 + 8), "flops": 0}
    V = case["V"]
    visited = min(VISITED[case["draft"]], n)
    extra = V * 4 * (2 if case["draft"] == "chain" else 1)
    return {"bytes": B * (visited * V * _size(case) + extra), "flops": 3.0 * B * visited * V}


def D_of(case):
    return case["D"]


# ---- inputs -----------------------------------------------------------------------------------------------------

def _trees(case, rng):
    """Parents of every request's tree (ragged): a greedy chain, then nodes hung on earlier ones, at most four
    children each; numbered so that a parent comes before its children."""
    B, n = case["B"], case["n"]
    counts = _counts(n, B)
    rng.shuffle(counts)
    parents = np.full((B, n), -1, dtype=np.int32)
    for b, k in enumerate(counts):
        depth = max(1, min(k, 10 if case.get("draft") != "chain" else k))
        kids = np.zeros(k, dtype=np.int64)
        for i in range(1, k):
            p = i - 1 if i < depth else int(rng.integers(0, min(i, 2 * depth)))
            while kids[p] >= 4:
                p = (p + 1) % i
            parents[b, i] = p
            kids[p] += 1
    return parents, np.asarray(counts, dtype=np.int32)


def _pair_order():
    """Nibble of each of a word's eight elements: the even ones in the low half-word, the odd ones in the high one."""
    return [(e >> 1) + 4 * (e & 1) for e in range(8)]


def _chunk(D):
    """Place of a token's 16-byte chunk c (32 channels) among its D/32 key chunks."""
    t = np.arange(PAGE)[:, None]
    c = np.arange(D // 32)[None, :]
    x = {256: ((t & 1) << 2) | ((t >> 1) & 3), 128: (t >> 1) & 3, 64: (t >> 2) & 1}[D]
    return torch.from_numpy(c ^ x).to(DEV)


def _quantise(x):
    """x [..., D] -> codes 0..15 (uint8, same shape) and scales f16 [..., D/32]."""
    g = x.float().unflatten(-1, (-1, GROUP))
    a = g.abs()
    big = a.amax(-1, keepdim=True)
    first = torch.where(a == big, torch.arange(GROUP, device=x.device), GROUP).amin(-1, keepdim=True)
    m = g.gather(-1, first.clamp(max=GROUP - 1))
    d = (m * -0.125).bfloat16().float().clamp(-2720.0, 2720.0).half().float()
    d = torch.where(torch.isfinite(g).all(-1, keepdim=True), d, torch.full_like(d, float("nan")))
    r = torch.where(d != 0, g / d, torch.zeros_like(g))
    r = torch.nan_to_num(r.round(), nan=0.0).clamp(-8, 7)
    return (r + 8).to(torch.uint8).flatten(-2), d.half().squeeze(-1)


def _pack_words(e):
    """e [..., 8] codes -> [..., 4] bytes of one word."""
    o = e[..., [0, 2, 4, 6, 1, 3, 5, 7]]         # nibble order
    return o[..., 0::2] | (o[..., 1::2] << 4)


def _pack_pages(k, v, D):
    """k, v [pages, 64, Hkv, D] 32-bit values -> blocks [pages, Hkv, 72 D] bytes."""
    P, H = k.shape[0], k.shape[2]
    kc, kd = _quantise(k.transpose(1, 2))          # [P, H, 64, D]
    vc, vd = _quantise(v.transpose(1, 2))
    kb = _pack_words(kc.view(P, H, PAGE, D // 32, 4, 8)).reshape(P, H, PAGE, D // 32, 16)
    idx = _chunk(D)[None, None, :, :, None].expand(P, H, -1, -1, 16)
    kb = torch.empty_like(kb).scatter_(3, idx, kb)
    w = vc.view(P, H, 2, 4, 8, D // 4, 4)           # token = ((kb, o), e), channel = (cq, c)
    w = _pack_words(w.permute(0, 1, 2, 5, 3, 6, 4))   # [P, H, kb, cq, o, c, 4 bytes]
    return torch.cat([kb.reshape(P, H, -1), kd.contiguous().view(torch.uint8).reshape(P, H, -1),
                      w.reshape(P, H, -1), vd.transpose(2, 3).contiguous().view(torch.uint8).reshape(P, H, -1)], -1)


def _gen(seed, salt):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 1000003 + salt)


def _rand_rows(gen, *shape):
    """Key or value rows as projections give them: normal, with a few channels several times the others."""
    x = torch.randn(*shape, generator=gen, device=DEV)
    c = torch.randint(0, shape[-1], (max(1, shape[-1] // 64),), generator=gen, device=DEV)
    x[..., c] *= 4.0
    return x


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _prepare_cache(case, seed, lens, layers, pages_max, fill):
    """Pool, shuffled page table and lengths; with fill, the pages of the committed tokens hold quantised rows."""
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    gen = _gen(seed, 1)
    n_pages = B * pages_max + 3
    order = torch.randperm(n_pages, generator=gen, device=DEV)[:B * pages_max]
    table = order.view(B, pages_max).to(torch.int32)
    pool = torch.zeros(layers, n_pages, Hkv, 72 * D, dtype=torch.uint8, device=DEV)
    if fill:
        step = max(1, (1 << 25) // (PAGE * Hkv * D))
        for at in range(0, n_pages, step):
            k = min(step, n_pages - at)
            pool[0, at:at + k] = _pack_pages(_rand_rows(gen, k, PAGE, Hkv, D), _rand_rows(gen, k, PAGE, Hkv, D), D)
    return pool, table, torch.tensor(lens, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    rng = np.random.default_rng([int(seed), 77])
    s = {"case": case}
    B, n = case["B"], case["n"]
    if case["kind"] == "attention":
        Hq, Hkv, D, dt = case["Hq"], case["Hkv"], case["D"], _dtype(case)
        lens = _counts(case["length"], B)
        rng.shuffle(lens)
        s["max_len"] = max(lens)
        s["pool"], s["table"], s["len"] = _prepare_cache(case, seed, lens, 1, -(-max(lens) // PAGE), True)
        parents, counts = _trees(case, rng)
        gen = _gen(seed, 2)
        s["q"] = (2.0 * torch.randn(B, 1, n, Hq, D, generator=gen, device=DEV)).to(dt)
        s["k"] = _rand_rows(gen, B, 1, n, Hkv, D).to(dt)
        s["v"] = _rand_rows(gen, B, 1, n, Hkv, D).to(dt)
        s["out"] = torch.zeros(B, 1, n, Hq, D, dtype=dt, device=DEV)
        s["scale"] = D ** -0.5
        _with_trees(s, parents, counts)
    elif case["kind"] == "append":
        Hkv, D, L, dt = case["Hkv"], case["D"], case["layers"], _dtype(case)
        lens = _counts(case["length"], B)
        rng.shuffle(lens)
        pages_max = -(-(max(lens) + n) // PAGE)
        s["pool"], s["table"], s["len"] = _prepare_cache(case, seed, lens, L, pages_max, False)
        s["len0"] = s["len"].clone()
        gen = _gen(seed, 2)
        s["k"] = _rand_rows(gen, B, L, n, Hkv, D).to(dt)
        s["v"] = _rand_rows(gen, B, L, n, Hkv, D).to(dt)
        counts = _counts(n, B)
        rng.shuffle(counts)
        path = np.zeros((B, n), dtype=np.int32)
        if case["path"]:       # a root path: node 0, then increasing indices
            counts = [max(1, c // 2) for c in counts]
            for b, c in enumerate(counts):
                path[b, 1:c] = np.sort(rng.choice(np.arange(1, n), size=c - 1, replace=False)) if c > 1 else 0
            s["path"] = torch.from_numpy(path).to(DEV)
        else:
            s["path"] = None
        s["count"] = torch.tensor(counts, dtype=torch.int32, device=DEV)
        s["most"] = max(counts)
    else:
        V, dt = case["V"], _dtype(case)
        gen = _gen(seed, 2)
        parents, counts = _trees(case, rng)
        z = 2.0 * torch.randn(B, n, V, generator=gen, device=DEV)
        # a few likely tokens carry about half the mass, as in a language model's rows
        likely = torch.randint(0, V, (B, n, 4), generator=gen, device=DEV)
        base = math.log(V) + 2.0
        z.scatter_(2, likely, base + 0.7 - 1.2 * torch.arange(4, device=DEV).expand(B, n, 4))
        par = torch.from_numpy(np.maximum(parents, 0)).to(DEV).long()
        if case["draft"] == "chain":
            # the draft's distribution: the target's, blurred; each node's token drawn from its parent's row
            q = (z + 0.5 * torch.randn(B, n, V, generator=gen, device=DEV)).softmax(-1)
            u = torch.rand(B, n, V, generator=gen, device=DEV).clamp_(1e-9, 1 - 1e-7)
            drawn = (q.clamp_min(1e-30).log() - torch.log(-torch.log(u))).argmax(-1)
            tokens = drawn.gather(1, par)
            s["q_probs"] = q.to(torch.float32)
        else:
            rank = torch.from_numpy(_ranks(parents)).to(DEV).long()
            tokens = likely.gather(1, par[..., None].expand(-1, -1, 4)).gather(2, rank[..., None]).squeeze(2)
            other = torch.rand(B, n, generator=gen, device=DEV) < 0.1      # a draft that misses
            tokens = torch.where(other, torch.randint(0, V, (B, n), generator=gen, device=DEV), tokens)
            s["q_probs"] = None
        s["z"] = z.to(dt)
        s["tokens"] = tokens.to(torch.int32).contiguous()
        s["u"] = torch.rand(B, n, generator=gen, device=DEV)
        e = torch.rand(B, V, generator=gen, device=DEV).clamp_(1e-9, 1 - 1e-7)
        s["gumbel"] = -torch.log(-torch.log(e))
        t = 0.7 + 0.6 * torch.rand(B, generator=gen, device=DEV)
        if case["draft"] == "chain":
            t = torch.ones_like(t)          # the draft was sampled at the target's temperature
        if case["zero_t"]:
            t[::case["zero_t"]] = 0.0
        s["temperature"] = t
        _with_trees(s, parents, counts)
    if own:
        _handles(s)
    return s


def _ranks(parents):
    """Position of each node among its siblings."""
    r = np.zeros_like(parents)
    for b in range(parents.shape[0]):
        seen = {}
        for i, p in enumerate(parents[b]):
            r[b, i] = seen.get(p, 0) if p >= 0 else 0
            seen[p] = r[b, i] + 1
    return np.minimum(r, 3)


def _with_trees(s, parents, counts):
    s["parents"], s["counts"] = parents, counts
    s["par"] = torch.from_numpy(parents).to(DEV).long()
    s["n"] = torch.from_numpy(counts).to(DEV).long()


def _handles(s):
    """The library's handles over the same buffers: what a user's program keeps between steps."""
    from gated_deltanet_tree_gb300 import runtime as R
    case = s["case"]
    if case["kind"] in ("attention", "append"):
        dims = R.make_attn_dims(case.get("Hq", case["Hkv"]), case["Hkv"], case["D"],
                                dtype=_dtype(case), scale=s.get("scale", 1.0))
        s["cache"] = R.KV4Cache(dims, s["pool"], s["table"], s["len"])
    else:
        s["acceptor"] = R.TreeAcceptor(case["B"], case["n"], case["V"], DEV)
    if case["kind"] == "accept" or (case["kind"] == "attention" and case["n"] > 1):
        trees = [s["parents"][b, :c] for b, c in enumerate(s["counts"])]
        s["sched"] = R.DeviceSchedule(trees, case["n"], DEV)


# ---- one pass ---------------------------------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return {"attention": _plain_attention, "append": _plain_append, "accept": _plain_accept}[s["case"]["kind"]](s)


def _run_own(s):
    kind = s["case"]["kind"]
    if kind == "attention":
        s["cache"].attention(s["q"], s["k"], s["v"], s["out"], sched=s.get("sched"), max_len=s["max_len"])
        return s["out"]
    if kind == "append":
        s["len"].copy_(s["len0"])
        s["cache"].append(s["k"], s["v"], s["count"], path=s["path"])
        k, v = s["cache"].read(s["len0"], s["most"])
        return {"k": k, "v": v, "len": s["len"]}
    path, length, token = s["acceptor"].accept(s["sched"], s["z"], s["tokens"], s["u"], s["gumbel"],
                                               s["temperature"], draft_probs=s["q_probs"])
    return {"path": path, "len": length, "next": token}


def _unpack(s):
    """The committed rows of the cache, 32 bits: k, v [B, Hkv, S, D], S = the table's tokens."""
    D, Hkv = s["case"]["D"], s["case"]["Hkv"]
    B, P = s["table"].shape
    blocks = s["pool"][0][s["table"].long()]          # [B, P, Hkv, 72 D]
    nk, ns = 32 * D, 4 * D
    kb = blocks[..., :nk].reshape(B, P, Hkv, PAGE, D // 32, 16)
    kb = kb.gather(4, _chunk(D)[None, None, None, :, :, None].expand(B, P, Hkv, -1, -1, 16))
    kd = blocks[..., nk:nk + ns].contiguous().view(torch.float16).reshape(B, P, Hkv, PAGE, D // 32, 1)
    vb = blocks[..., nk + ns:2 * nk + ns].reshape(B, P, Hkv, 2, D // 4, 4, 4, 4)
    vd = blocks[..., 2 * nk + ns:].contiguous().view(torch.float16).reshape(B, P, Hkv, D // 32, PAGE)
    order = _pair_order()

    def values(b):        # [..., 4] bytes -> [..., 8] elements
        nib = torch.stack([b & 15, b >> 4], -1).flatten(-2)
        return nib[..., order].float() - 8.0

    k = values(kb.unflatten(-1, (4, 4))).flatten(-2) * kd.float()           # [B, P, Hkv, 64, D/32, 32]
    k = k.flatten(-2).permute(0, 2, 1, 3, 4).reshape(B, Hkv, P * PAGE, D)
    v = values(vb)                                                          # [B, P, Hkv, kb, cq, o, c, 8]
    v = v.permute(0, 1, 2, 3, 5, 7, 4, 6).reshape(B, P, Hkv, PAGE, D // 32, 32)
    v = v * vd.float().transpose(3, 4)[..., None]
    v = v.reshape(B, P, Hkv, PAGE, D).transpose(1, 2).reshape(B, Hkv, P * PAGE, D)
    return k, v


def _ancestors(par, dtype=torch.float32):
    """[B, n, n]: 1 where column j is an ancestor of row i or i itself."""
    B, n = par.shape
    step = torch.nn.functional.one_hot(par.clamp_min(0), n).to(dtype) * (par >= 0)[..., None]
    near = (step + torch.eye(n, dtype=dtype, device=par.device)).clamp_max(1)
    for _ in range(6):       # paths of up to 64 nodes
        near = (near @ near).clamp_max(1)
    return near > 0


def _plain_attention(s):
    case = s["case"]
    B, n, Hq, Hkv, D = case["B"], case["n"], case["Hq"], case["Hkv"], case["D"]
    G = Hq // Hkv
    k, v = _unpack(s)
    S = k.shape[2]
    q = s["q"][:, 0].float().reshape(B, n, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D)
    gone = torch.arange(S, device=DEV) >= s["len"][:, None]
    v = v.masked_fill(gone[:, None, :, None], 0.0)
    a = (q @ k.transpose(-1, -2)) * s["scale"]
    a.masked_fill_(gone[:, None, None, :], -math.inf)
    kn = s["k"][:, 0].float().transpose(1, 2)         # [B, Hkv, n, D]
    vn = s["v"][:, 0].float().transpose(1, 2)
    b = (q @ kn.transpose(-1, -2)) * s["scale"]
    see = _ancestors(s["par"]).repeat_interleave(G, dim=1)
    b.masked_fill_(~see[:, None], -math.inf)
    m = torch.maximum(a.amax(-1, keepdim=True), b.amax(-1, keepdim=True))
    a = a.sub_(m).exp_()
    b = b.sub_(m).exp_()
    o = (a @ v + b @ vn) / (a.sum(-1, keepdim=True) + b.sum(-1, keepdim=True))
    o = o.reshape(B, Hkv, n, G, D).permute(0, 2, 1, 3, 4).reshape(B, 1, n, Hq, D)
    real = torch.arange(n, device=DEV) < s["n"][:, None]
    return o.masked_fill(~real[:, None, :, None, None], 0.0).to(s["q"].dtype)


def _plain_append(s):
    case = s["case"]
    B, T = case["B"], s["most"]
    at = torch.arange(T, device=DEV).expand(B, T) if s["path"] is None else s["path"][:, :T].long()
    real = torch.arange(T, device=DEV) < s["count"][:, None]
    at = torch.where(real, at, 0)
    got = []
    for x in (s["k"], s["v"]):
        rows = x.gather(2, at[:, None, :, None, None].expand(-1, x.shape[1], -1, *x.shape[3:]))
        c, d = _quantise(rows)
        y = (c.float() - 8.0).unflatten(-1, (-1, GROUP)) * d.float()[..., None]
        got.append(y.flatten(-2).masked_fill(~real[:, None, :, None, None], 0.0))
    return {"k": got[0], "v": got[1], "len": s["len0"] + s["count"]}


def _first_max(x):
    """Lowest index of the largest value along the last axis."""
    at = torch.arange(x.shape[-1], device=x.device)
    return torch.where(x == x.amax(-1, keepdim=True), at, x.shape[-1]).amin(-1)


def _plain_accept(s):
    z, tok, par, u, T = s["z"].float(), s["tokens"].long(), s["par"], s["u"], s["temperature"]
    B, n, V = z.shape
    node = torch.arange(n, device=DEV)
    real = node < s["n"][:, None]
    up = par.clamp_min(0)
    cold = (T == 0)[:, None]
    zt = z / torch.where(T == 0, torch.ones_like(T), T)[:, None, None]
    m = zt.amax(-1, keepdim=True)
    total = (zt - m).exp().sum(-1, keepdim=True)
    top = _first_max(z)
    # each node's token under its parent's row
    row = zt.flatten(1)
    pt = (row.gather(1, up * V + tok) - m.squeeze(-1).gather(1, up)).exp() / total.squeeze(-1).gather(1, up)
    kin = (par[:, :, None] == par[:, None, :]) & (node[:, None] > node)     # [i, j]: j an earlier sibling of i
    if s["q_probs"] is None:
        again = (kin & (tok[:, :, None] == tok[:, None, :])).any(-1)
        w = torch.where(again, torch.zeros_like(pt), pt)
        left = 1.0 - (kin * w[:, None, :]).sum(-1)
        yes = u * left < w
    else:
        qt = s["q_probs"].flatten(1).gather(1, up * V + tok)
        yes = u * qt < pt
    yes = torch.where(cold, tok == top.gather(1, up), yes)
    yes = yes & ~(kin & yes[:, None, :]).any(-1) & real
    yes[:, 0] = True
    see = _ancestors(par)
    on = ~(see & ~yes[:, None, :]).any(-1) & real
    length = on.sum(-1)
    path = torch.where(on, node, n).sort(-1).values
    path = torch.where(path < n, path, -1)
    stop = torch.where(on, node, -1).amax(-1)
    # the next token: from what is left of the stop node's row
    here = torch.arange(B, device=DEV)
    mine = (par == stop[:, None]) & real
    zs = zt[here, stop]
    if s["q_probs"] is None:
        out = torch.zeros(B, V + 1, dtype=torch.bool, device=DEV)
        out.scatter_(1, torch.where(mine, tok, V), True)
        score = zs.masked_fill(out[:, :V], -math.inf) + s["gumbel"]
    else:
        p = (zs - m[here, stop]).exp() / total[here, stop]
        rest = (p - s["q_probs"][here, stop] * mine.any(-1, keepdim=True)).clamp_min(0.0)
        rest = torch.where((rest > 0).any(-1, keepdim=True), rest, p)
        score = rest.log() + s["gumbel"]
    token = torch.where(T == 0, top[here, stop], _first_max(score))
    return {"path": path.int(), "len": length.int(), "next": token.int()}


# ---- the definition in 64 bits ----------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "attention":
        B, n, Hq, Hkv, D = case["B"], case["n"], case["Hq"], case["Hkv"], case["D"]
        if work(case)["flops"] > 1.2e13:
            return None
        G = Hq // Hkv
        out = torch.zeros(B, 1, n, Hq, D, dtype=torch.float64, device=DEV)
        for b in range(B):
            L = int(s["len"][b])
            k, v = _rows64(s, b, L)                                          # [L, Hkv, D]
            for h in range(Hkv):
                q = s["q"][b, 0, :, h * G:(h + 1) * G].double()              # [n, G, D]
                kn, vn = s["k"][b, 0, :, h].double(), s["v"][b, 0, :, h].double()
                a = torch.einsum("ngd,td->ngt", q, k[:, h])
                for i in range(int(s["counts"][b])):
                    line, j = [], i
                    while j >= 0:
                        line.append(j)
                        j = int(s["parents"][b, j])
                    w = torch.cat([a[i], q[i] @ kn[line].T], -1) * s["scale"]
                    w = torch.softmax(w, -1)
                    out[b, 0, i, h * G:(h + 1) * G] = w[:, :L] @ v[:, h] + w[:, L:] @ vn[line]
        return out
    if case["kind"] == "append":
        T = s["most"]
        if s["k"].numel() > 1 << 28:
            return None
        got = []
        for x in (s["k"], s["v"]):
            y = torch.zeros(case["B"], case["layers"], T, case["Hkv"], case["D"], dtype=torch.float64, device=DEV)
            for b in range(case["B"]):
                c = int(s["count"][b])
                at = slice(0, c) if s["path"] is None else s["path"][b, :c].long()
                g = x[b][:, at].double().unflatten(-1, (-1, GROUP))
                m = g.gather(-1, g.abs().argmax(-1, keepdim=True))
                low = -g.abs().amax(-1, keepdim=True)
                # the first of the largest magnitudes decides the sign
                has_lo, has_hi = (g == low), (g == -low)
                at_lo = torch.where(has_lo, torch.arange(GROUP, device=DEV), GROUP).amin(-1, keepdim=True)
                at_hi = torch.where(has_hi, torch.arange(GROUP, device=DEV), GROUP).amin(-1, keepdim=True)
                m = torch.where(at_lo < at_hi, low, -low)
                d = (m / -8.0).to(torch.bfloat16).double().clamp(-2720.0, 2720.0).to(torch.float16).double()
                t = torch.where(d == 0, torch.zeros_like(g), torch.round(g / d).clamp(-8, 7))
                y[b, :, :c] = (t * d).flatten(-2)
            got.append(y)
        return {"k": got[0], "v": got[1], "len": None}
    # whole numbers: the rule, request by request
    B, n, V = case["B"], case["n"], case["V"]
    path = torch.full((B, n), -1, dtype=torch.int32)
    length = torch.zeros(B, dtype=torch.int32)
    token = torch.zeros(B, dtype=torch.int32)
    tokens, u = s["tokens"].cpu().tolist(), s["u"].double().cpu().tolist()
    for b in range(B):
        t = float(s["temperature"][b])
        at, k = 0, 0
        while True:
            path[b, k] = at
            k += 1
            z = s["z"][b, at].double()
            kids = [j for j in range(int(s["counts"][b])) if int(s["parents"][b, j]) == at]
            took = None
            if t == 0:
                best = int(_first_max(z))
                took = next((j for j in kids if tokens[b][j] == best), None)
                pick = best
            else:
                p = torch.softmax(z / t, -1)
                for j in kids:
                    x = tokens[b][j]
                    if s["q_probs"] is None:
                        if u[b][j] * float(p.sum()) < float(p[x]):
                            took = j
                            break
                        p[x] = 0.0
                    else:
                        q = s["q_probs"][b, at].double()
                        if u[b][j] * float(q[x]) < float(p[x]):
                            took = j
                            break
                        r = (p - q).clamp_min(0.0)
                        if float(r.sum()) > 0:
                            p = r / r.sum()
                pick = int(_first_max(p.log() + s["gumbel"][b].double()))
            if took is None:
                break
            at = took
        length[b], token[b] = k, pick
    return {"path": path, "len": length, "next": token}


def _rows64(s, b, L):
    """The first L committed rows of request b in 64 bits, [L, Hkv, D], read word by word as the page format says."""
    D, Hkv = s["case"]["D"], s["case"]["Hkv"]
    pages = -(-L // PAGE)
    raw = s["pool"][0][s["table"][b, :pages].long()].contiguous()            # [P, Hkv, 72 D]
    words = raw.view(torch.int32).long() & 0xFFFFFFFF
    halves = raw.view(torch.float16).double()
    t = torch.arange(L, device=DEV)
    page, r = t // PAGE, t % PAGE
    h = torch.arange(Hkv, device=DEV)
    c = torch.arange(D, device=DEV)
    turn = {256: ((r & 1) << 2) | ((r >> 1) & 3), 128: (r >> 1) & 3, 64: (r >> 2) & 1}[D]
    # keys: word of channel c of token r, scale of group c // 32
    at = r[:, None] * (D // 8) + ((c // 32)[None] ^ turn[:, None]) * 4 + (c % 32)[None] // 8
    bit = 4 * (((c % 8) >> 1) + 4 * (c & 1))
    w = words[page[:, None, None], h[None, :, None], at[:, None, :]]
    d = halves[page[:, None, None], h[None, :, None], (16 * D + r[:, None] * (D // 32) + c[None] // 32)[:, None, :]]
    k = (((w >> bit) & 15) - 8).double() * d
    # values: word of channel c and tokens 8 o .. 8 o + 7
    o = r // 8
    at = 9 * D + (((o // 4)[:, None] * (D // 4) + c[None] // 4) * 4 + (o % 4)[:, None]) * 4 + c[None] % 4
    bit = 4 * (((r % 8) >> 1) + 4 * (r & 1))
    w = words[page[:, None, None], h[None, :, None], at[:, None, :]]
    d = halves[page[:, None, None], h[None, :, None], (34 * D + (c[None] // 32) * PAGE + r[:, None])[:, None, :]]
    v = (((w >> bit[:, None, None]) & 15) - 8).double() * d
    return k, v
