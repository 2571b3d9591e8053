"""Timed cases of what surrounds a tree verify: prompts and single tokens through a GDN layer, the draft's candidates.

Before a request's first tree its prompt goes through the Gated DeltaNet layers; where nothing is drafted, single tokens
do; and the next tree is built from log-probabilities of the draft's best tokens.  Three operators do that:

- ``prefill``: the rows of a ragged batch of prompts through one layer (causal conv, SiLU, normalised q and k, gated
  delta rule): the output of every token, and the state and conv window after the last;
- ``step``: the same for one token of each request;
- ``logprobs``: of rows of logits the log-probability of a given token, the entropy, and the best tokens with theirs.

``run`` computes each in its plain form with torch (32 bits) or, where ``own`` is set, through the library.  The rule is
the one include/gdn_tree.h states.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
CHUNK = 64


# ---- cases ------------------------------------------------------------------------------------------------------

def listed():
    """16 q/k heads and 48 v-heads of size 128 with 4 taps are the GDN layers of the library's own workloads, batches of
    32 and 128 requests theirs too, and so is the head size of 64 or 32 bits in the smaller layers."""
    return [
        # a short question to an idle server: the first answer's latency
        dict(name="prefill_short", kind="prefill", B=1, T=70, Hk=16, Hv=48, dk=128, dv=128, K=4, dtype="bf16"),
        # one long document
        dict(name="prefill_document", kind="prefill", B=1, T=8191, Hk=16, Hv=48, dk=128, dv=128, K=4, dtype="bf16"),
        # a batch of ordinary prompts, ragged
        dict(name="prefill_batched", kind="prefill", B=32, T=500, Hk=16, Hv=48, dk=128, dv=128, K=4, dtype="bf16"),
        # two very long contexts of unequal length
        dict(name="prefill_long", kind="prefill", B=2, T=20001, Hk=16, Hv=48, dk=128, dv=128, K=4, dtype="bf16"),
        # 32-bit sessions with smaller heads
        dict(name="prefill_f32_d64", kind="prefill", B=4, T=1000, Hk=4, Hv=8, dk=64, dv=64, K=4, dtype="f32"),
        # one token of one request: plain decoding, where latency counts
        dict(name="step_one", kind="step", B=1, Hk=16, Hv=48, dk=128, dv=128, K=4, dtype="bf16"),
        # one token of each of the largest workload's requests: bound by the states' bytes
        dict(name="step_batched", kind="step", B=128, Hk=16, Hv=48, dk=128, dv=128, K=4, dtype="bf16"),
        # 32-bit sessions with smaller heads, an odd batch
        dict(name="step_f32_d64", kind="step", B=37, Hk=4, Hv=8, dk=64, dv=64, K=4, dtype="f32"),
        # the draft's rows of one request's tree: ten depths, four candidates each
        dict(name="logprobs_draft_one", kind="logprobs", rows=10, V=131072, top=4, dtype="bf16", pad=0),
        # the batched workload's drafts
        dict(name="logprobs_draft_batched", kind="logprobs", rows=320, V=131072, top=8, dtype="bf16", pad=0),
        # a prompt's tokens scored, with alternatives: 32-bit logits of an odd vocabulary with padding at its end
        dict(name="logprobs_prompt", kind="logprobs", rows=1500, V=65537, top=20, dtype="f32", pad=300),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case from the same ranges: sizes over their logarithm, odd ones among them; no larger than the listed ones."""
    kind = rng.choice(["prefill", "prefill", "step", "logprobs"])
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    if kind == "logprobs":
        V = rng.choice([4099, 32000, 50001, 65537, 131072, 150001])
        rows = max(1, min(_log(rng, 1, 4000), int(9e7 / V)))
        return dict(kind=kind, rows=rows, V=V, top=rng.choice([1, 4, 8, 20, 32]), dtype=dtype,
                    pad=rng.choice([0, 0, 77]))
    Hk, Hv, dk, dv = rng.choice([(16, 48, 128, 128), (16, 48, 128, 128), (16, 32, 128, 128), (4, 4, 32, 32),
                                 (4, 8, 64, 64), (2, 6, 128, 64), (8, 8, 64, 128)])
    c = dict(kind=kind, B=_log(rng, 1, 40), Hk=Hk, Hv=Hv, dk=dk, dv=dv, K=rng.choice([4, 4, 4, 2]), dtype=dtype)
    if kind == "step":
        c["B"] = _log(rng, 1, 128)
        return c
    T = _log(rng, 1, 20001)
    c["T"] = max(1, min(T, int(24000 / c["B"])))
    return c


def _lens(T, B):
    """Ragged lengths T/2 .. T, evenly spaced over the requests (prepare shuffles them)."""
    return [max(1, T - (T // 2) * i // B) for i in range(B)]


def _size(case):
    return 4 if case["dtype"] == "f32" else 2


def work(case):
    size = _size(case)
    if case["kind"] == "logprobs":
        R, V, top = case["rows"], case["V"], case["top"]
        return {"bytes": R * (V * size + 4 + 8 + 8 * top), "flops": 6.0 * R * V}
    Hk, Hv, dk, dv, K, B = (case[x] for x in ("Hk", "Hv", "dk", "dv", "K", "B"))
    C = 2 * Hk * dk + Hv * dv
    tokens = B if case["kind"] == "step" else sum(_lens(case["T"], B))
    kept = 4.0 * (Hv * dk * dv + (K - 1) * C)            # a request's state and window
    return {"bytes": tokens * size * (C + 2 * Hv + Hv * dv) + 2 * B * kept + 4 * C * K,
            "flops": tokens * (6.0 * Hv * dk * dv + 2.0 * C * K)}


# ---- inputs -----------------------------------------------------------------------------------------------------

def _gen(seed, salt):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 1000003 + salt)


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def prepare(case, seed):
    gen, dt = _gen(seed, 5), _dtype(case)
    s = {"case": case}

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    if case["kind"] == "logprobs":
        R, V, top = case["rows"], case["V"], case["top"]
        z = 2.0 * normal(R, V)
        # a few likely tokens carry about half the mass, as in a language model's rows
        likely = torch.randint(0, V - case["pad"], (R, 4), generator=gen, device=DEV)
        z.scatter_(1, likely, math.log(V) + 2.7 - 1.2 * torch.arange(4, device=DEV).expand(R, 4))
        if case["pad"]:
            z[:, V - case["pad"]:] = -math.inf
        s["z"] = z.to(dt)
        other = torch.randint(0, V - case["pad"], (R,), generator=gen, device=DEV)
        known = torch.rand(R, generator=gen, device=DEV) < 0.7
        s["tokens"] = torch.where(known, likely[:, 0], other).to(torch.int32)
    else:
        Hk, Hv, dk, dv, K, B = (case[x] for x in ("Hk", "Hv", "dk", "dv", "K", "B"))
        C = 2 * Hk * dk + Hv * dv
        lens = [1] * B
        if case["kind"] == "prefill":
            lens = _lens(case["T"], B)
            np.random.default_rng([int(seed), 78]).shuffle(lens)
        rows = sum(lens)
        s["lens"], s["q_scale"], s["eps"] = lens, dk ** -0.5, 1e-6
        s["x"] = normal(rows, C).to(dt)
        s["w"] = normal(1, C, K) * K ** -0.5
        s["beta"] = torch.sigmoid(normal(rows, Hv)).to(dt)
        # decay rates of the heads from long memories to short ones
        rate = torch.exp(math.log(0.01) * torch.linspace(1, 0, Hv, device=DEV))
        s["log_g"] = (-rate * torch.nn.functional.softplus(normal(rows, Hv))).to(dt)
        s["state"] = 0.1 * normal(B, 1, Hv, dk, dv)
        s["conv"] = normal(B, 1, K - 1, C)
    if own:
        _handles(s)
    return s


def _handles(s):
    """The library's handles and the buffers that a user's program keeps between steps."""
    from gated_deltanet_tree_gb300 import runtime as R
    case = s["case"]
    if case["kind"] == "logprobs":
        s["scorer"] = R.TokenScorer(case["rows"], case["V"], case["top"], DEV)
        return
    from gated_deltanet_tree_gb300 import _native as N
    code = N.GDN_DTYPE_F32 if case["dtype"] == "f32" else N.GDN_DTYPE_BF16
    dims = R.make_dims(case["Hk"], case["Hv"], case["dk"], case["dv"], case["K"], in_dtype=code,
                       q_scale=s["q_scale"], l2_eps=s["eps"])
    s["runner"] = R.SequenceRunner(dims, case["B"], 1, DEV)
    s["out"] = torch.empty(s["x"].shape[0], case["Hv"], case["dv"], dtype=_dtype(case), device=DEV)
    s["state_out"], s["conv_out"] = torch.empty_like(s["state"]), torch.empty_like(s["conv"])


# ---- one pass ---------------------------------------------------------------------------------------------------

def run(s):
    if own:
        return _run_own(s)
    return _plain_logprobs(s) if s["case"]["kind"] == "logprobs" else _plain_layer(s)


def _run_own(s):
    kind = s["case"]["kind"]
    if kind == "logprobs":
        top, tokens, given, entropy = s["scorer"].score(s["z"], s["tokens"])
        return {"top": top, "top_tokens": tokens, "given": given, "entropy": entropy}
    args = (s["x"], s["w"], s["beta"], s["log_g"], s["state"], s["conv"], s["out"])
    if kind == "prefill":
        s["runner"].prefill(s["lens"], *args, state_out=s["state_out"], conv_out=s["conv_out"])
    else:
        s["runner"].step(*args, state_out=s["state_out"], conv_out=s["conv_out"])
    return {"o": s["out"], "state": s["state_out"], "conv": s["conv_out"]}


def _plain_logprobs(s):
    z = s["z"].float()
    m = z.amax(-1, keepdim=True)
    d = z - m
    e = d.exp()
    total = e.sum(-1, keepdim=True, dtype=torch.float64)
    log_total = total.log()
    order = torch.sort(z, dim=-1, descending=True, stable=True).indices[:, :s["case"]["top"]]
    mean = torch.where(e > 0, e * d, 0.0).sum(-1, dtype=torch.float64) / total.squeeze(-1)
    return {"top": (d.gather(1, order).double() - log_total).float(), "top_tokens": order.int(),
            "given": (d.gather(1, s["tokens"].long()[:, None]).double() - log_total).squeeze(1).float(),
            "entropy": (log_total.squeeze(1) - mean).float()}


def _padded(s):
    """[B, T] index of each request's rows in the packed ones (the last of its rows repeated behind its end), and which
    are real."""
    lens = torch.tensor(s["lens"], device=DEV)
    start = lens.cumsum(0) - lens
    t = torch.arange(int(max(s["lens"])), device=DEV)
    real = t < lens[:, None]
    return start[:, None] + torch.minimum(t, lens[:, None] - 1), real, lens


def _plain_layer(s):
    """The rule in chunks of up to 64 tokens: within a chunk the updates u solve a triangular system."""
    case = s["case"]
    Hk, Hv, dk, dv, K, B = (case[x] for x in ("Hk", "Hv", "dk", "dv", "K", "B"))
    rows, real, lens = _padded(s)
    T = rows.shape[1]
    x = s["x"][rows].float()                                              # [B, T, C]
    past = torch.cat([s["conv"][:, 0], x], 1)
    y = sum(past[:, j:j + T] * s["w"][0, :, j] for j in range(K))         # taps, oldest first
    last = lens[:, None] + torch.arange(K - 1, device=DEV)
    window = past.gather(1, last[..., None].expand(-1, -1, past.shape[2]))[:, None]
    y = y / (1.0 + (-y).exp())
    y = y * real[..., None]
    size = min(CHUNK, T)
    n = -(-T // size)

    def heads(a, H, d):          # [B, T, H d] -> [B, H, n, size, d], zeros behind the end
        a = torch.nn.functional.pad(a, (0, 0, 0, n * size - T))
        return a.view(B, n, size, H, d).permute(0, 3, 1, 2, 4)

    q, k, v = heads(y[..., :Hk * dk], Hk, dk), heads(y[..., Hk * dk:2 * Hk * dk], Hk, dk), heads(y[..., 2 * Hk * dk:], Hv, dv)
    q = q / (q.square().sum(-1, keepdim=True) + s["eps"]).sqrt() * s["q_scale"]
    k = k / (k.square().sum(-1, keepdim=True) + s["eps"]).sqrt()
    beta = heads(s["beta"][rows].float() * real[..., None], Hv, 1)        # [B, Hv, n, size, 1]
    g = heads(s["log_g"][rows].float() * real[..., None], Hv, 1).double()
    c = g.cumsum(3)                                                       # differences of far sums: in 64 bits
    low = torch.ones(size, size, device=DEV).tril()
    share = Hv // Hk
    pair = ((c - c.transpose(3, 4)).clamp(max=0.0).exp().float()) * low   # decay from token j to token i
    gram = (k @ k.transpose(3, 4)).repeat_interleave(share, 1)
    A = beta * gram * pair * low.tril(-1)
    M = torch.diag_embed(torch.ones(B, Hv, n, size, device=DEV))         # (1 + A)^-1, a row at a time
    for i in range(1, size):
        M[..., i, :i] = -(A[..., i:i + 1, :i] @ M[..., :i, :i]).squeeze(-2)
    M = M * beta.transpose(3, 4)
    del A, gram
    N = (q @ k.transpose(3, 4)).repeat_interleave(share, 1) * pair
    del pair
    first, left = c.exp().float(), (c[..., -1:, :] - c).exp().float()     # decay since the chunk's start, to its end
    whole = first[..., -1:, :]
    q, k = q.repeat_interleave(share, 1), k.repeat_interleave(share, 1)
    S = s["state"][:, 0]
    o = torch.empty(B, Hv, n, size, dv, device=DEV)
    for i in range(n):           # the chunks depend on each other through the state
        u = M[:, :, i] @ (v[:, :, i] - first[:, :, i] * (k[:, :, i] @ S))
        o[:, :, i] = first[:, :, i] * (q[:, :, i] @ S) + N[:, :, i] @ u
        S = whole[:, :, i] * S + k[:, :, i].transpose(2, 3) @ (left[:, :, i] * u)
    o = o.permute(0, 2, 3, 1, 4).reshape(B, n * size, Hv, dv)[:, :T]
    return {"o": o[real].to(s["x"].dtype), "state": S[:, None], "conv": window}


# ---- the definition in 64 bits ----------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["kind"] == "logprobs":
        z = s["z"].cpu().numpy() if case["dtype"] == "f32" else s["z"].float().cpu().numpy()
        R, top = case["rows"], case["top"]
        best = np.empty((R, top))
        tokens = np.empty((R, top), dtype=np.int32)
        given, entropy = np.empty(R), np.empty(R)
        for r in range(R):
            row = z[r].astype(np.float64)
            logp = row - row.max()
            logp -= math.log(np.exp(logp).sum())
            order = np.argsort(-row, kind="stable")[:top]
            best[r], tokens[r] = logp[order], order
            given[r] = logp[int(s["tokens"][r])]
            there = np.isfinite(logp)
            entropy[r] = -(np.exp(logp[there]) * logp[there]).sum()
        return {"top": best, "top_tokens": tokens, "given": given, "entropy": entropy}
    # the rule token by token; requests that have ended keep their state
    Hk, Hv, dk, dv, K, B = (case[x] for x in ("Hk", "Hv", "dk", "dv", "K", "B"))
    lens = np.asarray(s["lens"])
    start = np.cumsum(lens) - lens
    order = np.argsort(-lens, kind="stable")                              # longest first: the running ones are a prefix
    S = s["state"][order, 0].double()
    W = s["conv"][order, 0].double()
    w = s["w"][0].double()
    o = torch.empty(s["x"].shape[0], Hv, dv, dtype=torch.float64, device=DEV)
    begin = torch.from_numpy(start[order]).to(DEV)
    running = (lens[order][None, :] > np.arange(lens.max())[:, None]).sum(1).tolist()
    step = 2048
    for t0 in range(0, int(lens.max()), step):
        # y of up to 2048 tokens of the requests that still run
        b0, m = running[t0], min(step, int(lens.max()) - t0)
        at = begin[:b0, None] + torch.arange(t0, t0 + m, device=DEV)
        at = at.clamp(max=s["x"].shape[0] - 1)
        x = torch.cat([W[:b0], s["x"][at].double()], 1)
        y = torch.stack([x[:, j:j + m] * w[:, j] for j in range(K)]).sum(0)
        y = y * torch.sigmoid(y)
        q = y[..., :Hk * dk].reshape(b0, m, Hk, dk)
        k = y[..., Hk * dk:2 * Hk * dk].reshape(b0, m, Hk, dk)
        v = y[..., 2 * Hk * dk:].reshape(b0, m, Hv, dv)
        q = q * s["q_scale"] * torch.rsqrt((q * q).sum(-1, keepdim=True) + s["eps"])
        k = k * torch.rsqrt((k * k).sum(-1, keepdim=True) + s["eps"])
        q, k = (a.repeat_interleave(Hv // Hk, 2) for a in (q, k))
        beta, g = s["beta"][at].double()[..., None], s["log_g"][at].double().exp()[..., None]
        for i in range(m):
            b = running[t0 + i]
            kt = k[:b, i, :, None]                                        # [b, Hv, 1, dk]
            T = S[:b] * g[:b, i, :, None]
            u = beta[:b, i] * (v[:b, i] - (kt @ T).squeeze(-2))
            torch.add(T, kt.transpose(2, 3) * u[..., None, :], out=S[:b])
            o[at[:b, i]] = (q[:b, i, :, None] @ S[:b]).squeeze(-2)
        # each request's last K - 1 rows
        for j in range(b0):
            e = min(int(lens[order][j]) - t0, m)
            W[j] = x[j, e:e + K - 1].clone()
    back = torch.from_numpy(np.argsort(order)).to(DEV)
    return {"o": o, "state": S[back][:, None], "conv": W[back][:, None]}
