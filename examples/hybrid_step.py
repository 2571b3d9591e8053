"""Speculative steps of a small hybrid stack: GDN layers, full-attention layers over a 4-bit cache, acceptance.

Prompts go through the GDN layers (gdn_prefill) and into the attention layers' cache.  Each step drafts a tree per request
from the log-probabilities of a draft's best tokens (gdn_top_logprobs, gdn_ddtree_build), verifies it through the GDN
layers (gdn_tree_verify), lets its nodes attend to the 4-bit cache (gdn_kv4_attention), decides on the device which nodes
are accepted (gdn_tree_accept) and commits that path in both kinds of layers (gdn_commit_fold, gdn_kv4_append).  From the
drafted trees on, nothing returns to the host within a step.  After gdn_finish single tokens follow (gdn_step).

There are no weights here: projections are fixed random matrices and the target's logits a random projection of the
layers' outputs, so the numbers mean nothing -- the calls, their order and their buffers are a model's.

    python examples/hybrid_step.py
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from gated_deltanet_tree_gb300 import _native as N  # noqa: E402
from gated_deltanet_tree_gb300.runtime import (DeviceSchedule, KV4Cache, SequenceRunner, TokenScorer,  # noqa: E402
                                               TreeAcceptor, TreeVerifier, channels, make_attn_dims, make_dims)

DEPTH, TOP_K = 10, 4            # of the drafts


class HybridStack:
    """GDN layers and attention layers of one small model, with the state a batch of requests keeps."""

    def __init__(self, B=4, n_max=22, V=4096, gdn_layers=3, attn_layers=1, Hk=2, Hv=6, Hq=6, Hkv=1, D=256, width=512,
                 pages_max=8, seed=0, device="cuda"):
        self.B, self.n_max, self.V, self.device = B, n_max, V, torch.device(device)
        gen = torch.Generator(device=device).manual_seed(seed)

        def rnd(*shape, scale=1.0):
            return scale * torch.randn(*shape, generator=gen, device=device)

        self.gdn = make_dims(Hk, Hv, 128, 128, 4)
        self.gdn_layers, self.attn_layers, self.width = gdn_layers, attn_layers, width
        C = channels(self.gdn)
        self.verifier = TreeVerifier(self.gdn, B, gdn_layers, n_max, device)
        self.runner = SequenceRunner(self.gdn, B, gdn_layers, device, verifier=self.verifier)
        self.scorer = TokenScorer(B * DEPTH, V, TOP_K, device)
        self.state = rnd(B, gdn_layers, Hv, 128, 128, scale=0.1)
        self.conv_state = torch.zeros(B, gdn_layers, 3, C, device=device)
        self.conv_w = rnd(gdn_layers, C, 4, scale=0.5)
        self.cache = KV4Cache.empty(make_attn_dims(Hq, Hkv, D), B, attn_layers, pages_max, device)
        self.acceptor = TreeAcceptor(B, n_max, V, device)
        self.heads = (Hq, Hkv, D)
        # stand-ins for the model's matrices
        self.embed = rnd(V, width)
        self.w_gdn = rnd(width, C + 2 * Hv, scale=width ** -0.5)
        self.w_qkv = rnd(width, (Hq + 2 * Hkv) * D, scale=width ** -0.5)
        self.w_logit = rnd(Hv * 128 + Hq * D, V, scale=0.05)
        self.w_draft = rnd(DEPTH, width, V, scale=2 * width ** -0.5)     # a draft that looks at the last token only
        self.out_o = torch.zeros(B, gdn_layers, n_max, Hv, 128, device=device)
        self.out_a = torch.zeros(B, attn_layers, n_max, Hq, D, dtype=torch.bfloat16, device=device)
        self.last = torch.zeros(B, dtype=torch.long, device=device)      # each request's last token, its tree's root
        self.gen = gen

    def gdn_inputs(self, x: torch.Tensor):
        """The GDN layers' raw rows, beta and log gates of rows x [..., width]."""
        y = x @ self.w_gdn
        C, Hv = channels(self.gdn), self.gdn.Hv
        log_g = -torch.nn.functional.softplus(y[..., C + Hv:])
        return tuple(t.bfloat16().contiguous() for t in (y[..., :C], torch.sigmoid(y[..., C:C + Hv]), log_g))

    def prompt(self, tokens: torch.Tensor, count: torch.Tensor):
        """A prompt [B, n] (its first count[b] tokens) through the GDN layers and into the attention layers' cache."""
        Hq, Hkv, D = self.heads
        lens = count.tolist()
        rows = torch.cat([tokens[b, :n] for b, n in enumerate(lens)])
        raw, beta, log_g = self.gdn_inputs(self.embed[rows])
        out = torch.empty(len(rows), self.gdn.Hv, 128, dtype=torch.bfloat16, device=self.device)
        for layer in range(self.gdn_layers):                             # (a model's layers would each have their own rows)
            self.runner.prefill(lens, raw, self.conv_w, beta, log_g, self.state, self.conv_state, out, layer=layer)
        x = self.embed[tokens] @ self.w_qkv
        qkv = x.view(self.B, 1, -1, Hq + 2 * Hkv, D).expand(-1, self.attn_layers, -1, -1, -1).bfloat16().contiguous()
        self.cache.append(qkv[..., Hq:Hq + Hkv, :], qkv[..., Hq + Hkv:, :], count)

    def step(self, logp: np.ndarray, draft_tokens: np.ndarray, temperature: torch.Tensor):
        """One speculative step.  logp, draft_tokens [B, depth, top_k]: the draft's candidates at each depth."""
        B, n_max, dev = self.B, self.n_max, self.device
        Hq, Hkv, D = self.heads
        trees = [N.gdn_ddtree_build(logp[b], n_max, tau=6.0) for b in range(B)]
        sched = DeviceSchedule([t["parent"] for t in trees], n_max, dev)
        tokens = np.zeros((B, n_max), dtype=np.int64)
        for b, t in enumerate(trees):
            for i in range(1, len(t["parent"])):
                tokens[b, i] = draft_tokens[b, t["depth"][i] - 1, t["rank"][i]]
        tok = torch.from_numpy(tokens).to(dev)
        tok[:, 0] = self.last
        x = self.embed[tok]                                              # [B, n, width]
        # GDN layers: every node's output from its root path
        Hv = self.gdn.Hv
        raw, beta, log_g = self.gdn_inputs(x.unsqueeze(1).expand(-1, self.gdn_layers, -1, -1))
        boundary = torch.empty(B, self.gdn_layers, max(1, sched.nb_max), Hv, 128, 128, device=dev)
        self.verifier.verify(sched, raw, self.conv_w, beta, log_g, self.state, self.conv_state, self.out_o, boundary,
                             boundary_scratch=True)
        # attention layers: the nodes over the 4-bit cache and their own root paths (rows of one fused projection)
        qkv = (x @ self.w_qkv).view(B, 1, n_max, Hq + 2 * Hkv, D).expand(-1, self.attn_layers, -1, -1, -1)
        qkv = qkv.bfloat16().contiguous()
        q, k, v = qkv[..., :Hq, :], qkv[..., Hq:Hq + Hkv, :], qkv[..., Hq + Hkv:, :]
        self.cache.attention(q, k, v, self.out_a, sched=sched)
        # the target's logits, and which nodes it accepts
        h = torch.cat([self.out_o[:, -1].flatten(2), self.out_a[:, -1].flatten(2).float()], -1)
        logits = h @ self.w_logit
        # (stands for a draft that knows the target: drafted tokens are likely ones)
        parents = torch.from_numpy(np.maximum(sched.parents, 0)).to(dev).long()
        logits.view(B, -1).scatter_add_(1, parents * self.V + tok, torch.full_like(tok, 7, dtype=logits.dtype))
        logits = logits.bfloat16()
        uniform = torch.rand(B, n_max, generator=self.gen, device=dev)
        noise = torch.rand(B, self.V, generator=self.gen, device=dev).clamp_(1e-9, 1 - 1e-7)
        path, length, token = self.acceptor.accept(sched, logits, tok.int(), uniform, -torch.log(-torch.log(noise)),
                                                   temperature)
        # commit: the path, still on the device, in both kinds of layers
        self.verifier.commit(sched, path, length)
        self.cache.append(k, v, length, path=path)
        self.last.copy_(token)
        return path, length, token

    def draft(self):
        """The draft's candidates at each depth: log-probabilities and tokens, numpy [B, DEPTH, TOP_K]."""
        z = torch.einsum("bw,dwv->bdv", self.embed[self.last], self.w_draft).bfloat16()
        top, tokens, _, _ = self.scorer.score(z.view(self.B * DEPTH, self.V))
        shape = (self.B, DEPTH, TOP_K)
        return top.view(shape).cpu().numpy(), tokens.view(shape).cpu().numpy()

    def decode(self):
        """One token without a tree, greedily (after finish)."""
        B, (Hq, Hkv, D) = self.B, self.heads
        x = self.embed[self.last]
        raw, beta, log_g = self.gdn_inputs(x)
        out_o = torch.empty(B, self.gdn.Hv, 128, device=self.device)
        for layer in range(self.gdn_layers):
            self.runner.step(raw, self.conv_w, beta, log_g, self.state, self.conv_state, out_o, layer=layer)
        qkv = (x @ self.w_qkv).view(B, 1, 1, Hq + 2 * Hkv, D).expand(-1, self.attn_layers, -1, -1, -1).bfloat16().contiguous()
        out_a = torch.empty(B, self.attn_layers, 1, Hq, D, dtype=torch.bfloat16, device=self.device)
        q, k, v = qkv[..., :Hq, :], qkv[..., Hq:Hq + Hkv, :], qkv[..., Hq + Hkv:, :]
        self.cache.attention(q, k, v, out_a)
        self.cache.append(k, v, torch.ones(B, dtype=torch.int32, device=self.device))
        h = torch.cat([out_o.flatten(1), out_a[:, -1].flatten(1).float()], -1)
        _, tokens, _, entropy = self.scorer.score((h @ self.w_logit).bfloat16())
        self.last.copy_(tokens[:, 0])
        return self.last, entropy

    def finish(self):
        self.verifier.finish(self.state, self.conv_state)
        self.verifier.check_error()
        self.cache.check_error()
        self.acceptor.check_error()
        self.scorer.check_error()


def main(steps: int = 4, B: int = 4, show=print, decode: int = 0, **shape):
    model = HybridStack(B=B, **shape)
    rng = np.random.default_rng(1)
    dev = model.device
    count = torch.from_numpy(rng.integers(5, 70, B).astype(np.int32)).to(dev)
    model.prompt(torch.from_numpy(rng.integers(0, model.V, (B, 70))).to(dev), count)
    temperature = torch.full((B,), 0.8, device=dev)
    temperature[0] = 0.0
    lengths = [count]
    for s in range(steps):
        path, length, token = model.step(*model.draft(), temperature)
        lengths.append(length.clone())
        show(f"step {s}: accepted {length.tolist()} nodes, next tokens {token.tolist()}")
    model.finish()
    for s in range(decode):
        token, entropy = model.decode()
        lengths.append(torch.ones_like(count))
        show(f"token {s}: {token.tolist()}, entropies {[round(e, 2) for e in entropy.tolist()]}")
    cached = model.cache.seq_len
    assert torch.equal(cached, torch.stack(lengths).sum(0, dtype=torch.int32)), "the cache holds what was accepted"
    show(f"cached tokens {cached.tolist()}")
    return model


if __name__ == "__main__":
    main(decode=2)
