"""Speculative cycles of a small target model over the paged cache.

`CachedCycle` joins the draft/schedule/verify calls (`cycle.DeviceCycle`) with
the paged cache (`kv_cache.PagedCache`): in `DeviceCycle` alone the logits of
draft and target are given, here they come from attention over what the
requests hold in the cache. One cycle of B requests, nothing waiting on the host:

  draft backbone   K mask rows a request attend to its cached context (not causal)
  ds_draft_block, ds_confidence_schedule            K tokens, lengths L_b <= K
  update           room for the anchor and L_b draft tokens
  target           per layer append and (causal) attend, 1 + L_b rows a request
  ds_verify        the accepted prefix and one more token, the next anchor
  update           back to the anchor and the accepted tokens

    python -m speculative_decoding_draft_block_gb300.cached --requests 8 --cycles 16

The model is an illustration with random weights: root-mean-square norms,
attention with grouped heads, residuals, no feed-forward blocks; PyTorch does its
projections. Draft and target share the head's transition term E[x] P, so drafts
are accepted now and then. The cache holds a request's tokens up to the one
before its anchor, the last token emitted.
"""

import argparse

import torch

from .cycle import DeviceCycle
from .kv_cache import PagedCache
from .workloads import TINY, make_inputs, scaled


def _norm(x):
    y = x.float()
    return (y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class TargetModel:
    """Random weights of a decoder with `n_layers` layers of width d."""

    def __init__(self, V, d, n_layers, n_heads, n_kv_heads, head_dim, E, P, dtype, device, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def w(n, m, gain=1.0):
            return (torch.randn((n, m), device=device, generator=g) * (gain * n ** -0.5)).to(dtype)

        self.n_heads, self.n_kv_heads, self.head_dim, self.d = n_heads, n_kv_heads, head_dim, d
        self.embed = w(V + 1, d, (V + 1) ** 0.5)          # the last row: the draft's mask token
        self.qkv = [w(d, (n_heads + 2 * n_kv_heads) * head_dim) for _ in range(n_layers)]
        self.out = [w(n_heads * head_dim, d) for _ in range(n_layers)]
        self.head = w(d, V, 0.3)
        self.E, self.P = E, P
        self.mask = V
        self.freq = torch.exp(torch.arange(0, d, 2, device=device) * (-9.0 / d))

    def rows(self, token, position):
        angle = position.unsqueeze(-1).float() * self.freq
        return (self.embed[token].float() + torch.cat([angle.sin(), angle.cos()], -1)).to(self.embed.dtype)

    def forward(self, x, attention):
        """`attention(layer, q, k, v)` for the rows x; the last layer's normalised states."""
        Hq, Hk, D = self.n_heads, self.n_kv_heads, self.head_dim
        for layer, (wi, wo) in enumerate(zip(self.qkv, self.out)):
            q, k, v = (_norm(x) @ wi).view(-1, Hq + 2 * Hk, D).split([Hq, Hk, Hk], 1)
            x = x + attention(layer, q, k, v).reshape(-1, Hq * D) @ wo
        return _norm(x)

    def logits(self, states, token):
        return states @ self.head + self.E[token] @ self.P


class CachedCycle:
    def __init__(self, inp, n_layers=2, n_heads=4, n_kv_heads=2, head_dim=64, page_size=16, n_pages=512,
                 max_len=1024, device="cuda", seed=0):
        self.cyc = cyc = DeviceCycle(inp, device=device)
        t = cyc.t
        self.B, self.K = cyc.B, cyc.K
        dtype = t["E"].dtype
        self.model = TargetModel(cyc.V, cyc.d, n_layers, n_heads, n_kv_heads, head_dim, t["E"], t["P"], dtype, device,
                                 seed)
        self.cache = PagedCache(n_layers, n_pages, page_size, n_kv_heads, head_dim, self.B, max_len, dtype=dtype,
                                device=device)
        self.anchor = t["anchor"]
        self.step_of = torch.arange(self.K + 1, device=device, dtype=torch.int32)
        self.request_of = torch.arange(self.B, device=device, dtype=torch.int32)
        self.draft_start = torch.arange(self.B + 1, device=device, dtype=torch.int32) * self.K

    def _run(self, token, q_start, max_q, first):
        """The model over ragged rows, their keys and values going to the cache. `first`
        [B]: position of a request's first row. Rows past q_start[B] belong to nobody."""
        row = torch.arange(token.shape[0], device=token.device, dtype=torch.int32)
        b = (torch.searchsorted(q_start, row, right=True) - 1).clamp(max=self.B - 1)
        x = self.model.rows(token, first[b] + row - q_start[b])

        def attention(layer, q, k, v):
            self.cache.append(layer, k, v, q_start)
            return self.cache.attend(layer, q, q_start, max_q, out=torch.zeros_like(q))

        return self.model.forward(x, attention)

    def prompt(self, prompts):
        """Fills the cache: `prompts` holds B lists of tokens, the last of each the anchor."""
        dev = self.anchor.device
        n = torch.tensor([len(p) - 1 for p in prompts], dtype=torch.int32, device=dev)
        q_start = torch.nn.functional.pad(n.cumsum(0, dtype=torch.int32), (1, 0))
        self.anchor.copy_(torch.tensor([p[-1] for p in prompts], dtype=torch.int32))
        self.cache.update(n)
        token = torch.tensor([x for p in prompts for x in p[:-1]], dtype=torch.int32, device=dev)
        if token.numel():
            self._run(token, q_start, max(len(p) - 1 for p in prompts), torch.zeros_like(n))

    def _draft_context(self):
        """Base logits and states of the draft block, from K mask rows a request."""
        B, K, cyc = self.B, self.K, self.cyc
        past = self.cache.kv_len
        position = past[:, None] + 1 + self.step_of[:K]
        x = self.model.rows(torch.full((B * K,), self.model.mask, device=past.device), position.reshape(-1))
        x = self.model.forward(x, lambda layer, q, k, v: self.cache.attend(layer, q, self.draft_start, K, causal=False))
        cyc.t["h"].copy_(x.view(B, K, -1))
        cyc.t["base_logits"].copy_((x @ self.model.head).view(B, K, -1))

    def step(self, seed):
        """One cycle. The emitted tokens are in `cyc.out_tokens`, `cyc.num_emitted` of them."""
        B, K, cyc, cache = self.B, self.K, self.cyc, self.cache
        self._draft_context()
        cyc.draft(seed)
        cyc.schedule()
        past = cache.kv_len.clone()
        n = cyc.sched_len + 1
        q_start = torch.nn.functional.pad(n.cumsum(0, dtype=torch.int32), (1, 0))
        block = torch.cat([self.anchor[:, None], cyc.draft_tokens], 1)          # [B][K + 1]
        at = q_start[:-1, None] + torch.minimum(self.step_of, n[:, None] - 1)   # row of a block's token
        token = torch.zeros(B * (K + 1), dtype=torch.int32, device=past.device)
        token.scatter_(0, at.reshape(-1).long(), block.gather(1, torch.minimum(self.step_of, n[:, None] - 1).long()).reshape(-1))
        cache.update(past + n)
        states = self._run(token, q_start, K + 1, past)
        cyc.t["target_logits"].copy_(self.model.logits(states, token)[at])
        cyc.verify(seed)
        emitted = cyc.num_emitted
        cache.update(past + emitted)
        self.anchor.copy_(cyc.out_tokens.gather(1, (emitted - 1).long()[:, None])[:, 0])

    def fork(self, parent):
        """Request b continues as a copy of request parent[b]; their pages are shared until written."""
        p = parent.long()
        self.cache.update(self.cache.kv_len[p], parent=parent)
        self.anchor.copy_(self.anchor[p])

    def check_status(self):
        self.cyc.check_status()
        self.cache.check_status()


def small_inputs(B=4, K=4, temperature=0.0, seed=0):
    """Weights and shapes of a float32 cycle (V = 1024, hidden size 256), with a
    transition term that outweighs the states' part of the logits."""
    w = scaled(TINY, name="cached", B=B, K=K, temps=(temperature,), seed=seed)
    inp = make_inputs(w)
    inp["E"] = inp["E"] * 8
    return inp


def main(argv=None):
    ap = argparse.ArgumentParser(description="speculative cycles of a small model over the paged cache")
    ap.add_argument("--requests", type=int, default=8)
    ap.add_argument("--cycles", type=int, default=16)
    ap.add_argument("--temperature", type=float, default=0.0)
    a = ap.parse_args(argv)
    inp, page = small_inputs(a.requests, temperature=a.temperature), 16
    prompts = [range(7 * b, 7 * b + 3 + 9 * b) for b in range(a.requests)]
    # room for the longest request to grow by K + 1 tokens every cycle, in pages of its own
    longest = len(prompts[-1]) + a.cycles * (inp["base_logits"].shape[1] + 1)
    c = CachedCycle(inp, page_size=page, n_pages=a.requests * -(-longest // page), max_len=longest)
    c.prompt([[i % c.cyc.V for i in p] for p in prompts])
    emitted = torch.zeros(a.requests, dtype=torch.int32, device=c.anchor.device)
    for i in range(a.cycles):
        if i == a.cycles // 2:   # the first request ends, a copy of the last takes its place
            parent = c.request_of.clone()
            parent[0] = a.requests - 1
            c.fork(parent)
            c.cache.compact()
        c.step(0x5EED + i)
        emitted += c.cyc.num_emitted
    c.check_status()
    held = int((c.cache.ref > 0).sum())
    print("%d cycles of %d requests: %.2f tokens a cycle and request, lengths %s, %d pages held of which %d shared" %
          (a.cycles, a.requests, emitted.sum().item() / max(1, a.cycles * a.requests), c.cache.kv_len.tolist(), held,
           int((c.cache.ref > 1).sum())))


if __name__ == "__main__":
    main()
