"""The whole decode step around a paged cache, run together on a small model:
draft, plan and pack the verify window, normalise and rotate its queries and
keys and append them to the cache, attend over it, accept.

``PagedCache`` owns one layer's pages and the attention's workspace and makes
the two calls a layer needs.  ``ToyTarget`` is a target model of random
weights around it (no checkpoint is needed), and ``generate`` is the loop a
server would run: prompts enter in windows of up to 32 tokens, then each step
verifies what the drafter proposed.  Nothing but the committed tokens leaves
the device.  The drafter here is the target without its attention.

    python -m confidence_scheduled_speculative_gb300.decode --cache e4m3
"""

from __future__ import annotations

import argparse
import dataclasses

import numpy as np
import torch

from . import api
from .engine import StepConfig, VerifyStep

CACHE_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


class PagedCache:
    """One layer's cache for B requests of up to ``max_len`` tokens, every
    request with its own pages (handed out in a shuffled order, as a server's
    free list would), and the calls that write and read it."""

    def __init__(self, B, max_len, n_q_heads, n_kv_heads, head_dim, *, page_size=64,
                 dtype=torch.bfloat16, seed=0, device="cuda"):
        width = -(-max_len // page_size)
        shape = (B * width, page_size, n_kv_heads, head_dim)
        order = torch.randperm(B * width, generator=torch.Generator().manual_seed(seed))
        self.block_table = order.to(torch.int32).view(B, width).to(device)
        self.k = torch.zeros(shape, device=device, dtype=dtype)
        self.v = torch.zeros(shape, device=device, dtype=dtype)
        scale = None
        if dtype == torch.float8_e4m3fn:
            scale = [torch.ones((B * width, n_kv_heads, page_size), device=device)
                     for _ in range(2)]
        self.k_scale, self.v_scale = scale or (None, None)
        self.cache = api.KVCache(self.k, self.v, self.block_table, self.k_scale, self.v_scale)
        self.workspace = api.workspace(
            api.dspark_tree_attention_workspace_bytes(n_q_heads, head_dim), device)

    def append(self, q, k, v, *, req, pos, status, cache_pos=None, totals=None, q_out=None, norm=None,
               cos_sin=None, stream=None) -> None:
        """The window's keys and values into their pages, its queries
        normalised and rotated in the same pass (in place, or to ``q_out``).
        ``norm``: the query's and the key's norm weights.  ``cache_pos``: where
        the rows are stored, if that is not where they are rotated to (a
        tree's tokens rotate by their depth and lie in window order)."""
        q_weight, k_weight = norm or (None, None)
        api.dspark_kv_append(k, v, self.cache, req=req, pos=pos, cache_pos=cache_pos, q=q, q_out=q_out,
                             totals=totals, q_weight=q_weight, k_weight=k_weight, cos_sin=cos_sin,
                             status=status, stream=stream)

    def attend(self, q, out, *, cu_seqlens, prefix_lens, scale, status, ancestors=None,
               stream=None) -> None:
        api.dspark_tree_attention(q, self.cache, cu_seqlens=cu_seqlens, prefix_lens=prefix_lens,
                                  scale=scale, out=out, ancestors=ancestors,
                                  workspace=self.workspace, status=status, stream=stream)


@dataclasses.dataclass
class ToyConfig:
    vocab: int = 512
    layers: int = 2
    n_q_heads: int = 8
    n_kv_heads: int = 2
    head_dim: int = 64
    max_len: int = 512
    dtype: torch.dtype = torch.bfloat16
    cache: torch.dtype = torch.bfloat16
    mix: float = 0.5  # how much of the residual stream the attention adds


class ToyTarget:
    """Embedding, ``layers`` attention layers with a residual, output head."""

    def __init__(self, cfg: ToyConfig, B: int, seed: int = 0, device="cuda"):
        self.cfg, self.B = cfg, B
        gen = torch.Generator().manual_seed(seed)
        hidden = cfg.n_q_heads * cfg.head_dim
        columns = (cfg.n_q_heads + 2 * cfg.n_kv_heads) * cfg.head_dim

        def weight(*shape, by):
            return (torch.randn(shape, generator=gen) * by).to(cfg.dtype).to(device)

        self.embed = weight(cfg.vocab, hidden, by=1.0)
        self.w_qkv = [weight(hidden, columns, by=hidden ** -0.5) for _ in range(cfg.layers)]
        self.w_out = [weight(hidden, hidden, by=cfg.mix * hidden ** -0.5) for _ in range(cfg.layers)]
        self.norms = [(weight(cfg.head_dim, by=1.0).abs() + 0.5, weight(cfg.head_dim, by=1.0).abs() + 0.5)
                      for _ in range(cfg.layers)]
        self.head = weight(hidden, cfg.vocab, by=hidden ** -0.5)
        angle = torch.arange(cfg.max_len, dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, cfg.head_dim, 2, dtype=torch.float64) / cfg.head_dim)
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().to(device)
        self.caches = [PagedCache(B, cfg.max_len, cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim,
                                  dtype=cfg.cache, seed=seed + i, device=device)
                       for i in range(cfg.layers)]

    def forward(self, ids, *, req, pos, cu_seqlens, prefix_lens, totals, status) -> torch.Tensor:
        """Logits of the packed rows; their keys and values enter the caches.
        Only the first totals[0] rows are real."""
        c = self.cfg
        rows = ids.numel()
        heads = c.n_q_heads, c.n_q_heads + c.n_kv_heads
        x = self.embed[ids.long()]
        out = torch.zeros((rows, c.n_q_heads, c.head_dim), device=x.device, dtype=c.dtype)
        for cache, w_qkv, w_out, norm in zip(self.caches, self.w_qkv, self.w_out, self.norms):
            qkv = (x @ w_qkv).view(rows, -1, c.head_dim)
            q, k, v = qkv[:, :heads[0]], qkv[:, heads[0]:heads[1]], qkv[:, heads[1]:]
            cache.append(q, k, v, req=req, pos=pos, totals=totals, norm=norm, cos_sin=self.cos_sin,
                         status=status)
            cache.attend(q, out, cu_seqlens=cu_seqlens, prefix_lens=prefix_lens,
                         scale=c.head_dim ** -0.5, status=status)
            x = x + out.view(rows, -1) @ w_out
        return x @ self.head

    def draft(self, anchor: torch.Tensor, gamma: int) -> torch.Tensor:
        """What the target would say without its attention, gamma tokens on."""
        token, tokens = anchor.long(), []
        for _ in range(gamma):
            token = (self.embed[token] @ self.head).argmax(-1)
            tokens.append(token)
        return torch.stack(tokens, 1).to(torch.int32)


def prefill(target: ToyTarget, prompts, status) -> torch.Tensor:
    """Every prompt but its last token into the caches, in windows of up to
    32 tokens; returns the cached lengths."""
    device, i32 = target.embed.device, torch.int32
    lens = [len(p) - 1 for p in prompts]
    for at in range(0, max(lens), api.MAX_WINDOW):
        part = [p[at:min(at + api.MAX_WINDOW, n)] for p, n in zip(prompts, lens)]
        sizes = [len(p) for p in part]
        req = np.repeat(np.arange(len(part)), sizes)
        pos = np.concatenate([np.arange(at, at + n) for n in sizes])
        cu = torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=i32, device=device)
        prefix = torch.tensor([min(at, n) for n in lens], dtype=i32, device=device)
        target.forward(torch.tensor(np.concatenate(part), dtype=i32, device=device),
                       req=torch.tensor(req, dtype=i32, device=device),
                       pos=torch.tensor(pos, dtype=i32, device=device), cu_seqlens=cu,
                       prefix_lens=prefix, totals=cu[-1:], status=status)
    return torch.tensor(lens, dtype=i32, device=device)


def generate(target: ToyTarget, prompts, steps: int, gamma: int = 7):
    """``steps`` decode steps; returns the committed tokens of each request
    and the verified rows of each step."""
    B, device = target.B, target.embed.device
    budget = np.arange(1, B * (gamma + 1) + 1)
    vs = VerifyStep(StepConfig(
        B=B, gamma=gamma, V=target.cfg.vocab, logits_dtype=target.cfg.dtype, survival_eps=1e-3,
        min_verify_len=1, max_verify_len=gamma + 1, forced_budget=-1, cost_kind=0,
        cost_M=budget, cost_val=1000.0 / (1.0 + 0.02 * budget), bias_ms=0.0, alpha_ms=0.0, tiers=(),
        capacity=B * (gamma + 1)), device)
    vs.prefix_lens.copy_(prefill(target, prompts, vs.status))
    vs.anchor.copy_(torch.tensor([int(p[-1]) for p in prompts], dtype=torch.int32))
    # the drafter's confidence: falls with the depth, differs between requests
    depth = torch.arange(gamma, device=device)
    vs.conf_logits.copy_(2.5 - 0.4 * depth - 0.1 * torch.arange(B, device=device)[:, None])
    committed, rows = [], []
    for _ in range(steps):
        vs.draft.copy_(target.draft(vs.anchor, gamma))
        vs.plan_pack()
        logits = target.forward(vs.packed_ids, req=vs.packed_req, pos=vs.packed_pos,
                                cu_seqlens=vs.cu_seqlens, prefix_lens=vs.prefix_lens,
                                totals=vs.totals, status=vs.status)
        vs.greedy_accept(logits)
        committed.append((vs.out_tokens.clone(), vs.commit_lens.clone()))
        rows.append(vs.totals.clone())
        # rejected rows' keys and values are overwritten by the next window
        vs.prefix_lens.copy_(vs.new_seq_lens)
        vs.anchor.copy_(vs.bonus)
    if int(vs.status) != 0:
        raise RuntimeError(f"device status {int(vs.status):#x}")
    out = [[] for _ in range(B)]
    for tokens, lens in committed:
        for r, (row, n) in enumerate(zip(tokens.tolist(), lens.tolist())):
            out[r] += row[:n]
    return out, [int(t[0]) for t in rows]


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--gamma", type=int, default=7)
    ap.add_argument("--cache", choices=CACHE_DTYPES, default="bf16")
    args = ap.parse_args()
    target = ToyTarget(ToyConfig(cache=CACHE_DTYPES[args.cache]), args.requests)
    gen = np.random.default_rng(0)
    prompts = [gen.integers(0, target.cfg.vocab, 5 + 23 * r) for r in range(args.requests)]
    tokens, rows = generate(target, prompts, args.steps, args.gamma)
    for r, t in enumerate(tokens):
        print(f"request {r}: {len(t)} tokens in {args.steps} steps: {t[:12]} ...")
    print(f"rows verified a step: {sum(rows) / len(rows):.1f}")


if __name__ == "__main__":
    main()
