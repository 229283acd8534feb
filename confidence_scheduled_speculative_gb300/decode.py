"""The whole decode step around a paged cache, run together on a small model:
draft, plan and pack the verify window, normalise and rotate its queries and
keys and append them to the cache, attend over it, accept.

``PagedCache`` owns one layer's pages and the attention's workspace and makes
the two calls a layer needs.  ``ToyTarget`` is a target model of random
weights around it (no checkpoint is needed), and ``generate`` is the loop a
server would run: prompts enter in windows of up to 32 tokens, then each step
verifies what the drafter proposed.  Nothing but the committed tokens leaves
the device.  The drafter here is the target without its attention.

With ``keep`` the caches are kept short: each step adds the accepted rows' attention to
what every entry has gathered and evicts those that gathered least.  ``LatentToyTarget``
holds one latent vector a token instead of keys and values: prompts enter whole, in the
expanded form, windows attend in the absorbed one.

    python -m confidence_scheduled_speculative_gb300.decode --cache e4m3
    python -m confidence_scheduled_speculative_gb300.decode --keep 96 --recent 32
    python -m confidence_scheduled_speculative_gb300.decode --attention latent
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
    free list would), and the calls that write and read it.  ``ledger``: with what
    ``gather`` and ``evict`` need."""

    def __init__(self, B, max_len, n_q_heads, n_kv_heads, head_dim, *, page_size=64,
                 dtype=torch.bfloat16, seed=0, device="cuda", ledger=False):
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
        if ledger:  # what each entry has gathered, and its token's position
            lines = (B, n_kv_heads, width * page_size)
            self.weights = torch.zeros(lines, device=device)
            self.positions = torch.zeros(lines, dtype=torch.int32, device=device)
            self.evict_workspace = api.workspace(api.dspark_kv_evict_workspace_bytes(*lines), device)

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

    def attend(self, q, out, *, cu_seqlens, prefix_lens, scale, status, ancestors=None, lse=None,
               stream=None) -> None:
        api.dspark_tree_attention(q, self.cache, cu_seqlens=cu_seqlens, prefix_lens=prefix_lens,
                                  scale=scale, out=out, ancestors=ancestors, lse=lse,
                                  workspace=self.workspace, status=status, stream=stream)

    def gather(self, q, lse, *, cu_seqlens, prefix_lens, scale, pos, status, counts=None, decay=1.0,
               ancestors=None, stream=None) -> None:
        """Notes the window's accepted rows (``counts`` of each window): their positions, and
        what they attended to (``q`` and ``lse`` as ``attend`` had and left them)."""
        api.dspark_attention_weights(q, self.cache, lse=lse, cu_seqlens=cu_seqlens,
                                     prefix_lens=prefix_lens, scale=scale, ancestors=ancestors,
                                     counts=counts, decay=decay, weights=self.weights, pos=pos,
                                     positions=self.positions, status=status, stream=stream)

    def evict(self, *, lens, now, keep, recent, new_lens, status, stream=None) -> None:
        """Cuts every request down to ``keep`` entries a head, the ``recent`` last tokens
        among them; ``lens`` entries of ``now`` tokens become ``new_lens``."""
        api.dspark_kv_evict(self.cache, lens=lens, now=now, keep=keep, recent=recent,
                            weights=self.weights, positions=self.positions, new_lens=new_lens,
                            workspace=self.evict_workspace, status=status, stream=stream)


class PagedLatentCache:
    """One layer's latent cache for B requests of up to ``max_len`` tokens, as
    ``PagedCache``."""

    def __init__(self, B, max_len, n_q_heads, latent_dim, rope_dim, *, page_size=64,
                 dtype=torch.bfloat16, seed=0, device="cuda"):
        width = -(-max_len // page_size)
        order = torch.randperm(B * width, generator=torch.Generator().manual_seed(seed))
        self.block_table = order.to(torch.int32).view(B, width).to(device)
        self.pages = torch.zeros((B * width, page_size, latent_dim + rope_dim), device=device, dtype=dtype)
        self.cache = api.LatentCache(self.pages, self.block_table, latent_dim)
        self.workspace = api.workspace(
            api.dspark_latent_attention_workspace_bytes(n_q_heads, latent_dim), device)

    def append(self, rows, q_rope, q_rope_out, *, req, pos, cos_sin, weight, status, cache_pos=None,
               totals=None, stream=None) -> None:
        """The window's latent rows into their pages, its queries' rotated parts to
        ``q_rope_out`` in the same pass."""
        api.dspark_latent_append(rows, self.cache, req=req, pos=pos, cache_pos=cache_pos,
                                 q_rope=q_rope, q_rope_out=q_rope_out, totals=totals, weight=weight,
                                 cos_sin=cos_sin, status=status, stream=stream)

    def attend(self, q, out, *, cu_seqlens, prefix_lens, scale, status, ancestors=None,
               stream=None) -> None:
        api.dspark_latent_attention(q, self.cache, cu_seqlens=cu_seqlens, prefix_lens=prefix_lens,
                                    scale=scale, out=out, ancestors=ancestors,
                                    workspace=self.workspace, status=status, stream=stream)

    def rows(self, req, pos) -> torch.Tensor:
        """The entries of tokens at ``pos`` of requests ``req``, for the expanded form."""
        page = self.pages.size(1)
        return self.pages[self.block_table[req, pos // page].long(), pos % page]


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
    keep: int | None = None  # entries that a cache is kept to
    recent: int = 32  # of these, the last tokens whatever they gathered
    latent_dim: int = 512  # of LatentToyTarget, whose heads have head_dim + rope_dim elements
    rope_dim: int = 64


class ToyTarget:
    """Embedding, ``layers`` attention layers with a residual, output head."""

    def __init__(self, cfg: ToyConfig, B: int, seed: int = 0, device="cuda"):
        self.cfg, self.B, self.device = cfg, B, device
        self.gen = torch.Generator().manual_seed(seed)
        hidden = cfg.n_q_heads * cfg.head_dim
        self.embed = self._weight(cfg.vocab, hidden, by=1.0)
        self._layers(hidden, seed)
        self.head = self._weight(hidden, cfg.vocab, by=hidden ** -0.5)

    def _weight(self, *shape, by):
        return (torch.randn(shape, generator=self.gen) * by).to(self.cfg.dtype).to(self.device)

    def _angles(self, dim):
        angle = torch.arange(self.cfg.max_len, dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
        return torch.cat([angle.cos(), angle.sin()], 1).float().to(self.device)

    def _layers(self, hidden, seed):
        cfg, weight = self.cfg, self._weight
        columns = (cfg.n_q_heads + 2 * cfg.n_kv_heads) * cfg.head_dim
        self.w_qkv = [weight(hidden, columns, by=hidden ** -0.5) for _ in range(cfg.layers)]
        self.w_out = [weight(hidden, hidden, by=cfg.mix * hidden ** -0.5) for _ in range(cfg.layers)]
        self.norms = [(weight(cfg.head_dim, by=1.0).abs() + 0.5, weight(cfg.head_dim, by=1.0).abs() + 0.5)
                      for _ in range(cfg.layers)]
        self.cos_sin = self._angles(cfg.head_dim)
        self.caches = [PagedCache(self.B, cfg.max_len, cfg.n_q_heads, cfg.n_kv_heads, cfg.head_dim,
                                  dtype=cfg.cache, seed=seed + i, device=self.device, ledger=cfg.keep is not None)
                       for i in range(cfg.layers)]

    def forward(self, ids, *, req, pos, cu_seqlens, prefix_lens, totals, status,
                cache_pos=None) -> torch.Tensor:
        """Logits of the packed rows; their keys and values enter the caches.
        Only the first totals[0] rows are real.  ``prefix_lens``: the caches' entries;
        ``cache_pos``: where the rows are stored, if not at ``pos``."""
        c = self.cfg
        rows = ids.numel()
        heads = c.n_q_heads, c.n_q_heads + c.n_kv_heads
        x = self.embed[ids.long()]
        out = torch.zeros((rows, c.n_q_heads, c.head_dim), device=x.device, dtype=c.dtype)
        # for ``accepted``: each layer's queries and log sums
        self.window = dict(cu_seqlens=cu_seqlens, prefix_lens=prefix_lens, pos=pos, layers=[])
        for cache, w_qkv, w_out, norm in zip(self.caches, self.w_qkv, self.w_out, self.norms):
            qkv = (x @ w_qkv).view(rows, -1, c.head_dim)
            q, k, v = qkv[:, :heads[0]], qkv[:, heads[0]:heads[1]], qkv[:, heads[1]:]
            lse = None if c.keep is None else torch.zeros((rows, c.n_q_heads), device=x.device)
            cache.append(q, k, v, req=req, pos=pos, cache_pos=cache_pos, totals=totals, norm=norm,
                         cos_sin=self.cos_sin, status=status)
            cache.attend(q, out, cu_seqlens=cu_seqlens, prefix_lens=prefix_lens,
                         scale=c.head_dim ** -0.5, lse=lse, status=status)
            if c.keep is not None:
                self.window["layers"].append((q, lse))
            x = x + out.view(rows, -1) @ w_out
        return x @ self.head

    def accepted(self, counts, *, lens, now, status) -> None:
        """With ``keep``, after the first ``counts`` rows of each window were accepted (None:
        all): what they attended to is gathered, and the caches, of ``lens`` entries now and
        ``now`` tokens, are cut; ``lens`` is updated."""
        c, w, before = self.cfg, self.window, lens.clone()
        for cache, (q, lse) in zip(self.caches, w["layers"]):
            cache.gather(q, lse, cu_seqlens=w["cu_seqlens"], prefix_lens=w["prefix_lens"],
                         scale=c.head_dim ** -0.5, pos=w["pos"], counts=counts, status=status)
            cache.evict(lens=before, now=now, keep=c.keep, recent=c.recent, new_lens=lens, status=status)

    def draft(self, anchor: torch.Tensor, gamma: int) -> torch.Tensor:
        """What the target would say without its attention, gamma tokens on."""
        token, tokens = anchor.long(), []
        for _ in range(gamma):
            token = (self.embed[token] @ self.head).argmax(-1)
            tokens.append(token)
        return torch.stack(tokens, 1).to(torch.int32)


class LatentToyTarget(ToyTarget):
    """The same with latent attention: a token's keys and values are projections (w_uk, w_uv)
    of one latent vector, and a rotated key part is shared by all heads."""

    def _layers(self, hidden, seed):
        cfg, weight = self.cfg, self._weight
        if cfg.keep is not None:
            raise ValueError("keep: a latent cache is not cut")
        H, D, L, R = cfg.n_q_heads, cfg.head_dim, cfg.latent_dim, cfg.rope_dim
        n = range(cfg.layers)
        self.w_q = [weight(hidden, H * (D + R), by=hidden ** -0.5) for _ in n]
        self.w_kv = [weight(hidden, L + R, by=hidden ** -0.5) for _ in n]
        self.norms = [weight(L, by=1.0).abs() + 0.5 for _ in n]
        self.w_uk = [weight(H, D, L, by=L ** -0.5) for _ in n]
        self.w_uv = [weight(H, L, D, by=L ** -0.5) for _ in n]
        self.w_out = [weight(hidden, hidden, by=cfg.mix * hidden ** -0.5) for _ in n]
        self.cos_sin = self._angles(R)
        self.scale = (D + R) ** -0.5
        self.caches = [PagedLatentCache(self.B, cfg.max_len, H, L, R, dtype=cfg.cache, seed=seed + i,
                                        device=self.device) for i in n]

    def forward(self, ids, *, req, pos, cu_seqlens, prefix_lens, totals, status,
                cache_pos=None) -> torch.Tensor:
        c, rows = self.cfg, ids.numel()
        H, D, L, R = c.n_q_heads, c.head_dim, c.latent_dim, c.rope_dim
        x = self.embed[ids.long()]
        out = torch.zeros((rows, H, L), device=x.device, dtype=c.dtype)
        q_latent = torch.zeros((rows, H, L + R), device=x.device, dtype=c.dtype)
        for i, cache in enumerate(self.caches):
            q = (x @ self.w_q[i]).view(rows, H, D + R)
            # the key projection goes into the queries
            q_latent[..., :L] = torch.bmm(q[..., :D].transpose(0, 1), self.w_uk[i]).transpose(0, 1)
            cache.append(x @ self.w_kv[i], q[..., D:], q_latent[..., L:], req=req, pos=pos,
                         cache_pos=cache_pos, totals=totals, weight=self.norms[i], cos_sin=self.cos_sin,
                         status=status)
            cache.attend(q_latent, out, cu_seqlens=cu_seqlens, prefix_lens=prefix_lens, scale=self.scale,
                         status=status)
            o = torch.bmm(out.transpose(0, 1), self.w_uv[i]).transpose(0, 1)
            x = x + o.reshape(rows, -1) @ self.w_out[i]
        return x @ self.head

    def prompt(self, ids, *, req, pos, cu_seqlens, status) -> torch.Tensor:
        """Whole prompts into empty caches, in the expanded form: the cache's entries times
        the up projections are every head's keys and values."""
        c, rows = self.cfg, ids.numel()
        H, D, L, R = c.n_q_heads, c.head_dim, c.latent_dim, c.rope_dim
        x = self.embed[ids.long()]
        at = req.long(), pos.long()
        for i, cache in enumerate(self.caches):
            q = (x @ self.w_q[i]).view(rows, H, D + R)
            cache.append(x @ self.w_kv[i], q[..., D:], None, req=req, pos=pos, weight=self.norms[i],
                         cos_sin=self.cos_sin, status=status)
            entries = cache.rows(*at)
            latent = entries[:, :L].to(c.dtype)
            k, v = latent @ self.w_uk[i].flatten(0, 1).t(), torch.matmul(latent, self.w_uv[i])
            out = torch.zeros((rows, H, D), device=x.device, dtype=c.dtype)
            api.dspark_prompt_attention(q, k.view(rows, H, D), v.transpose(0, 1).contiguous(),
                                        k_shared=entries[:, L:].to(c.dtype), cu_seqlens=cu_seqlens,
                                        cu_keys=cu_seqlens, scale=self.scale, out=out, status=status)
            x = x + out.view(rows, -1) @ self.w_out[i]
        return x @ self.head


def prefill(target: ToyTarget, prompts, status) -> torch.Tensor:
    """Every prompt but its last token into the caches, in windows of up to 32 tokens (of a
    latent target whole, expanded); returns the caches' entries of each request: its tokens,
    or with ``keep`` those that are left."""
    device, i32 = target.embed.device, torch.int32
    lens = [len(p) - 1 for p in prompts]
    put = lambda x: torch.tensor(x, dtype=i32, device=device)
    latent, short = isinstance(target, LatentToyTarget), target.cfg.keep is not None
    # what is left of each request so far, if its caches are kept short
    cached = put([0] * len(lens) if short else lens)
    most = max(max(lens), 1) if latent else api.MAX_WINDOW
    for at in range(0, max(lens), most):
        part = [p[at:min(at + most, n)] for p, n in zip(prompts, lens)]
        sizes = [len(p) for p in part]
        req = put(np.repeat(np.arange(len(part)), sizes))
        pos = put(np.concatenate([np.arange(at, at + n) for n in sizes]))
        cu = put(np.concatenate([[0], np.cumsum(sizes)]))
        ids = put(np.concatenate(part))
        if latent:
            target.prompt(ids, req=req, pos=pos, cu_seqlens=cu, status=status)
            continue
        seen = put([min(at, n) for n in lens])
        where = dict(prefix_lens=seen)
        if short:
            where = dict(prefix_lens=cached.clone(), cache_pos=pos - (seen - cached)[req.long()])
        target.forward(ids, req=req, pos=pos, cu_seqlens=cu, totals=cu[-1:], status=status, **where)
        if short:
            cached += put(sizes)
            target.accepted(None, lens=cached, now=seen + put(sizes), status=status)
    return cached


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
    cached = prefill(target, prompts, vs.status)
    vs.prefix_lens.copy_(torch.tensor([len(p) - 1 for p in prompts], dtype=torch.int32))
    short = target.cfg.keep is not None
    vs.anchor.copy_(torch.tensor([int(p[-1]) for p in prompts], dtype=torch.int32))
    # the drafter's confidence: falls with the depth, differs between requests
    depth = torch.arange(gamma, device=device)
    vs.conf_logits.copy_(2.5 - 0.4 * depth - 0.1 * torch.arange(B, device=device)[:, None])
    committed, rows = [], []
    for _ in range(steps):
        vs.draft.copy_(target.draft(vs.anchor, gamma))
        vs.plan_pack()
        where = dict(prefix_lens=vs.prefix_lens)
        if short:  # the window is stored from the caches' ends on (pads have no request)
            evicted = torch.cat([vs.prefix_lens - cached, torch.zeros(1, dtype=torch.int32, device=device)])
            where = dict(prefix_lens=cached.clone(), cache_pos=vs.packed_pos - evicted[vs.packed_req.long()])
        logits = target.forward(vs.packed_ids, req=vs.packed_req, pos=vs.packed_pos, cu_seqlens=vs.cu_seqlens,
                                totals=vs.totals, status=vs.status, **where)
        vs.greedy_accept(logits)
        committed.append((vs.out_tokens.clone(), vs.commit_lens.clone()))
        rows.append(vs.totals.clone())
        # rejected rows' keys and values are overwritten by the next window
        if short:
            cached += vs.commit_lens
            target.accepted(vs.commit_lens, lens=cached, now=vs.new_seq_lens, status=vs.status)
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
    ap.add_argument("--attention", choices=("heads", "latent"), default="heads")
    ap.add_argument("--keep", type=int, help="entries that a cache is kept to")
    ap.add_argument("--recent", type=int, default=32, help="of these, the last tokens")
    args = ap.parse_args()
    if args.attention == "latent" and (args.cache == "e4m3" or args.keep is not None):
        ap.error("--attention latent holds bf16 or f32 and is not cut")
    if args.keep is not None and not 0 <= args.recent <= args.keep >= 1:
        ap.error("--keep: expected at least 1, and --recent no more than that")
    cfg = ToyConfig(cache=CACHE_DTYPES[args.cache], keep=args.keep, recent=args.recent)
    target = (LatentToyTarget if args.attention == "latent" else ToyTarget)(cfg, args.requests)
    gen = np.random.default_rng(0)
    prompts = [gen.integers(0, target.cfg.vocab, 5 + 23 * r) for r in range(args.requests)]
    tokens, rows = generate(target, prompts, args.steps, args.gamma)
    for r, t in enumerate(tokens):
        print(f"request {r}: {len(t)} tokens in {args.steps} steps: {t[:12]} ...")
    print(f"rows verified a step: {sum(rows) / len(rows):.1f}")


if __name__ == "__main__":
    main()
