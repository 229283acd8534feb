"""The decode loop over an 8-bit cache against a replay in 64 bits: what lies in the
pages is what the definition stores there, and the tokens committed are those that the
model decodes greedily over these pages."""

import numpy as np
import pytest
import torch

import window_oracle as wo
from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def decode():
    require_gpu()
    from confidence_scheduled_speculative_gb300 import decode
    return decode


def stored(paged, r, n):
    """Keys and values of request r's first n positions, in 64 bits, from the pages."""
    page = paged.k.size(1)
    p = torch.arange(n, device="cuda")
    g, t = paged.block_table[r][p // page].long(), p % page
    return [wo.e4m3_values(x.view(torch.uint8)[g, t]) * s[g, :, t].double()[..., None]
            for x, s in ((paged.k, paged.k_scale), (paged.v, paged.v_scale))]


def replay(target, r, tokens, attend=True):
    """The target over one whole sequence in 64 bits with the pages' keys and values;
    logits, and for each layer the keys and values that the definition would store."""
    c, f, n = target.cfg, lambda t: t.double(), len(tokens)
    x = f(target.embed)[torch.tensor(tokens, device="cuda")]
    half = c.head_dim // 2
    cos, sin = (t[:, None] for t in f(target.cos_sin[:n]).split(half, 1))

    def norm_rope(h, w):
        h = h / (h.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * f(w)
        a, b = h[..., :half], h[..., half:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    causal = torch.ones(n, n, device="cuda", dtype=torch.bool).tril()
    group = c.n_q_heads // c.n_kv_heads
    due = []
    for paged, w_qkv, w_out, (wq, wk) in zip(target.caches, target.w_qkv, target.w_out, target.norms):
        q, k, v = (x @ f(w_qkv)).view(n, -1, c.head_dim).split([c.n_q_heads, c.n_kv_heads, c.n_kv_heads], 1)
        due.append((norm_rope(k, wk), v))
        k, v = (t.repeat_interleave(group, 1) for t in stored(paged, r, n))
        s = torch.einsum("ihd,jhd->hij", norm_rope(q, wq), k) * c.head_dim ** -0.5
        o = torch.einsum("hij,jhd->ihd", s.masked_fill(~causal, -torch.inf).softmax(-1), v)
        if attend:
            x = x + o.reshape(n, -1) @ f(w_out)
    return x @ f(target.head), due


# The error of the model's own bfloat16 run, relative to a row's largest values, after so
# many layers: a sum of some 8 roundings a layer and 4 outside, each of at most half a
# unit, grown by at most 4 by the layers' products (their norm is near 1, mix adds half).
def grown(layers):
    return 4 * (8 * layers + 4) * 2.0 ** -9


@pytest.mark.parametrize("gamma", [1, 7, 15])
def test_pages_and_tokens(decode, gamma):
    cfg = decode.ToyConfig(cache=torch.float8_e4m3fn)
    target = decode.ToyTarget(cfg, B=4, seed=40 + gamma)
    gen = np.random.default_rng(gamma)
    prompts = [gen.integers(0, cfg.vocab, n).tolist() for n in (2, 33, 70, 129)]
    out, rows = decode.generate(target, prompts, steps=8, gamma=gamma)
    assert max(rows) > 4 and sum(map(len, out)) > 4 * 8  # drafts were verified, and some accepted
    # one step more, of the tokens that are not stored yet, for the logits themselves
    i32 = dict(dtype=torch.int32, device="cuda")
    lens = torch.tensor([len(p) + len(t) - 1 for p, t in zip(prompts, out)], **i32)
    status, cu = torch.zeros(1, **i32), torch.arange(5, **i32)
    last = target.forward(torch.tensor([t[-1] for t in out], **i32), req=cu[:4], pos=lens, cu_seqlens=cu,
                          prefix_lens=lens, totals=cu[-1:], status=status).double()
    assert int(status) == 0
    for r, (prompt, tokens) in enumerate(zip(prompts, out)):
        assert len(tokens) >= 8
        sequence = prompt + tokens
        logits, due = replay(target, r, sequence)
        for layer, (paged, want) in enumerate(zip(target.caches, due)):
            for got, w in zip(stored(paged, r, len(sequence)), want):
                # half a step of an E4M3 code, 2^-4 of it, and of the smallest one
                most = w.abs().amax(-1, keepdim=True)
                bound = (w.abs() / 16 + most * 2.0 ** -18) * (1 + grown(layer)) + most * grown(layer)
                assert bool(((got - w).abs() <= bound).all()), (r, layer)
        error = grown(cfg.layers) * logits.abs().amax(-1)
        assert bool(((last[r] - logits[-1]).abs() <= error[-1]).all()), r
        # (and the bound sees the attention: without it the logits are others)
        bare = replay(target, r, sequence, attend=False)[0][-1]
        assert bool(((last[r] - bare).abs() > error[-1]).any()), r
        taken = torch.tensor(tokens, device="cuda")[:, None]
        before = slice(len(prompt) - 1, len(sequence) - 1)
        gap = logits[before].max(-1).values - logits[before].gather(1, taken)[:, 0]
        assert bool((gap <= 2 * error[before]).all()), (r, gap.max())
