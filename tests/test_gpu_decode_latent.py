"""The decode loop over a latent cache: prompts enter in the expanded form, windows attend
in the absorbed one, and what is committed is the target's own greedy decoding."""

import numpy as np
import pytest
import torch

from gpu_helpers import require_gpu
from test_gpu_decode import UNIT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def decode():
    require_gpu()
    from confidence_scheduled_speculative_gb300 import decode
    return decode


def logits64(target, tokens):
    """The target over one whole sequence in 64 bits: keys and values of every head, no
    cache and no paging."""
    c, n, f = target.cfg, len(tokens), lambda t: t.double()
    H, D, L, R = c.n_q_heads, c.head_dim, c.latent_dim, c.rope_dim
    x = f(target.embed)[torch.tensor(tokens, device="cuda")]
    cos, sin = (t[:, None] for t in f(target.cos_sin[:n]).split(R // 2, 1))

    def turn(h):
        a, b = h[..., :R // 2], h[..., R // 2:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)

    causal = torch.ones(n, n, device="cuda", dtype=torch.bool).tril()
    for w_q, w_kv, w, uk, uv, w_out in zip(target.w_q, target.w_kv, target.norms, target.w_uk, target.w_uv,
                                           target.w_out):
        q = (x @ f(w_q)).view(n, H, D + R)
        kv = x @ f(w_kv)
        latent = kv[:, :L] / (kv[:, :L].pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * f(w)
        k = torch.einsum("jl,hdl->jhd", latent, f(uk))
        s = torch.einsum("ihd,jhd->hij", q[..., :D], k)
        s = s + torch.einsum("ihd,jd->hij", turn(q[..., D:]), turn(kv[:, None, L:])[:, 0])
        p = (s * target.scale).masked_fill(~causal, -torch.inf).softmax(-1)
        o = torch.einsum("hij,jl,hld->ihd", p, latent, f(uv))
        x = x + o.reshape(n, -1) @ f(w_out)
    return x @ f(target.head)


# As in test_gpu_decode: roundings of at most half a unit of the row's largest values, some
# 12 a layer here (two projections in, the absorbed query, norm, rotation, weights, the
# latent output, two projections out, the sum) and 4 outside, grown by at most 4.
@pytest.mark.parametrize("dtype,head_dim", [("bf16", 128), ("bf16", 64), ("f32", 64)])
@pytest.mark.parametrize("gamma", [1, 7])
def test_speculative_steps_commit_the_greedy_tokens(decode, dtype, head_dim, gamma):
    cfg = decode.ToyConfig(dtype=decode.CACHE_DTYPES[dtype], cache=decode.CACHE_DTYPES[dtype], head_dim=head_dim,
                           max_len=512)
    target = decode.LatentToyTarget(cfg, B=5, seed=gamma)
    gen = np.random.default_rng(gamma)
    prompts = [gen.integers(0, cfg.vocab, n).tolist() for n in (1, 2, 33, 70, 300)]
    out, rows = decode.generate(target, prompts, steps=8, gamma=gamma)
    unit = UNIT[cfg.dtype]
    for prompt, tokens in zip(prompts, out):
        assert len(tokens) >= 8
        logits = logits64(target, prompt + tokens)[len(prompt) - 1:-1]
        best = logits.max(-1).values
        taken = logits.gather(1, torch.tensor(tokens, device="cuda")[:, None])[:, 0]
        error = 4 * (12 * cfg.layers + 4) * unit / 2 * logits.abs().amax(-1)
        assert bool((best - taken <= 2 * error).all()), (best - taken).max()
    assert max(rows) > 5 and sum(map(len, out)) > 5 * 8
