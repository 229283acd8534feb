"""The decode step around the paged cache: what speculative steps commit is
what the target's own greedy decoding gives."""

import numpy as np
import pytest
import torch

from gpu_helpers import require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def decode():
    require_gpu()
    from confidence_scheduled_speculative_gb300 import decode
    return decode


def logits64(target, tokens):
    """The target over one whole sequence in 64 bits, no cache and no paging."""
    c = target.cfg
    n = len(tokens)
    f = lambda t: t.double()
    x = f(target.embed)[torch.tensor(tokens, device="cuda")]
    half = c.head_dim // 2
    cos, sin = f(target.cos_sin[:n, :half]), f(target.cos_sin[:n, half:])

    def norm_rope(h, w):
        h = h / (h.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * f(w)
        a, b = h[..., :half], h[..., half:]
        cs, sn = cos[:, None], sin[:, None]
        return torch.cat([a * cs - b * sn, b * cs + a * sn], -1)

    causal = torch.ones(n, n, device="cuda", dtype=torch.bool).tril()
    for w_qkv, w_out, (wq, wk) in zip(target.w_qkv, target.w_out, target.norms):
        qkv = (x @ f(w_qkv)).view(n, -1, c.head_dim)
        q, k, v = qkv.split([c.n_q_heads, c.n_kv_heads, c.n_kv_heads], 1)
        group = c.n_q_heads // c.n_kv_heads
        q, k = norm_rope(q, wq), norm_rope(k, wk).repeat_interleave(group, 1)
        s = torch.einsum("ihd,jhd->hij", q, k) * c.head_dim ** -0.5
        p = s.masked_fill(~causal, -torch.inf).softmax(-1)
        o = torch.einsum("hij,jhd->ihd", p, v.repeat_interleave(group, 1))
        x = x + o.reshape(n, -1) @ f(w_out)
    return x @ f(target.head)


# The committed token's 64-bit logit is within twice the logits' error of the
# best one.  The error is a sum of some 8 roundings a layer and 4 outside, each of
# at most half a unit of its type relative to the row's largest values, grown by
# at most 4 by the layers' products (their norm is near 1, and mix adds half).
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -11}  # fp32 products may run as TF32


@pytest.mark.parametrize("dtype,cache", [("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("gamma", [1, 7, 31])
def test_speculative_steps_commit_the_greedy_tokens(decode, dtype, cache, gamma):
    cfg = decode.ToyConfig(dtype=decode.CACHE_DTYPES[dtype], cache=decode.CACHE_DTYPES[cache],
                           max_len=512)
    target = decode.ToyTarget(cfg, B=5, seed=gamma)
    gen = np.random.default_rng(gamma)
    prompts = [gen.integers(0, cfg.vocab, n).tolist() for n in (2, 33, 34, 70, 129)]
    out, rows = decode.generate(target, prompts, steps=8, gamma=gamma)
    unit = UNIT[cfg.dtype]
    for prompt, tokens in zip(prompts, out):
        assert len(tokens) >= 8
        logits = logits64(target, prompt + tokens)[len(prompt) - 1:-1]
        best = logits.max(-1).values
        taken = logits.gather(1, torch.tensor(tokens, device="cuda")[:, None])[:, 0]
        error = 4 * (8 * cfg.layers + 4) * unit / 2 * logits.abs().amax(-1)
        assert bool((best - taken <= 2 * error).all()), (best - taken).max()
    # drafts were verified, and some were accepted
    assert max(rows) > 5 and sum(map(len, out)) > 5 * 8


def test_8_bit_cache(decode):
    """The same loop over an 8-bit cache: every step commits between one and
    gamma + 1 tokens of the vocabulary, and drafts are accepted."""
    cfg = decode.ToyConfig(cache=torch.float8_e4m3fn, mix=0.25)
    prompts = [[3, 1, 4, 1, 5], [9, 2, 6]]
    out, rows = decode.generate(decode.ToyTarget(cfg, B=2, seed=4), prompts, steps=8)
    assert all(8 <= len(t) <= 64 for t in out) and sum(map(len, out)) > 16 and max(rows) > 2
    assert all(0 <= x < cfg.vocab for t in out for x in t)
