"""Plain 64-bit definitions of the verify window's cache operators, and the
random problems their tests run on (test infrastructure only).

Written from the formulas with elementary float64 torch operations; nothing
here calls the library.  The bounds next to the definitions are the rounding
errors that the library's number formats allow, worked out from the formulas:
u32 = 2^-24 a 32-bit operation, u16 = 2^-8 a rounding to bfloat16."""

import math

import torch

U32, BF16, F16 = 2.0 ** -24, 2.0 ** -8, 2.0 ** -11
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}


def out_unit(dtype):
    """Largest relative error of the one rounding to an output's type."""
    return BF16 if dtype == torch.bfloat16 else U32


# ------------------------------------------------------------------ cache

class Cache:
    """A random paged cache: tensors for the library and the values they
    stand for, as [request, position, head, element] in 64 bits."""

    def __init__(self, gen, kind, tokens, heads, dim, page, layout="tokens", filled=True, spare=2,
                 pool=None, scale=1.0):
        self.kind, self.page, self.heads, self.dim = kind, page, heads, dim
        need = [-(-t // page) for t in tokens]
        self.n_pages = pool or sum(need) + spare
        width = max(need + [1])
        order = torch.randperm(self.n_pages, generator=gen)[:sum(need)].to(torch.int32)
        self.table = torch.full((len(tokens), width), -1, dtype=torch.int32)  # unused: no page
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = order[at:at + n]
            at += n
        self.table = self.table.cuda()
        shape = {"tokens": (self.n_pages, page, heads, dim), "heads": (self.n_pages, heads, page, dim)}[layout]
        g = torch.Generator("cuda").manual_seed(int(torch.randint(1 << 30, (1,), generator=gen)))
        self.k_scale = self.v_scale = None
        if kind == "e4m3":
            self.k_scale, self.v_scale = (
                (0.5 + torch.rand((self.n_pages, heads, page), generator=g, device="cuda")) * scale / 200
                for _ in range(2))
        tensors = []
        for _ in range(2):
            if kind == "e4m3":
                t = torch.zeros(shape, device="cuda", dtype=torch.uint8)
                if filled:
                    t.random_(0, 255, generator=g)
                    t[(t & 0x7F) == 0x7F] = 0  # NaN codes
                t = t.view(torch.float8_e4m3fn)
            else:
                t = torch.zeros(shape, device="cuda", dtype=DTYPES[kind])
                if filled:
                    t.normal_(0, scale, generator=g)
            tensors.append(t if layout == "tokens" else t.transpose(1, 2))
        self.k, self.v = tensors

    def kv(self):
        from confidence_scheduled_speculative_gb300 import api
        return api.KVCache(self.k, self.v, self.table, self.k_scale, self.v_scale)

    def slots(self, r, lo, hi):
        p = torch.arange(lo, hi, device="cuda")
        return self.table[r][p // self.page].long(), p % self.page

    def values(self, which, r, lo, hi):
        page, tok = self.slots(r, lo, hi)
        t = self.k if which == "k" else self.v
        if self.kind != "e4m3":
            return t[page, tok].double()
        s = self.k_scale if which == "k" else self.v_scale
        return e4m3_values(t.view(torch.uint8)[page, tok]) * s[page, :, tok].double()[..., None]

    def put(self, which, r, p, value):
        """Overwrite the entries of one position (every head) with a value."""
        page, tok = int(self.table[r, p // self.page]), p % self.page
        t = self.k if which == "k" else self.v
        if self.kind == "e4m3":
            t.view(torch.uint8)[page, tok] = 0x7F if math.isnan(value) else 0x38
            (self.k_scale if which == "k" else self.v_scale)[page, :, tok] = value
        else:
            t[page, tok] = value


def e4m3_values(code):
    """The numbers that E4M3 codes (uint8) stand for."""
    code = code.int()
    e, f = code >> 3 & 15, (code & 7).double()
    mag = torch.where(e > 0, (1 + f / 8) * torch.exp2(e.double() - 7), f / 8 * 2.0 ** -6)
    mag = torch.where((code & 0x7F) == 0x7F, math.nan, mag)
    return torch.where(code > 127, -mag, mag)


def e4m3_step(x):
    """Distance of neighbouring E4M3 numbers at |x|."""
    return torch.exp2(torch.floor(torch.log2(x.abs().clamp(2.0 ** -6, 448))) - 3)


# ---------------------------------------------------------- norm, rotation

def norm_rope(x, weight, eps, cos_sin, pos, interleaved):
    """[rows, heads, D] in 64 bits, and the largest error that 32-bit
    arithmetic may leave in each element before it is rounded."""
    D = x.size(-1)
    y = x.double()
    # each of x, 1/sqrt and the weight's product rounds; the sum of squares
    # has at most D terms one after the other
    units = 0.0
    if weight is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * weight.double()
        units = 0.5 * (D + 3) + 4
    tol = units * U32 * y.abs()
    if cos_sin is not None:
        R = cos_sin.size(1)
        c, s = (t[:, None, :] for t in cos_sin.double()[pos.long()].split(R // 2, 1))
        even = torch.arange(0, R, 2) if interleaved else torch.arange(R // 2)
        odd = even + (1 if interleaved else R // 2)
        a, b, ta, tb = (y[..., even].clone(), y[..., odd].clone(), tol[..., even].clone(),
                        tol[..., odd].clone())
        y[..., even], y[..., odd] = a * c - b * s, b * c + a * s
        ca, sa = c.abs(), s.abs()  # two products and a sum
        tol[..., even] = ta * ca + tb * sa + 3 * U32 * (a.abs() * ca + b.abs() * sa)
        tol[..., odd] = tb * ca + ta * sa + 3 * U32 * (b.abs() * ca + a.abs() * sa)
    return y, tol


# --------------------------------------------------------------- attention

def attention(q, cache, r, P, L, bits, scale):
    """Request r's rows q [L, heads, D]: out, lse and the largest errors that
    32-bit sums and `weight_unit` allow (see below), in 64 bits."""
    n, heads, D = P + L, q.size(1), q.size(2)
    G = heads // cache.heads
    sees = torch.ones((L, n), dtype=torch.bool)
    for i in range(L):
        for t in range(L):
            sees[i, P + t] = bool(bits[i] >> t & 1)
    sees = sees.cuda()[None]
    k = cache.values("k", r, 0, n).permute(1, 0, 2).repeat_interleave(G, 0)  # [heads, n, D]
    v = cache.values("v", r, 0, n).permute(1, 0, 2).repeat_interleave(G, 0)
    qq = q.double().permute(1, 0, 2)
    z = (qq @ k.transpose(1, 2) * scale).masked_fill(~sees, -math.inf)
    m = z.amax(-1, keepdim=True) if n else torch.full((heads, L, 1), -math.inf, device="cuda").double()
    m0 = m.masked_fill(m == -math.inf, 0.0)
    w = torch.exp(z - m0)
    w = torch.where(sees, w, 0.0)
    total = w.sum(-1, keepdim=True)
    w = torch.where(total > 0, w / total, 0.0) if n else w
    w = torch.where(torch.isnan(total), total, w)
    # what a row does not see has no effect on it: its values are left out
    # of the sum, not multiplied by zero
    if bool(torch.isfinite(v).all()):
        o, o_abs = w @ v, w @ v.abs()
    else:
        terms = [torch.where(sees[0, i][None, :, None], w[:, i, :, None] * v, 0.0) for i in range(L)]
        o, o_abs = (torch.stack([f(t).sum(1) for t in terms], 1) for f in (torch.Tensor.clone, torch.abs))
    lse = (m0 + total.log()).squeeze(-1)
    # a score: D products summed in 32 bits, times the scale; its exponential
    # is off by the same amount (relative) and by a few units of its own; a
    # weight's share is off by that twice over, and sums of n terms by n units
    s_abs = (qq.abs() @ torch.nan_to_num(k, 0, 0, 0).abs().transpose(1, 2)).amax(-1, keepdim=True) * abs(scale)
    s_tol = (D + 4) * U32 * s_abs + 16 * U32
    tol = o_abs * (2 * s_tol + 2 * (n + 16) * U32)
    lse_tol = s_tol.squeeze(-1) + (n + 16) * U32 + 4 * U32 * lse.abs()
    return (o.permute(1, 0, 2), lse.permute(1, 0), tol.permute(1, 0, 2), lse_tol.permute(1, 0),
            o_abs.permute(1, 0, 2))


def chain_bits(L):
    return [(2 << i) - 1 for i in range(L)]


def tree_bits(gen, L, orphans=False):
    """Ancestor words of a random tree; with `orphans` some rows see none of
    the window, themselves included."""
    bits = [1]
    for i in range(1, L):
        p = int(torch.randint(max(0, i - 4), i, (1,), generator=gen))
        bits.append(bits[p] | 1 << i)
    if orphans:
        bits = [0 if i % 3 == 1 else b for i, b in enumerate(bits)]
    return bits


def as_int32(bits):
    return torch.tensor([b - (1 << 32) if b >> 31 & 1 else b for b in bits], dtype=torch.int32)
