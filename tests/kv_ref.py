"""Plain 64-bit forms of the cache appends and of attention over a 4-bit cache (CPU tensors), and
builders of caches, for the tests of those calls."""
import math

import torch

from speculative_decoding_attention_verify_b200 import sdattn as sd

PAGE = 16
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


# ---- rotation ---------------------------------------------------------------------------

def frequencies(rot, theta=10000.0, scaling=sd.SD_ROPE_UNSCALED, factor=1.0, original_len=0,
                inv_freq=None, gain=0.0):
    """(frequencies, gain) in 64 bits, from the header's definitions."""
    if inv_freq is not None:
        f = torch.tensor([float(torch.tensor(x, dtype=torch.float32)) for x in inv_freq],
                         dtype=torch.float64)
        return f, gain or 1.0
    if scaling == sd.SD_ROPE_NTK:
        theta = theta * factor ** (rot / (rot - 2))
    m = torch.arange(rot // 2, dtype=torch.float64)
    f = torch.tensor(theta, dtype=torch.float64) ** (-2 * m / rot)
    if scaling == sd.SD_ROPE_LINEAR:
        f = f / factor
    if scaling == sd.SD_ROPE_YARN:
        c = lambda n: rot * math.log(original_len / (2 * math.pi * n)) / (2 * math.log(theta))  # noqa: E731
        lo, hi = max(math.floor(c(32)), 0), min(math.ceil(c(1)), rot - 1)
        hi = hi if hi > lo else lo + 0.001
        t = ((m - lo) / (hi - lo)).clamp(0, 1)
        f = f * (1 - t) + t * f / factor
        gain = gain or 0.1 * math.log(factor) + 1
    return f, gain or 1.0


def rotate(x, pos, rot, layout, f, gain):
    """x [rows][heads][d] (any dtype) rotated in 64 bits, and |a| + |b| of every element's pair."""
    x = x.double()
    if rot == 0:
        return x, torch.zeros_like(x)
    angle = pos.double()[:, None, None] * f
    c, s = gain * angle.cos(), gain * angle.sin()
    i = torch.arange(rot // 2)
    ia, ib = (i, i + rot // 2) if layout == sd.SD_ROPE_HALF else (2 * i, 2 * i + 1)
    a, b = x[..., ia], x[..., ib]
    y, size = x.clone(), torch.zeros_like(x)
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = a.abs() + b.abs()
    return y, size * gain


# ---- 4 bits -----------------------------------------------------------------------------

def quantise(x):
    """Rows of x (in their own dtype): (codes uint8, param bf16 [..., 2]) as the header defines."""
    xd = x.double()
    bad = ~torch.isfinite(xd).all(-1, keepdim=True)
    lo = xd.amin(-1, keepdim=True).float().bfloat16()
    hi = xd.amax(-1, keepdim=True)
    s = ((hi - lo.double()) / 15).float().bfloat16()
    s = torch.where(hi > lo.double(), s, torch.zeros_like(s))
    bad |= ~torch.isfinite((hi - lo.double()).float()) | ~torch.isfinite(lo)
    sd_ = torch.where(s > 0, s, torch.ones_like(s)).double()
    c = ((xd - lo.double()) / sd_).round().clamp(0, 15)
    c = torch.where((s > 0) & ~bad, c, torch.zeros_like(c))
    s = torch.where(bad, torch.zeros_like(s), s)
    lo = torch.where(bad, torch.full_like(lo, float("nan")), lo)
    return c.to(torch.uint8), torch.cat([s, lo], -1)


def pack(c):
    return c[..., 0::2] | (c[..., 1::2] << 4)


def unpack(codes):
    return torch.stack([codes & 15, codes >> 4], -1).flatten(-2)


def values(codes, param):
    """Values (64 bits) that stored rows stand for."""
    p = param.double()
    return p[..., 1:] + p[..., :1] * unpack(codes).double()


class Cache4:
    """A filled 4-bit cache on the CPU: sequences of the given lengths, contiguous with room for
    the longest or in shuffled pages, unused slots holding NaN parameters and random codes."""

    def __init__(self, lens, h_kv, d, paged, seed=0, spare=5, scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.h_kv, self.d, self.paged = list(lens), h_kv, d, paged
        b, longest = len(lens), max(max(lens), 1)
        if paged:
            used = [-(-n // PAGE) for n in lens]
            pool = sum(used) + 3
            order = torch.randperm(pool, generator=g)
            self.table = torch.full((b, max(max(used), 1) + 1), -1, dtype=torch.int32)
            at = 0
            for i, u in enumerate(used):
                self.table[i, :u] = order[at:at + u].int()
                at += u
            shape = (pool, h_kv, PAGE)
        else:
            self.table = None
            shape = (b, h_kv, longest + spare)
        self.codes = [torch.randint(0, 256, (*shape, d // 2), generator=g).to(torch.uint8)
                      for _ in range(2)]
        self.param = [torch.full((*shape, 2), float("nan"), dtype=torch.bfloat16) for _ in range(2)]
        self.kv = []  # per sequence: K, V values in 64 bits [h_kv][n][d]
        self.parts = []
        for i, n in enumerate(lens):
            pair, raw = [], []
            for w in range(2):
                x = (scale * torch.randn(h_kv, n, d, generator=g)).bfloat16()
                c, p = quantise(x)
                self.store(w, i, pack(c), p)
                pair.append(values(pack(c), p))
                raw.append((c, p))
            self.kv.append(pair)
            self.parts.append(raw)

    def slots(self, i, n):
        j = torch.arange(n)
        if self.paged:
            return self.table[i, j // PAGE].long(), j % PAGE
        return torch.full((n,), i), j

    def store(self, w, i, codes, param):
        a, j = self.slots(i, codes.shape[1])
        self.codes[w][a, :, j] = codes.transpose(0, 1)
        self.param[w][a, :, j] = param.transpose(0, 1)

    def cuda(self, dtype=torch.bfloat16, kv_len=None):
        t = lambda x: x.cuda() if x is not None else None  # noqa: E731
        lens = torch.tensor(self.lens if kv_len is None else kv_len, dtype=torch.int32).cuda()
        return sd.KV4Cache(t(self.codes[0]), t(self.codes[1]), t(self.param[0]), t(self.param[1]),
                           lens, t(self.table), dtype=dtype)


def attention(q, k, v, scale=None):
    """q [n][h_q][d], k / v [h_kv][len][d] in 64 bits: the rows are the last n positions."""
    n, h_q, d = q.shape
    h_kv, length, _ = k.shape
    g = h_q // h_kv
    s = torch.einsum("nhd,hld->hnl", q.double(), k.repeat_interleave(g, 0))
    s = s * (scale if scale else 1 / math.sqrt(d))
    hide = torch.arange(length)[None] > (length - n + torch.arange(n))[:, None]
    p = torch.softmax(s.masked_fill(hide, -math.inf), -1)
    # (a row sums over the positions it sees alone: a hidden NaN stays hidden)
    vv = v.repeat_interleave(g, 0)
    return torch.stack([torch.einsum("hl,hld->hd", p[:, i, :length - n + i + 1],
                                     vv[:, :length - n + i + 1]) for i in range(n)])


def attention_bound(q, cache, i, dtype, scale=None):
    """Elementwise bound of the library's error for sequence i.

    bf16: the weight of every position, times V's scale, is rounded to fp16 (half a step, 2^-11)
    before it multiplies the code c; the output is rounded once (2^-8 of itself).  fp32 parts: a
    score's error is below scale * sum|q_e| * (15 s + |lo|) * 2^-20 (128 products of at most 15
    steps, each a few 2^-24 of the running sum), which moves every weight by that much relative to
    itself; 2^-18 covers the sums of weights, their exponentials and logarithms, and the merges.
    Both act on the codes' part s c and the low values' part of a value separately.  The kernel for
    many rows multiplies c - 8 instead of c and adds 8 s to lo, so the larger of c and |c - 8| (at
    most 15 as before) bounds what a rounded weight multiplies; for a row of one value (s = 0) it
    counts s = 2^-8 |lo| with the code -8, whose rounding is 2^-11 8 2^-8 |lo| = 2^-16 |lo|."""
    k, v = cache.kv[i]
    n, h_q, d = q.shape
    g = h_q // cache.h_kv
    sc = scale if scale else 1 / math.sqrt(d)
    (_, kp), (vc, vp) = cache.parts[i]
    out = attention(q, k, v, scale)
    step = kp[..., 0].double().abs() * 15 + kp[..., 1].double().abs()
    worst = step.amax(-1).repeat_interleave(g, 0)[None, :, None]
    err = sc * q.double().abs().sum(-1, keepdim=True) * worst * 2.0 ** -20 + 2.0 ** -18
    most = torch.maximum(vc.double(), (vc.double() - 8).abs())
    codes = attention(q, k, (vp[..., :1].double() * most).abs(), scale)
    lows = attention(q, k, vp[..., 1:].double().abs().expand_as(v), scale)
    parts = codes + lows
    bound = 2 * err * parts + HALF_STEP[dtype] * out.abs()
    if dtype == torch.bfloat16:
        bound = bound + 2.0 ** -11 * codes + 2.0 ** -16 * lows
    return out, bound
