"""Attention over a 4-bit cache: errors that a bound linear in the weights does not show."""
import math

import pytest
import torch

from speculative_decoding_attention_verify_b200 import sdattn as sd

from . import kv_ref as R
from .test_gpu_kv4_attention import BF, Call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("log_scale", [-6, -8, -10])
@pytest.mark.parametrize("low", [0.0, 2.0 ** -7])
@pytest.mark.parametrize("rows", [1, 2, 5, 9])
def test_a_sink_of_one_value(rows, low, log_scale):
    """Position 0 takes most of the softmax (its score is 24 powers of two above the others') and
    its value row is constant, so it has no scale of its own.  The others' weights, in fp16, must
    not be measured against its weight: with s = |low| / 256 for it, the largest p s is at most
    max(2^-15, the others' 2^-24 2^-6), and a weight is off by 2^-11 of itself or by 2^-35 of that
    largest: 2^-35 max(p s) sum max(c, |c - 8|) on top of attention_bound's terms.  The length is
    one that a single CTA takes as a whole, so that the sink meets many others in its warp."""
    h_q, h_kv, d, length = 7, 1, 128, 1280
    c = Call([length], [rows], h_q, h_kv, d, False, seed=rows)
    g = torch.Generator().manual_seed(rows)
    # keys: ones at position 0, zeros elsewhere (s = 0, lo = the value); queries of one sum
    param = torch.zeros(h_kv, length, 2, dtype=BF)
    param[:, 0, 1] = 1.0
    codes = torch.zeros(h_kv, length, d, dtype=torch.uint8)
    keep = [(codes, param)]
    x = (2.0 ** log_scale * 4 * torch.randn(h_kv, length, d, generator=g)).to(BF)
    x[:, 0] = low
    keep.append(R.quantise(x))
    for w, (codes, param) in enumerate(keep):
        c.cache.store(w, 0, R.pack(codes), param)
        c.cache.parts[0][w] = (codes, param)
        c.cache.kv[0][w] = R.values(R.pack(codes), param)
    c.kv = c.cache.cuda()
    q = torch.full((rows, h_q, d), 0.5, dtype=BF)
    soft = 24 * math.log(2) / (0.5 * d)
    c.queries = sd.Queries(q.cuda(), c.queries.q_start, rows, length, soft)
    out, flag = c.run()
    assert flag == 0
    ref, bound = R.attention_bound(q, c.cache, 0, BF, soft)
    vc, vp = (t.double() for t in c.cache.parts[0][1])
    scale = torch.where(vp[..., :1] == 0, vp[..., 1:].abs() / 256, vp[..., :1])[0, :, 0]
    p = torch.full((length,), 2.0 ** -24, dtype=torch.float64)
    p[0] = 1.0
    top = (p * scale).max() / p.sum()
    most = torch.maximum(vc, (vc - 8).abs())[0].sum(0)
    bound = bound + 2.0 ** -35 * top * most
    err = (out.double() - ref).abs()
    assert (err <= bound).all(), (err / bound).max()


class Long:
    """One sequence in a contiguous cache on the GPU, and 64-bit attention over it there."""

    def __init__(self, q, h_kv, codes, param, softmax_scale=0.0):
        rows, h_q, d = q.shape
        length = codes[0].shape[1]
        self.shape, self.q = (length, rows, h_q, h_kv, d), q
        self.codes, self.param = codes, param
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        kv = sd.KV4Cache(*(R.pack(c)[None].contiguous() for c in codes),
                         *(x[None].contiguous() for x in param), i32([length]))
        self.out = sd.sd_kv4_verify_attention(
            sd.Queries(self.q, i32([0, rows]), rows, length, softmax_scale), kv).double()

    def weights(self, head):
        """Softmax weights [rows][length] of a query head, in 64 bits."""
        length, rows, h_q, h_kv, d = self.shape
        g = head // (h_q // h_kv)
        k = self.param[0][g, :, 1:].double() + self.param[0][g, :, :1].double() * self.codes[0][g].double()
        s = (self.q[:, head].double() @ k.T) / math.sqrt(d)
        j = torch.arange(length, device="cuda")
        hide = j[None] > (length - rows + torch.arange(rows, device="cuda"))[:, None]
        return torch.softmax(s.masked_fill(hide, -math.inf), -1)


@pytest.mark.parametrize("odd", [0, 1])
@pytest.mark.parametrize("rows", [1, 2, 5, 9])
def test_values_that_cancel(rows, odd):
    """140,000 positions in pairs of one key, values s (c - 8) and -s (c - 8) with s = 1 (lo = -8, c
    from 1 to 15): the exact output of a row that sees whole pairs is zero, and the rounding of a
    pair's weights cancels too (the same weight multiplies c - 8 and 8 - c).  What is left is how
    the products are summed.  A sum of 16 products and an accumulator in 24 bits cuts each term at
    2^-23 of the largest, and a product is at most 8 w: 17 2^-23 8 max(w) for 16 positions.  1 / s,
    lo / s + 8 and their sums are fp32: 8 2^-23 sum(p) = 2^-20.  An unpaired last position has its
    weight's rounding, 2^-11 8 p; the output is rounded once."""
    h_q, h_kv, d, length = 28, 4, 128, 140000
    g = torch.Generator(device="cuda").manual_seed(rows)
    rnd = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    kc = rnd(0, 16, h_kv, length // 2, d).repeat_interleave(2, 1)
    half = rnd(1, 16, h_kv, length // 2, d)
    vc = torch.stack([half, 16 - half], 2).flatten(1, 2)
    param = lambda s, lo: torch.tensor([s, lo], device="cuda").to(BF).expand(h_kv, length, 2)  # noqa: E731
    q = torch.randn(rows, h_q, d, generator=g, device="cuda").to(BF)
    c = Long(q, h_kv, (kc, vc), (param(0.35, -2.6), param(1.0, -8.0)))
    for head in range(h_q):
        p = c.weights(head)
        ref = p @ (vc[head // 7].double() - 8)
        tol = 17 * 2.0 ** -23 * 8 * p.view(rows, -1, 16).amax(-1).sum(-1) + 2.0 ** -20
        seen = length - rows + 1 + torch.arange(rows, device="cuda")
        last = p[torch.arange(rows, device="cuda"), seen - 1] * (seen % 2)
        tol = tol + 2.0 ** -11 * 8 * last
        err = ((c.out[:, head] - ref).abs() - 2.0 ** -8 * ref.abs())[:, odd::2]
        assert (err <= tol[:, None]).all(), (head, (err / tol[:, None]).max().item())


@pytest.mark.parametrize("rows", [1, 2, 5, 9])
def test_long_random_contexts(rows):
    """100,003 random positions quantised as sd_kv4_append does, of which 1% have keys that point where
    the queries do and take most of the softmax: the output is a small part of the values, and what
    the many others leave is cut off first where a sum is short of bits.  Three independent roundings, in rms over all outputs: the
    output's (known exactly); every weight's to 11 bits, uniform within half a step and so of variance
    (2^-10 p)^2 / 12 at most, times s (c - 8); and what is held in fp32, which may add as much as the
    weights' again (it is a tenth of it).  Even and odd channels apart, 2% for the spread of an rms of
    more than 3,000 values, whose squares vary by 0.9 of their mean (3 sigma: 3 0.9 / 2 / 57)."""
    h_q, h_kv, d, length = 56, 8, 128, 100003
    g = torch.Generator(device="cuda").manual_seed(rows + 20)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    q, k, v = normal(rows, h_q, d).to(BF), normal(h_kv, length, d), normal(h_kv, length, d)
    hit = torch.rand(h_kv, length, generator=g, device="cuda") < 0.01
    to = 4 * q[-1].float().view(h_kv, -1, d).mean(1)
    both = [R.quantise(x.to(BF)) for x in (torch.where(hit[..., None], to[:, None], k), v)]
    c = Long(q, h_kv, [x[0] for x in both], [x[1] for x in both])
    total = torch.zeros(3, 2, dtype=torch.float64, device="cuda")  # squares: error, output's, weights'
    for head in range(h_q):
        p = c.weights(head)
        s, lo = (both[1][1][head // 7, :, i:i + 1].double() for i in range(2))
        codes = both[1][0][head // 7].double()
        ref = p @ (lo + s * codes)
        var = p.square() @ (s * (codes - 8)).square() * (2.0 ** -20 / 12)
        for i, x in enumerate(((c.out[:, head] - ref).square(),
                               (ref.to(BF).double() - ref).square(), 4 * var)):
            total[i] += x.view(-1, 2).sum(0)
    ratio = (total[0] / (total[1] + total[2])).sqrt()
    assert (ratio <= 1.02).all(), ratio.tolist()


@pytest.mark.parametrize("A,B", [(0.9921875, 4.96875), (0.671875, 4.3125)])
@pytest.mark.parametrize("rows", [1, 2, 3, 9, 10, 18])
def test_weights_are_rounded_once(rows, A, B):
    """A row's maximum moves within a tile, after weights of the tile have been rounded: position 0
    scores 0, positions 1 to 31 A below it, position 40 B above it (in log2 units), the rest nothing.
    Values are zero: codes 8 with lo = -8, but codes 0 with lo = 0 at positions 1 to 31, so that the
    output is 8 times the error of their weights, which is half a step, 2^-11, at most; A and B are such
    that rounding 2^-A and then 2^-B times that gives 1.7 times as much.  Sums in fp32: 2^-20."""
    h_q, h_kv, d, length = 7, 1, 128, 200
    score = torch.full((length,), -100.0)
    score[0], score[1:32], score[40] = 0.0, -A, B
    assert torch.equal(score, score.to(BF).float())
    kc = torch.zeros(h_kv, length, d, dtype=torch.uint8, device="cuda")
    kp = torch.stack([torch.zeros(length), score], -1).to(BF)[None].cuda()
    low = torch.zeros(length, dtype=torch.bool)
    low[1:32] = True
    vc = torch.where(low, 0, 8).to(torch.uint8)[None, :, None].expand(h_kv, length, d).cuda()
    vp = torch.stack([torch.ones(length), torch.where(low, 0.0, -8.0)], -1).to(BF)[None].cuda()
    q = torch.zeros(rows, h_q, d, dtype=BF, device="cuda")
    q[..., 5] = 1.0
    c = Long(q, h_kv, (kc, vc), (kp, vp), softmax_scale=math.log(2))
    p = 2.0 ** score.double()
    share = p[1:32].sum() / p.sum()
    assert (c.out.abs() <= 2.0 ** -11 * 8 * share * (1 + 2.0 ** -8) + 2.0 ** -20).all(), \
        (c.out.abs().max() / share * 2 ** 8).item()
