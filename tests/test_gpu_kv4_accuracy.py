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
