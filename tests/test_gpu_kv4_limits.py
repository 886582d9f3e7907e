"""Attention over a 4-bit cache at its limits: weights far below a row's largest, bounded waits,
one workspace for two captured graphs, query and scale extremes."""
import math

import pytest
import torch

from speculative_decoding_attention_verify_b200 import sdattn as sd

from . import kv_ref as R
from .test_gpu_kv4_attention import BF, Call, i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("gap", [20.0, 24.5, 28.5, 32.0])
@pytest.mark.parametrize("rows", [1, 3, 9])
def test_many_positions_of_next_to_no_weight(rows, gap, paged):
    """One position `gap` powers of two above 30,000 others, whose codes are zero (its values too): the
    output is what the others leave.  A weight is rounded to fp16 below a largest weight of 2^10 or more, so
    it is off by half a step, 2^-11 of itself, or by half of 2^-24, 2^-35 of the row's largest: over
    all positions 2^-11 sum p s c + 2^-35 max(p s) sum max(c, |c - 8|) on top of
    attention_bound's other terms."""
    h_q, h_kv, d, length = 7, 1, 128, 30000
    c = Call([length], [rows], h_q, h_kv, d, paged, seed=rows)
    # keys: position 5 all ones, the others zeros (s = 0, lo = the value); queries of one sum
    for w in range(2):
        codes = torch.zeros(h_kv, length, d, dtype=torch.uint8)
        param = torch.zeros(h_kv, length, 2, dtype=torch.bfloat16)
        if w == 0:
            param[:, 5, 1] = 1.0
        else:  # values: codes 1..15 by channel and position, s = 1, lo = 0; zeros at position 5
            codes[:] = (torch.arange(length)[:, None] + torch.arange(d)[None]) % 15 + 1
            param[..., 0] = 1.0
            codes[:, 5] = 0
        c.cache.store(w, 0, R.pack(codes), param)
        c.cache.parts[0][w] = (codes, param)
        c.cache.kv[0][w] = R.values(R.pack(codes), param)
    c.kv = c.cache.cuda()
    q = torch.full((rows, h_q, d), 0.5, dtype=BF)
    c.q.copy_(q)
    soft = gap * math.log(2) / (0.5 * d)
    c.queries = sd.Queries(q.cuda(), c.queries.q_start, rows, length, soft)
    out, flag = c.run()
    assert flag == 0
    ref, bound = R.attention_bound(q, c.cache, 0, BF, soft)
    vc = c.cache.parts[0][1][0].double()
    # p s is largest at position 5, where p < 1 and s = 1
    bound = bound + 2.0 ** -35 * torch.maximum(vc, (vc - 8).abs()).sum(1)[:, None].expand(1, h_q, d).reshape(1, h_q, d)
    assert ((out.double() - ref).abs() <= bound).all(), ((out.double() - ref).abs() / bound).max()


@pytest.mark.parametrize("rows", [1, 3, 9])
def test_queries_far_from_one(rows):
    """Rows of 1e-30 and 1e30, rows of zeros and single channels: the power of two that brings a
    row into fp16 is the row's own."""
    for size, soft in ((1e-30, 1e29), (1e30, 1e-31), (0.0, 0.0)):
        c = Call([500], [rows], 14, 2, 128, True, seed=rows)
        q = (c.q.float() * size).to(BF)
        q[:, 3] = 0
        q[:, 3, 17] = size
        c.q = q
        c.queries = sd.Queries(q.cuda(), c.queries.q_start, rows, 500, soft)
        c.softmax_scale = soft
        out, flag = c.run()
        assert flag == 0
        c.check(out)


@pytest.mark.parametrize("rows", [1, 9])
def test_two_graphs_share_a_workspace(rows):
    """Captured one after the other with one workspace, replayed in turns on one stream."""
    a = Call([6000, 90], [rows] * 2, 14, 2, 128, True, seed=1)
    b = Call([4000], [rows], 14, 2, 128, False, seed=2)
    need = max(sd.sd_kv4_attention_workspace_size(x.queries, x.kv) for x in (a, b))
    ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")
    want = [x.run()[0] for x in (a, b)]
    outs, graphs = [], []
    for x in (a, b):
        out = torch.empty_like(x.queries.q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sd.sd_kv4_verify_attention(x.queries, x.kv, out=out, workspace=ws)
        outs.append(out)
        graphs.append(g)
    for i in (0, 1, 0, 0, 1):
        outs[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[i].cpu(), want[i])


@pytest.mark.parametrize("heads,rows", [((28, 4, 128), 9), ((28, 4, 128), 4), ((8, 1, 64), 16)])
def test_expired_waits_set_the_timeout_flag_and_return(heads, rows):
    """With a bound of 1 ns the tcgen05 kernel's waits run out at once: the flag is set, the launch
    reports no error and the next call with the default bound is right."""
    c = Call([9000, 300], [rows] * 2, *heads, True, seed=rows)
    prev = sd.sd_set_wait_timeout_ns(1)
    try:
        _, flag = c.run()
    finally:
        sd.sd_set_wait_timeout_ns(prev)
    assert flag & sd.SD_DEVERR_TIMEOUT
    out, flag = c.run()
    assert flag == 0
    c.check(out)


@pytest.mark.parametrize("n", [1, 9])
@pytest.mark.parametrize("length", [240, 1000, 1024, 2048, 2049])
def test_whole_units_and_even_shares_agree(n, length):
    """The hint decides how the tiles are divided; the sequences do not change."""
    batch = 28
    lens = [max(n, length - 37 * i) for i in range(batch)]
    c = Call(lens, [n] * batch, 14, 2, 64, False, seed=length)
    short, _ = c.run()
    c.check(short)
    # (a looser hint, still within the cache's room, may divide them otherwise)
    c.queries = sd.Queries(c.queries.q, c.queries.q_start, n, length + 5)
    loose, _ = c.run()
    c.check(loose)


def test_empty_batches_of_rows():
    """No sequence has rows: nothing is written."""
    c = Call([40, 50], [1, 1], 14, 2, 128, False)
    c.queries = sd.Queries(c.queries.q, i32([0, 0, 0]), 1, 64 - 10)
    out, flag = c.run()
    assert flag == 0 and (out == 9).all()


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 8, 9, 16, 17])
def test_rows_at_the_borders_of_the_kernels(n, d, paged):
    """8 heads of one group: 8, 16, 24, 32, 40, 64, 72, 128 and 136 rows per KV head."""
    c = Call([n, 129, 1500], [n, 1, n], 8, 1, d, paged, seed=n, pad_rows=1)
    out, flag = c.run()
    assert flag == 0
    c.check(out)


@pytest.mark.parametrize("n", [2, 5])
def test_constant_rows(n):
    """Rows of one value (s = 0, codes 0) among others, on both tensor-core kernels: they stand for
    lo, whatever s they are counted with."""
    for low in (0.0, 3.0, -1e-20, 1e20):
        c = Call([300], [n], 7, 1, 128, False, seed=n)
        for w in range(2):
            codes, param = (x.clone() for x in c.cache.parts[0][w])
            if w == 1:
                codes[:, ::3] = 0
                param[:, ::3, 0] = 0
                param[:, ::3, 1] = low
            c.cache.store(w, 0, R.pack(codes), param)
            c.cache.parts[0][w] = (codes, param)
            c.cache.kv[0][w] = R.values(R.pack(codes), param)
        c.kv = c.cache.cuda()
        out, flag = c.run()
        assert flag == 0
        c.check(out)
