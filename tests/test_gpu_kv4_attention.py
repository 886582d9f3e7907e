"""Attention over a 4-bit cache on the GPU against 64-bit attention over the values that the
cache's rows stand for.  The bound of every output element is derived in kv_ref.attention_bound."""
import pytest
import torch

import oracle
from speculative_decoding_attention_verify_b200 import device as dev
from speculative_decoding_attention_verify_b200 import inputs as gen
from speculative_decoding_attention_verify_b200 import sdattn as sd

from . import kv_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


class Call:
    def __init__(self, lens, rows, h_q, h_kv, d, paged, dtype=BF, seed=0, pad_rows=0, scale=1.0,
                 softmax_scale=0.0, rows_hint=0, len_hint=0):
        self.cache = R.Cache4(lens, h_kv, d, paged, seed=seed, scale=scale)
        self.rows, self.dtype, self.softmax_scale = rows, dtype, softmax_scale
        g = torch.Generator().manual_seed(seed + 1)
        self.starts = [0]
        for n in rows:
            self.starts.append(self.starts[-1] + n)
        total = self.starts[-1] + pad_rows
        self.q = torch.randn(total, h_q, d, generator=g).to(dtype)
        self.kv = self.cache.cuda(dtype)
        longest = len_hint or max(max(lens), 1)
        self.queries = sd.Queries(self.q.cuda(), i32(self.starts), rows_hint or max(max(rows), 1),
                                  longest, softmax_scale)

    def run(self, **kw):
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full_like(self.queries.q, 9.0)
        sd.sd_kv4_verify_attention(self.queries, self.kv, out=out, dev_err=flag, **kw)
        torch.cuda.synchronize()
        return out.cpu(), flag.item()

    def check(self, out, skip=()):
        for i, n in enumerate(self.rows):
            a, b = self.starts[i], self.starts[i + 1]
            if n == 0 or i in skip:
                assert (out[a:b] == 9).all()
                continue
            ref, bound = R.attention_bound(self.q[a:b], self.cache, i, self.dtype,
                                           self.softmax_scale)
            err = (out[a:b].double() - ref).abs()
            assert torch.isfinite(err).all(), f"sequence {i}"
            worst = (err / bound.clamp_min(1e-300)).max().item()
            assert (err <= bound).all(), f"sequence {i}: {worst} of the bound, error {err.max()}"
        assert (out[self.starts[-1]:] == 9).all()  # rows behind the last sequence


SHAPES = [(28, 4, 128), (4, 1, 64), (16, 16, 64), (8, 1, 128), (2, 2, 128)]
LENGTHS = [[1], [2, 15], [16, 17, 31], [127, 128, 129], [300, 8, 1], [1000], [4100, 33]]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("heads", SHAPES)
@pytest.mark.parametrize("lens", LENGTHS, ids=str)
def test_lengths_of_single_tokens(lens, heads, paged, dtype):
    h_q, h_kv, d = heads
    c = Call(lens, [1] * len(lens), h_q, h_kv, d, paged, dtype, seed=sum(lens))
    out, flag = c.run()
    assert flag == 0
    c.check(out)


ROWS = [2, 3, 4, 5, 9, 13, 16, 18, 19, 40]


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("heads", SHAPES[:3])
@pytest.mark.parametrize("n", ROWS)
def test_several_rows(n, heads, paged):
    """Every engine: from 2 rows per KV head to more than 128."""
    h_q, h_kv, d = heads
    c = Call([n, n + 1, 200, 777], [n, max(1, n - 1), 1, n], h_q, h_kv, d, paged, seed=n, pad_rows=2)
    out, flag = c.run()
    assert flag == 0
    c.check(out)


@pytest.mark.parametrize("n", [2, 9, 20])
def test_several_rows_fp32(n):
    c = Call([n, 130, 1000], [n, 1, n], 28, 4, 128, True, F32, seed=n)
    out, flag = c.run()
    assert flag == 0
    c.check(out)


@pytest.mark.parametrize("n", [1, 9])
def test_sequences_without_rows_between_others(n):
    c = Call([40, 0, 100, 7, 0], [n, 0, n, 0, 0], 28, 4, 128, True, seed=3, pad_rows=1)
    out, flag = c.run()
    assert flag == 0
    c.check(out)


@pytest.mark.parametrize("n", [1, 2, 4, 9])
@pytest.mark.parametrize("batch", [300, 700])
def test_many_short_sequences(batch, n):
    """More sequences than a block has threads, several units in one CTA's share."""
    lens = [n + (i * 37) % 150 for i in range(batch)]
    c = Call(lens, [n if i % 5 else 0 for i in range(batch)], 4, 2, 64, False, seed=batch)
    out, flag = c.run()
    assert flag == 0
    c.check(out)


@pytest.mark.parametrize("n", [1, 2, 5, 9, 17])
def test_one_long_sequence_among_short_ones(n):
    c = Call([20000, n, 50, 300], [n] * 4, 14, 2, 128, True, seed=n)
    out, flag = c.run()
    assert flag == 0
    c.check(out)


@pytest.mark.parametrize("n", [1, 3, 9])
def test_loose_hints_change_nothing_but_the_plan(n):
    a = Call([500, 2000], [n, n], 14, 2, 128, False, seed=5)
    out, _ = a.run()
    a.check(out)
    b = Call([500, 2000], [n, n], 14, 2, 128, True, seed=5, rows_hint=n + 5, len_hint=2009)
    out, _ = b.run()
    b.check(out)


@pytest.mark.parametrize("n", [1, 9])
def test_large_and_tiny_values(n):
    """Keys and values far from one, and a softmax that one position decides."""
    for scale, soft in ((1e4, 1e-5), (1e-4, 0.0), (30.0, 0.0)):
        c = Call([700], [n], 28, 4, 128, False, seed=9, scale=scale, softmax_scale=soft)
        out, flag = c.run()
        assert flag == 0
        c.check(out)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [2, 9, 40])
def test_nan_rows_reach_those_that_see_them_only(n, dtype):
    """A NaN key or value at the last position: earlier rows of the step must not see it."""
    for w in (0, 1):
        c = Call([300], [n], 14, 2, 64, False, dtype, seed=n)
        param = (c.kv.k_param, c.kv.v_param)[w]
        codes = (c.kv.k, c.kv.v)[w]
        codes[0, 1, 299] = 0
        param[0, 1, 299] = torch.tensor([0.0, float("nan")])
        out, _ = c.run()
        assert out[n - 1, 7:].isnan().all() and not out[n - 1, :7].isnan().any()
        assert not out[:n - 1].isnan().any()
        ref, bound = R.attention_bound(c.q, c.cache, 0, dtype)
        assert ((out.double() - ref).abs() <= bound)[:n - 1].all()


@pytest.mark.parametrize("n", [1, 9])
def test_rows_that_are_all_nan(n):
    c = Call([5 * n], [n], 14, 2, 64, False, seed=n)
    c.kv.k_param.fill_(float("nan"))
    out, _ = c.run()
    assert out.isnan().all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 2, 9])
def test_violated_hints_skip_the_sequence(n, dtype):
    for what in ("rows", "short", "long", "pages"):
        c = Call([60, 80, 90], [n, n, n], 14, 2, 64, True, dtype, seed=2)
        if what == "rows":
            if n == 1:
                continue
            c.queries = sd.Queries(c.queries.q, i32([0, n - 1, 2 * n, 3 * n]), n, 90)
            c.starts, c.rows = [0, n - 1, 2 * n, 3 * n], [n - 1, n + 1, n]
        elif what == "short":
            c.kv.kv_len[1] = n - 1
        elif what == "long":
            c.kv.kv_len[1] = 91
        else:
            c.queries = sd.Queries(c.queries.q, i32(c.starts), n, 4096)
            c.kv.kv_len[1] = 16 * c.kv.block_table.shape[1] + 1
        out, flag = c.run()
        assert flag == sd.SD_DEVERR_SHAPE, what
        c.check(out, skip=(1,))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 2, 9])
def test_bad_pages_count_as_zeros(n, dtype):
    c = Call([60, 80], [n, n], 14, 2, 128, True, dtype, seed=2)
    c.kv.block_table[1, 2] = c.kv.k.shape[0]
    out, flag = c.run()
    assert flag == sd.SD_DEVERR_PAGE
    for i in range(2):
        c.cache.kv[1][i][:, 32:48] = 0
        c.cache.parts[1][i][1][:, 32:48] = 0
    c.check(out)


@pytest.mark.parametrize("n", [1, 2, 4, 9])
def test_unaligned_rows_and_outputs(n):
    """Queries and outputs that are not 16-byte aligned take the CUDA-core engine."""
    c = Call([333], [n], 4, 1, 64, False, seed=n)
    flat = torch.zeros(c.q.numel() + 1, dtype=BF, device="cuda")
    q = flat[1:].view(c.q.shape)
    q.copy_(c.q)
    out = torch.full((c.q.numel() + 1,), 9.0, dtype=BF, device="cuda")
    c.queries = sd.Queries(q, c.queries.q_start, n, 333)
    got = sd.sd_kv4_verify_attention(c.queries, c.kv, out=out[1:].view(c.q.shape))
    c.check(got.cpu())
    assert out[0] == 9


@pytest.mark.parametrize("n", [1, 2, 9, 40])
def test_two_streams_with_their_own_workspaces_and_repeatability(n):
    a = Call([5000, 70], [n, n], 14, 2, 128, True, seed=1)
    b = Call([3000], [n], 14, 2, 128, False, seed=2)
    want = [x.run()[0] for x in (a, b)]
    for x, w in zip((a, b), want):
        x.check(w)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(3):
        for x, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                outs.append(sd.sd_kv4_verify_attention(x.queries, x.kv))
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        assert torch.equal(o.cpu().view(torch.int16), want[i % 2].view(torch.int16))


@pytest.mark.parametrize("n", [1, 2, 9])
def test_captured_and_replayed_as_the_cache_grows(n):
    """One graph, replayed with other lengths, rows and queries, and a workspace full of NaN."""
    c = Call([900, 40], [n, n], 14, 2, 128, True, seed=4)
    need = sd.sd_kv4_attention_workspace_size(c.queries, c.kv)
    ws = torch.full((max(need, 16) // 4 + 4,), float("nan"), device="cuda").view(torch.uint8)
    out = torch.empty_like(c.queries.q)
    sd.sd_kv4_verify_attention(c.queries, c.kv, out=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sd.sd_kv4_verify_attention(c.queries, c.kv, out=out, workspace=ws)
    for lens in ([900, 40], [n, 39], [450, n]):
        c.kv.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        c.queries.q.copy_(torch.randn_like(c.queries.q, dtype=F32).to(BF))
        ws.view(torch.float32).fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        got = out.cpu()
        q = c.queries.q.cpu()
        for i in range(2):
            short = R.Cache4.__new__(R.Cache4)
            short.__dict__ = dict(c.cache.__dict__)
            short.kv = [[x[:, :lens[i]] for x in c.cache.kv[i]]]
            short.parts = [[(a[:, :lens[i]], b[:, :lens[i]]) for a, b in c.cache.parts[i]]]
            ref, bound = R.attention_bound(q[i * n:(i + 1) * n], short, 0, BF)
            assert ((got[i * n:(i + 1) * n].double() - ref).abs() <= bound).all(), (lens, i)


@pytest.mark.parametrize("rows", [1, 9])
def test_offsets_beyond_32_bits(rows):
    """Pages past 2^32 bytes of the pool."""
    h_kv, d = 8, 128
    pages = (2 ** 32 // (h_kv * 16 * 64)) + 9
    small = R.Cache4([40], h_kv, d, True, seed=6)
    kv = small.cuda()
    at = torch.tensor([pages - 2, pages - 5, pages - 9])
    big = [torch.zeros((pages, *t.shape[1:]), dtype=t.dtype, device="cuda")
           for t in (kv.k, kv.v, kv.k_param, kv.v_param)]
    for t, s in zip(big, (kv.k, kv.v, kv.k_param, kv.v_param)):
        t[at.cuda()] = s[small.table[0, :3].long().cuda()]
    cache = sd.KV4Cache(*big, kv.kv_len, i32([at.tolist()]))
    q = torch.randn(rows, 16, d, generator=torch.Generator().manual_seed(1)).to(BF)
    out = sd.sd_kv4_verify_attention(sd.Queries(q.cuda(), i32([0, rows]), rows, 40), cache).cpu()
    ref, bound = R.attention_bound(q, small, 0, BF)
    assert ((out.double() - ref).abs() <= bound).all()


def test_against_the_oracle_with_the_workloads_of_the_repository():
    """The ragged paged batch's shapes (shrunk), quantised by sd_kv4_append itself: the oracle's
    dense verification over the stored values."""
    w = gen.make_attn_workload(4, l_vis=900, l_txt=80, batch=3, paged=False, nan_tail=False)
    lens = [int(n) for n in w.kv_len_verify]
    k, v = (dev.tensor(x, gen.BF16) for x in (w.k, w.v))
    cap = k.shape[2]
    cache = sd.KV4Cache.empty(3, 4, cap, 128, dev.int32(lens))
    rows = lambda t: torch.cat([t[i, :, :n].transpose(0, 1) for i, n in enumerate(lens)]).contiguous()  # noqa: E731
    starts = [0]
    for n in lens:
        starts.append(starts[-1] + n)
    k4, v4 = torch.empty_like(rows(k)), torch.empty_like(rows(v))
    sd.sd_kv4_append(None, sd.NewRows(rows(k), rows(v), i32(starts), cap), cache, k_out=k4, v_out=v4)
    out = sd.sd_kv4_verify_attention(dev.verify_queries(w), cache)
    kk, vv = torch.zeros_like(k), torch.zeros_like(v)
    for i, n in enumerate(lens):
        kk[i, :, :n] = k4[starts[i]:starts[i + 1]].transpose(0, 1)
        vv[i, :, :n] = v4[starts[i]:starts[i + 1]].transpose(0, 1)
    bits = lambda t: t.cpu().view(torch.int16).numpy().view("uint16")  # noqa: E731
    ref = oracle.verify_attention(w.h_q, w.q_verify, w.q_verify_start,
                                  oracle.Cache(w.dtype, bits(kk), bits(vv), w.kv_len_verify, 4, 128))
    # (k_out and v_out are rounded to bf16 once more than the cache: 2e-2 as every bf16 test)
    assert abs(dev.to_numpy_f64(out) - ref).max() <= 2e-2
    dense = sd.sd_verify_attention(dev.verify_queries(w), sd.KVCache(kk, vv, cache.kv_len))
    assert (dense.float() - out.float()).abs().max().item() <= 2e-2


@pytest.mark.parametrize("paged", [False, True])
def test_a_cycle_of_appends_verification_and_acceptance(paged):
    """As a program uses them: a prompt goes into a dense and a 4-bit cache, then steps append
    their rows with the rotation, attend, and accept on logits made from the attention."""
    h_q, h_kv, d, n, steps, prompt = 8, 2, 64, 4, 3, [70, 33]
    cap = 128
    g = torch.Generator().manual_seed(8)
    kv_len = i32([0, 0])
    if paged:
        table = i32([[9, 2, 5, 0, 11, 7, 1, 3], [4, 13, 6, 8, 10, 12, 14, 15]])
        mk = lambda w, t: torch.zeros((16, h_kv, 16, w), dtype=t, device="cuda")  # noqa: E731
    else:
        table = None
        mk = lambda w, t: torch.zeros((2, h_kv, cap, w), dtype=t, device="cuda")  # noqa: E731
    c16 = sd.KVCache(mk(d, BF), mk(d, BF), kv_len, table)
    c4 = sd.KV4Cache(mk(d // 2, torch.uint8), mk(d // 2, torch.uint8), mk(2, BF), mk(2, BF), kv_len,
                     table)
    rope = sd.Rope(d, theta=1e6)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    hist = [[torch.zeros(h_kv, 0, d).double() for _ in range(2)] for _ in range(2)]
    parts = [[[], []], [[], []]]
    lens = [0, 0]
    for step in range(steps + 1):
        counts = prompt if step == 0 else [n, n]
        starts = [0, counts[0], sum(counts)]
        lens = [a + b for a, b in zip(lens, counts)]
        kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        qkv = torch.randn(starts[-1], h_q + 2 * h_kv, d, generator=g).to(BF).cuda()
        rows = sd.NewRows(qkv[:, h_q:h_q + h_kv], qkv[:, h_q + h_kv:], i32(starts), cap,
                          q=qkv[:, :h_q])
        q16 = sd.sd_kv_append(rope, rows, c16, dev_err=flag)
        k4, v4 = (torch.empty(starts[-1], h_kv, d, dtype=BF, device="cuda") for _ in range(2))
        q4 = sd.sd_kv4_append(rope, rows, c4, k_out=k4, v_out=v4, dev_err=flag)
        assert torch.equal(q16, q4)
        for i in range(2):
            at = torch.arange(lens[i] - counts[i], lens[i])
            f, gain = R.frequencies(d, theta=1e6)
            src = qkv[starts[i]:starts[i + 1]].cpu()
            kr = R.rotate(src[:, h_q:h_q + h_kv], at, d, sd.SD_ROPE_HALF, f, gain)[0].to(BF)
            for w, x in enumerate((kr, src[:, h_q + h_kv:])):
                codes, param = R.quantise(x.transpose(0, 1))
                hist[i][w] = torch.cat([hist[i][w], R.values(R.pack(codes), param)], 1)
                parts[i][w].append((codes, param))
        if step == 0:
            continue
        queries = sd.Queries(q4, i32(starts), n, cap)
        out = sd.sd_kv4_verify_attention(queries, c4, dev_err=flag)
        view = R.Cache4.__new__(R.Cache4)
        view.h_kv, view.kv = h_kv, hist
        view.parts = [[tuple(torch.cat(y, 1) for y in zip(*p)) for p in s] for s in parts]
        for i in range(2):
            sl = slice(starts[i], starts[i + 1])
            ref, bound = R.attention_bound(q4[sl].cpu(), view, i, BF)
            assert ((out[sl].cpu().double() - ref).abs() <= bound).all(), (step, i)
        # the dense cache holds the same rows unquantised: half a step of either side apart
        dense = sd.sd_verify_attention(queries, c16)
        assert (dense.float() - out.float()).abs().max().item() < 0.5
        logits = out.float().flatten(1).contiguous()
        want = logits.argmax(1).view(2, n)
        draft = want[:, :n - 1].clone()
        draft[0, 1] += 1  # the first sequence keeps one token, the second all
        acc, tok = sd.sd_accept_greedy(logits, draft.flatten().int() % logits.shape[1],
                                       i32([n - 1, n - 1]), n - 1)
        assert acc.tolist() == [1, n - 1]
        assert tok[1].tolist() == want[1].tolist() and tok[0, 1].item() == want[0, 1].item()
        # the rejected rows are dropped: the next step writes over them
        for i, keep in enumerate((2, n)):
            drop = n - keep
            lens[i] -= drop
            hist[i] = [x[:, :lens[i]] for x in hist[i]]
            parts[i] = [[tuple(torch.cat(y, 1)[:, :lens[i]] for y in zip(*p))] for p in parts[i]]
    assert flag.item() == 0


def test_python_refusals():
    c = Call([30], [2], 4, 1, 64, False)
    kv = c.kv
    with pytest.raises(ValueError):
        sd.KV4Cache(kv.k.float(), kv.v, kv.k_param, kv.v_param, kv.kv_len)
    with pytest.raises(ValueError):
        sd.KV4Cache(kv.k, kv.v, kv.k_param.float(), kv.v_param, kv.kv_len)
    with pytest.raises(ValueError):
        sd.KV4Cache(kv.k, kv.v, kv.k_param, kv.v_param, kv.kv_len.long())
    with pytest.raises(ValueError):
        sd.KV4Cache(kv.k, kv.v, kv.k_param, kv.v_param, kv.kv_len, dtype=torch.float16)
    with pytest.raises(ValueError):  # not pages of 16
        sd.KV4Cache(kv.k, kv.v, kv.k_param, kv.v_param, kv.kv_len, i32([[0]]))
    with pytest.raises(ValueError):  # fp32 queries on a cache made for bf16 rows
        sd.sd_kv4_verify_attention(sd.Queries(c.queries.q.float(), i32([0, 2]), 2, 30), kv)
    with pytest.raises(ValueError):  # more positions than the cache holds
        sd.sd_kv4_verify_attention(sd.Queries(c.queries.q, i32([0, 2]), 2, 4000), kv)
    with pytest.raises(sd.SdError):
        sd.sd_kv4_verify_attention(c.queries, kv, workspace=torch.empty(
            0, dtype=torch.uint8, device="cuda")) if sd.sd_kv4_attention_workspace_size(
                c.queries, kv) else sd.sd_kv4_verify_attention(
                    sd.Queries(c.queries.q, i32([0, 2]), 0, 30), kv)
