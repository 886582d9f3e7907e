"""Cache appends on the GPU against 64-bit forms.

Tolerances: a rotated element is rounded once to its type (half a step, relative to itself) after
fp32 arithmetic on a sine and cosine whose argument, at most half a turn, is itself an fp32 number:
at most 2^-24 pi from the argument, 2^-23 from the function and three roundings of the products,
together below 2^-21 of |a| + |b|.  Everything 4-bit is exact: the definition leaves no freedom."""
import pytest
import torch

from speculative_decoding_attention_verify_b200 import sdattn as sd

from . import kv_ref as R

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


class Case:
    """Rows of a ragged batch and an empty cache with room for them."""

    def __init__(self, ctx, rows, h_q, h_kv, d, paged, dtype, seed=0, packed=True, pad_rows=0,
                 slack=0, kv4=False):
        g = torch.Generator().manual_seed(seed)
        self.ctx, self.n, self.h_q, self.h_kv, self.d, self.dtype = ctx, rows, h_q, h_kv, d, dtype
        self.paged, self.kv4 = paged, kv4
        total = sum(rows) + pad_rows
        width = (h_q + 2 * h_kv) * d + slack
        qkv = torch.randn(total, width, generator=g).to(dtype)
        self.qkv = qkv.cuda()
        part = lambda t, h0, h: t[:, h0 * d:(h0 + h) * d].unflatten(1, (h, d))  # noqa: E731
        cut = lambda t: (part(t, 0, h_q), part(t, h_q, h_kv), part(t, h_q + h_kv, h_kv))  # noqa: E731
        self.q, self.k, self.v = cut(qkv)
        self.dq, self.dk, self.dv = cut(self.qkv)
        if not packed:
            self.dq, self.dk, self.dv = (x.contiguous() for x in (self.dq, self.dk, self.dv))
        self.lens = [c + r for c, r in zip(ctx, rows)]
        starts = [0]
        for r in rows:
            starts.append(starts[-1] + r)
        self.starts, self.total = starts, total
        b, longest = len(rows), max(max(self.lens), 1)
        if paged:
            used = [-(-n // 16) for n in self.lens]
            self.table = torch.full((b, max(max(used), 1)), -1, dtype=torch.int32)
            order, at = torch.randperm(sum(used) + 2, generator=g), 0
            for i, u in enumerate(used):
                self.table[i, :u] = order[at:at + u].int()
                at += u
            shape = (sum(used) + 2, h_kv, 16)
        else:
            self.table, shape = None, (b, h_kv, longest + 3)
        self.shape = shape
        i32 = lambda x: torch.tensor(x, dtype=torch.int32).cuda()  # noqa: E731
        self.q_start, self.kv_len = i32(starts), i32(self.lens)
        if kv4:
            mk = lambda w, t, f: torch.full((*shape, w), f, dtype=t, device="cuda")  # noqa: E731
            self.cache = sd.KV4Cache(mk(d // 2, torch.uint8, 0xAB), mk(d // 2, torch.uint8, 0xAB),
                                     mk(2, BF, 7.0), mk(2, BF, 7.0), self.kv_len,
                                     self.table.cuda() if paged else None, dtype=dtype)
        else:
            mk = lambda: torch.full((*shape, d), 7.0, dtype=dtype, device="cuda")  # noqa: E731
            self.cache = sd.KVCache(mk(), mk(), self.kv_len,
                                    self.table.cuda() if paged else None)

    def new_rows(self, pos=None, q=True):
        return sd.NewRows(self.dk, self.dv, self.q_start, max(self.lens),
                          q=self.dq if q and self.h_q else None, pos=pos)

    def places(self):
        """(row, first index, third index) of every appended row."""
        for i, (c, n) in enumerate(zip(self.ctx, self.n)):
            for x in range(n):
                j = c + x
                yield (self.starts[i] + x, int(self.table[i, j // 16]), j % 16) if self.paged \
                    else (self.starts[i] + x, i, j)

    def positions(self):
        return torch.tensor([c + x for c, n in zip(self.ctx, self.n) for x in range(n)])


def check(c, rope_kw, rot, layout, pos=None):
    f, gain = R.frequencies(rot, **rope_kw) if rot else (None, 1.0)
    used = sum(c.n)
    at = c.positions() if pos is None else pos[:used].long()
    rope = sd.Rope(rot, layout=layout, **rope_kw) if rot else None
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = c.new_rows(pos=None if pos is None else pos.int().cuda())
    kw = {}
    if c.h_q:
        kw["q_out"] = torch.full((c.total, c.h_q, c.d), 9.0, dtype=c.dtype, device="cuda")
    if c.kv4:
        kw["k_out"], kw["v_out"] = (torch.full((c.total, c.h_kv, c.d), 9.0, dtype=c.dtype,
                                               device="cuda") for _ in range(2))
    call = sd.sd_kv4_append if c.kv4 else sd.sd_kv_append
    q_out = call(rope, rows, c.cache, dev_err=flag, **kw)
    torch.cuda.synchronize()
    assert flag.item() == 0
    half = R.HALF_STEP[c.dtype]
    turned, size = R.rotate(c.k[:used], at, rot, layout, f, gain)
    if c.h_q:
        ref, sq = R.rotate(c.q[:used], at, rot, layout, f, gain)
        got = q_out.cpu()
        err = (got[:used].double() - ref).abs()
        assert (err <= half * ref.abs() + 2.0 ** -21 * sq).all()
        assert (got[used:] == 9).all()  # rows behind the last sequence
    seen = torch.zeros(c.shape[0], c.shape[2], dtype=torch.bool)
    idx = list(c.places())
    r, a, j = (torch.tensor(x) for x in zip(*idx))
    seen[a, j] = True
    if not c.kv4:
        k, v = c.cache.k.cpu(), c.cache.v.cpu()
        err = (k[a, :, j].double() - turned[r]).abs()
        assert (err <= half * turned[r].abs() + 2.0 ** -21 * size[r]).all()
        assert torch.equal(v[a, :, j], c.v[r])
        for t in (k, v):
            assert (t.transpose(1, 2)[~seen] == 7).all()
        return
    for w, x in ((0, turned.to(c.dtype)), (1, c.v[:used])):
        codes, param = R.quantise(x)
        gc = (c.cache.k, c.cache.v)[w].cpu()
        gp = (c.cache.k_param, c.cache.v_param)[w].cpu()
        assert torch.equal(gp[a, :, j].view(torch.int16), param[r].view(torch.int16))
        assert torch.equal(gc[a, :, j], R.pack(codes)[r])
        assert (gc.transpose(1, 2)[~seen] == 0xAB).all()
        assert (gp.transpose(1, 2)[~seen] == 7).all()
        val = (kw["k_out"], kw["v_out"])[w].cpu()
        want = (param[..., 1:].float() + param[..., :1].float() * codes.float()).to(c.dtype)
        assert torch.equal(val[:used], want)
        assert (val[used:] == 9).all()


HEADS = [(28, 4, 128), (4, 1, 64), (16, 16, 64), (3, 3, 128), (0, 2, 128)]


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("heads", HEADS)
def test_ragged_batches(heads, paged, dtype, kv4):
    h_q, h_kv, d = heads
    c = Case([0, 37, 15, 200, 16], [1, 5, 0, 33, 16], h_q, h_kv, d, paged, dtype, seed=d + h_q,
             pad_rows=3, kv4=kv4)
    check(c, dict(theta=1e6), d, sd.SD_ROPE_HALF)


ROPES = [(128, {}), (64, dict(scaling=sd.SD_ROPE_LINEAR, factor=8.0)), (2, dict(gain=1.5)),
         (34, dict(scaling=sd.SD_ROPE_NTK, factor=4.0)), (126, dict(theta=5e5)), (0, {}),
         (128, dict(scaling=sd.SD_ROPE_YARN, factor=4.0, original_len=32768, theta=1e6)),
         (48, dict(scaling=sd.SD_ROPE_YARN, factor=16.0, original_len=64, theta=1e4)),
         (6, dict(inv_freq=[1.0, 0.25, 0.0]))]


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", [sd.SD_ROPE_HALF, sd.SD_ROPE_INTERLEAVED])
@pytest.mark.parametrize("rot,kw", ROPES)
def test_rotations(rot, kw, layout, dtype, kv4):
    c = Case([3, 900], [7, 2], 6, 2, 128, True, dtype, seed=rot, kv4=kv4)
    check(c, kw, rot, layout)


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_far_and_negative_positions(dtype, kv4):
    c = Case([10], [6], 4, 2, 128, False, dtype, kv4=kv4)
    pos = torch.tensor([0, -5, 10**6, 2**24 + 1, 2**31 - 1, -2**31])
    check(c, dict(theta=10000.0), 128, sd.SD_ROPE_HALF, pos=pos)


@pytest.mark.parametrize("kv4", [False, True])
@pytest.mark.parametrize("layout", [sd.SD_ROPE_HALF, sd.SD_ROPE_INTERLEAVED])
@pytest.mark.parametrize("slack,packed", [(0, False), (8, True), (3, True), (1, True)])
def test_row_strides_and_alignments(slack, packed, layout, kv4):
    """Separate tensors, and slices of wider rows whose stride does or does not allow 16-byte
    access."""
    c = Case([20, 5], [9, 4], 4, 2, 64, True, BF, slack=slack, packed=packed, kv4=kv4)
    check(c, {}, 64, layout)


@pytest.mark.parametrize("kv4", [False, True])
def test_many_rows(kv4):
    """Several rows per block, blocks that meet several sequences."""
    c = Case([0, 100, 7, 0], [701, 3, 611, 2], 4, 2, 128, True, BF, kv4=kv4)
    check(c, dict(theta=1e6), 64, sd.SD_ROPE_HALF)


@pytest.mark.parametrize("batch", [33, 1100])
def test_many_sequences(batch):
    """More sequences than one round of the search sees, some without rows."""
    rows = [(i * 7) % 3 for i in range(batch)]
    c = Case([i % 40 for i in range(batch)], rows, 2, 1, 64, False, BF)
    check(c, {}, 64, sd.SD_ROPE_HALF)


def test_queries_rotated_in_place():
    c = Case([11], [5], 8, 2, 128, False, BF, packed=False)
    keep = c.q.clone()
    rows = c.new_rows()
    out = sd.sd_kv_append(sd.Rope(128), rows, c.cache, q_out=c.dq)
    f, gain = R.frequencies(128)
    ref, size = R.rotate(keep, c.positions(), 128, sd.SD_ROPE_HALF, f, gain)
    assert out.data_ptr() == c.dq.data_ptr()
    assert ((out.cpu().double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -21 * size).all()


@pytest.mark.parametrize("wide", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_special_rows_in_4_bits(dtype, wide):
    """Constant rows, rows with infinities or NaN, the type's extremes, tiny and exact-tie rows."""
    d = 64
    big = float(torch.finfo(dtype).max)
    rows = torch.zeros(12, 1, d + (0 if wide else 1), dtype=torch.float64)
    rows[0] = 0.0
    rows[1] = 3.7
    rows[2, 0, 5] = float("inf")
    rows[3, 0, 63] = float("-inf")
    rows[4, 0, 0] = float("nan")
    rows[5, 0, :32], rows[5, 0, 32:] = -big, big     # the range overflows
    rows[6] = torch.arange(rows.shape[2]) % 31 * 0.5  # quotients that end in a half: ties
    rows[7, 0, 3] = 1e-39                            # a range below the smallest normal number
    rows[8] = -100.0
    rows[8, 0, 9] = -99.0
    rows[9, 0, 1] = big / 4
    rows[10] = torch.randn(rows.shape[2], generator=torch.Generator().manual_seed(1)) * 1e-30
    rows[11] = torch.linspace(-1, 1, rows.shape[2])
    x = rows.to(dtype)
    x = x[..., :d].contiguous() if wide else x
    dx = x.cuda()[..., :d]
    k = x[..., :d]
    cache = sd.KV4Cache.empty(1, 1, 16, d, torch.tensor([12], dtype=torch.int32, device="cuda"), dtype)
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    sd.sd_kv4_append(None, sd.NewRows(dx, dx, torch.tensor([0, 12], dtype=torch.int32).cuda(), 16),
                     cache, dev_err=flag)
    codes, param = R.quantise(k[:, 0])
    assert flag.item() == sd.SD_DEVERR_NUMERIC
    for got, gp in ((cache.k, cache.k_param), (cache.v, cache.v_param)):
        a, b = gp.cpu()[0, 0, :12], param
        assert torch.equal(a.isnan(), b.isnan())
        assert torch.equal(a.nan_to_num(7.0), b.nan_to_num(7.0))
        assert torch.equal(got.cpu()[0, 0, :12], R.pack(codes))
    assert param[:6].isnan().any(-1).tolist() == [False, False, True, True, True, True]


@pytest.mark.parametrize("kv4", [False, True])
def test_violated_hints_and_pages_are_skipped(kv4):
    call = sd.sd_kv4_append if kv4 else sd.sd_kv_append
    for what in ("short", "long", "page", "table"):
        c = Case([30, 20, 40], [4, 4, 4], 4, 2, 64, True, BF, kv4=kv4)
        lens, table = list(c.lens), c.table.clone()
        if what == "short":
            lens[1] = 3                      # fewer positions than rows
        elif what == "long":
            lens[1] = max(c.lens) + 1        # beyond max_kv_len
        elif what == "page":
            table[1, 1] = c.shape[0]         # rows 20..23 are on page 1
        else:
            lens[1] = 16 * table.shape[1] + 4
        c.cache.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        c.cache.block_table.copy_(table)
        flag = torch.zeros(1, dtype=torch.int32, device="cuda")
        q_out = torch.full((12, 4, 64), 9.0, dtype=BF, device="cuda")
        rows = sd.NewRows(c.dk, c.dv, c.q_start,
                          4096 if what == "table" else max(c.lens), q=c.dq)
        call(sd.Rope(64), rows, c.cache, q_out=q_out, dev_err=flag)
        want = sd.SD_DEVERR_PAGE if what == "page" else sd.SD_DEVERR_SHAPE
        assert flag.item() == want, what
        k = (c.cache.k_param if kv4 else c.cache.k).cpu()
        touched = {(a, j) for r, a, j in c.places() if (k[a, :, j] != 7).any()}
        assert touched == {(a, j) for r, a, j in c.places() if not 4 <= r < 8}, what
        assert (k.transpose(1, 2) != 7).any(-1).any(-1).sum() == 8
        q = q_out.cpu()
        assert (q[4:8] == 9).all() == (what != "page") and (q[:4] != 9).any() and (q[8:] != 9).any()


def test_rows_beyond_the_tensor_are_refused_on_the_device():
    """q_start that points past n_rows: the sequence is skipped, nothing is read out of range."""
    c = Case([30, 20], [4, 4], 4, 2, 64, False, BF)
    c.q_start.copy_(torch.tensor([0, 4, 4000], dtype=torch.int32))
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    sd.sd_kv_append(None, c.new_rows(), c.cache, dev_err=flag)
    assert flag.item() == sd.SD_DEVERR_SHAPE
    assert (c.cache.k[1] == 7).all()


@pytest.mark.parametrize("kv4", [False, True])
def test_offsets_beyond_32_bits(kv4):
    """Pages whose rows lie past 2^32 bytes (and 2^31 elements) of the pool."""
    h_kv, d = 8, 128
    per_page = h_kv * 16 * (d // 2 if kv4 else d)
    pages = (2 ** 32 // per_page) + 7 if kv4 else (2 ** 31 // per_page) + 7
    lens = torch.tensor([20], dtype=torch.int32, device="cuda")
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(20, h_kv, d, generator=g).to(BF) for _ in range(2))
    rows = sd.NewRows(k.cuda(), v.cuda(), torch.tensor([0, 20], dtype=torch.int32).cuda(), 20)
    new = lambda w, t: torch.zeros((pages, h_kv, 16, w), dtype=t, device="cuda")  # noqa: E731
    if kv4:
        cache = sd.KV4Cache(new(64, torch.uint8), new(64, torch.uint8), new(2, BF), new(2, BF), lens,
                            table)
        sd.sd_kv4_append(None, rows, cache)
        codes, param = R.quantise(v)
        assert torch.equal(cache.v[pages - 1].cpu(), R.pack(codes)[:16].transpose(0, 1))
        assert torch.equal(cache.v[pages - 3, :, :4].cpu(), R.pack(codes)[16:].transpose(0, 1))
        assert torch.equal(cache.v_param[pages - 3, :, :4].cpu(), param[16:].transpose(0, 1))
    else:
        cache = sd.KVCache(new(d, BF), new(d, BF), lens, table)
        sd.sd_kv_append(None, rows, cache)
        assert torch.equal(cache.v[pages - 1].cpu(), v[:16].transpose(0, 1))
        assert torch.equal(cache.k[pages - 3, :, :4].cpu(), k[16:].transpose(0, 1))
    assert not cache.v[:pages - 3].any()


@pytest.mark.parametrize("kv4", [False, True])
def test_captured_and_replayed_with_new_rows(kv4):
    """A graph replayed after rows, lengths and positions changed in place."""
    c = Case([0, 40], [3, 2], 4, 2, 64, True, BF, kv4=kv4)
    call = sd.sd_kv4_append if kv4 else sd.sd_kv_append
    rows, rope = c.new_rows(), sd.Rope(64)
    q_out = torch.empty(5, 4, 64, dtype=BF, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call(rope, rows, c.cache, q_out=q_out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(rope, rows, c.cache, q_out=q_out)
    c.qkv.copy_(torch.randn_like(c.qkv, dtype=F32).to(BF))
    c.kv_len.copy_(torch.tensor([2 + 3, 36 + 2], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in ((c.cache.k, c.cache.k_param, c.cache.v) if kv4
                               else (c.cache.k, c.cache.v))] + [q_out.clone()]
    call(rope, rows, c.cache, q_out=q_out)
    torch.cuda.synchronize()
    for a, b in zip(got, ((c.cache.k, c.cache.k_param, c.cache.v) if kv4
                          else (c.cache.k, c.cache.v)) + (q_out,)):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_python_refusals():
    c = Case([10], [4], 4, 2, 64, False, BF)
    k = c.dk.contiguous()
    i32 = c.q_start
    with pytest.raises(ValueError):
        sd.NewRows(k, k[:2], i32, 20)
    with pytest.raises(ValueError):
        sd.NewRows(k, k.float(), i32, 20)
    with pytest.raises(ValueError):
        sd.NewRows(k, k, i32.long(), 20)
    with pytest.raises(ValueError):
        sd.NewRows(k.cpu(), k.cpu(), i32.cpu(), 20)
    with pytest.raises(ValueError):
        sd.NewRows(k[..., ::2], k[..., ::2], i32, 20)
    with pytest.raises(ValueError):
        sd.NewRows(k, k, i32, 20, pos=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):  # more positions than the cache holds
        sd.sd_kv_append(None, sd.NewRows(k, k, i32, 4000), c.cache)
    with pytest.raises(ValueError):  # another dtype
        sd.sd_kv_append(None, sd.NewRows(k.float(), k.float(), i32, 14), c.cache)
    with pytest.raises(ValueError):  # an output of another shape
        sd.sd_kv_append(None, c.new_rows(), c.cache, q_out=k)
    with pytest.raises(ValueError):
        sd.Rope(64, inv_freq=[1.0, 2.0])
    with pytest.raises(sd.SdError):
        sd.sd_kv_append(sd.Rope(66), c.new_rows(), c.cache)
