"""Cases of the key/value cache operators: appending rotated rows to a cache, appending them in 4
bits, and attending over a cache held in 4 bits.

Each case is one call.  ``run`` computes it from elementary torch operations where ``own`` is
false, and through the library's calls where it is true; ``exact`` computes it in 64 bits from the
definition.

The operators, for sequence b with rows q_start[b] .. q_start[b+1] (n of them, the last n
positions of its cache, so row i is position kv_len[b] - n + i):

* rotation: pair m of a head's first ``rotary`` channels turns by angle = position * f_m, the
  cosine and the sine both multiplied by ``gain``.  The pairs are (m, m + rotary/2) in the half
  layout and (2m, 2m+1) in the interleaved one; channels from ``rotary`` on pass.
  f_m = theta^(-2m/rotary), scaled for longer contexts: linear f_m / factor; ntk
  theta' = theta * factor^(rotary/(rotary-2)); yarn f_m * (1 - t_m + t_m / factor) with t_m rising
  from 0 to 1 between the pairs that turn 32 times and once in the original length.
* 4 bits: a row x of d channels is kept as lo = bf16(min x), s = bf16((max x - lo) / 15) and codes
  c = min(15, max(0, round((x - lo) / s))), ties to even; it stands for lo + s * c.
* attention: row i sees positions j <= kv_len[b] - n + i; o = softmax(q . k_j / sqrt(d)) . v_j.
"""
import math
import random

import torch

own = False

PAGE = 16
THETA = 1000000.0
ORIGINAL = 32768  # the length that the yarn scaling starts from

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------- cases ----

def _attend(name, batch, h_q, h_kv, d, rows, length, paged=False, ragged=0, dtype="bf16"):
    return {"name": name, "op": "attend4", "batch": batch, "h_q": h_q, "h_kv": h_kv, "d": d,
            "rows": rows, "length": length, "paged": paged, "ragged": ragged, "dtype": dtype}


def _append(name, op, batch, h_q, h_kv, d, rows, length, paged=False, ragged=0, dtype="bf16",
            layout="half", rotary=0, scaling="none"):
    return {"name": name, "op": op, "batch": batch, "h_q": h_q, "h_kv": h_kv, "d": d,
            "rows": rows, "length": length, "paged": paged, "ragged": ragged, "dtype": dtype,
            "layout": layout, "rotary": rotary or d, "scaling": scaling}


def listed():
    return [
        # one new token of one sequence after a prompt of half a thousand: latency alone
        _append("append-token", "append", 1, 28, 4, 128, 1, 520),
        # a verify step's rows of 28 layers, contiguous caches
        _append("append-verify-28", "append", 28, 28, 4, 128, 9, 1033, scaling="yarn"),
        # a long prompt of 8 sequences of different lengths into pages, part of the head rotated
        _append("append-prompt-pages", "append", 8, 28, 4, 128, 4096, 34816, paged=True, ragged=3,
                layout="interleaved", rotary=64, scaling="linear"),
        # the same three uses with the cache in 4 bits
        _append("append4-token", "append4", 1, 28, 4, 128, 1, 520),
        _append("append4-verify-pages", "append4", 8, 28, 4, 128, 8, 34816, paged=True, ragged=5,
                scaling="yarn"),
        _append("append4-prompt", "append4", 1, 28, 4, 128, 26024, 26024, scaling="ntk"),
        # a short context with small heads
        _attend("attend4-short", 1, 4, 1, 64, 5, 325),
        # one layer's verify step
        _attend("attend4-layer", 1, 28, 4, 128, 6, 8710),
        # plain decoding over a long video, 28 layers
        _attend("attend4-decode-28", 28, 28, 4, 128, 1, 26025),
        # its verify step of 9 rows
        _attend("attend4-verify-28", 28, 28, 4, 128, 9, 26033),
        # 8 sequences of different lengths and rows, in pages
        _attend("attend4-pages", 8, 28, 4, 128, 8, 34823, paged=True, ragged=7),
        # a single long sequence: one token over 140,000 positions
        _attend("attend4-140k", 1, 28, 4, 128, 1, 140001),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append4", "attend4"])
    h_q, h_kv, d = rng.choice([(28, 4, 128), (4, 1, 64), (32, 8, 128), (16, 16, 64), (12, 2, 128),
                               (8, 1, 128)])
    paged = rng.random() < 0.5
    dtype = "f32" if rng.random() < 0.15 else "bf16"
    ragged = rng.randrange(1, 1000) if rng.random() < 0.5 else 0
    if op == "attend4":
        # no more bytes or products than the largest listed case
        batch, rows = rng.choice([1, 2, 3, 5, 8, 28]), rng.choice([1, 1, 2, 4, 6, 9, 13])
        most = min(140001, int(3.9e8) // (batch * h_kv * (d + 8)),
                   int(9e10) // (batch * rows * h_q * d * 4))
        if dtype == "f32":
            most = min(most, 40000 // batch)
        case = _attend("", batch, h_q, h_kv, d, rows, max(rows, _spread(rng, 40, most)), paged,
                       ragged, dtype)
    else:
        batch = rng.choice([1, 2, 3, 5, 8, 28])
        width = 2 * (h_q + 2 * h_kv) * d * (4 if dtype == "f32" else 2)
        rows = _spread(rng, 1, min(26024, int(3.9e8) // width) // batch)
        length = rows + (_spread(rng, 1, 100000) if paged else _spread(rng, 1, 1500))
        rotary = rng.choice([d, d, d // 2, d // 4, 2 * rng.randrange(2, d // 2)])
        case = _append("", op, batch, h_q, h_kv, d, rows, length, paged, ragged, dtype,
                       rng.choice(["half", "interleaved"]), rotary,
                       rng.choice(["none", "linear", "ntk", "yarn"]))
    del case["name"]
    return case


def _lengths(case):
    """(rows, cache length) of every sequence: the case's own, or spread below them."""
    if not case["ragged"]:
        return [(case["rows"], case["length"])] * case["batch"]
    rng = random.Random(case["ragged"])
    got = []
    for b in range(case["batch"]):
        n = case["rows"] if b == 0 else rng.randint(max(1, case["rows"] // 4), case["rows"])
        got.append((n, max(n, case["length"] if b == 0
                           else rng.randint(max(1, case["length"] // 8), case["length"]))))
    rng.shuffle(got)
    return got


def _rope(case):
    """The rotation's frequencies in 64 bits, and the factor of its cosine and sine."""
    r, kind = case["rotary"], case["scaling"]
    factor = 1.0 if kind == "none" else 4.0
    theta = THETA * factor ** (r / (r - 2.0)) if kind == "ntk" else THETA
    f = [theta ** (-2.0 * m / r) for m in range(r // 2)]
    if kind == "linear":
        f = [x / factor for x in f]
    if kind != "yarn":
        return f, 1.0
    at = lambda turns: r * math.log(ORIGINAL / (turns * 2 * math.pi)) / (2 * math.log(THETA))  # noqa: E731
    lo, hi = max(math.floor(at(32.0)), 0.0), min(math.ceil(at(1.0)), r - 1.0)
    hi = hi if hi > lo else lo + 0.001
    t = [min(1.0, max(0.0, (m - lo) / (hi - lo))) for m in range(r // 2)]
    return [x * (1 - y) + x * y / factor for x, y in zip(f, t)], 0.1 * math.log(factor) + 1.0


# ------------------------------------------------------------------------------ inputs ----

def _quantise(x):
    """(codes, scale, low) of the rows of x.  The differences and quotients are in 64 bits: values
    next to a border decide which code or scale they round to."""
    lo = x.float().amin(-1, keepdim=True).bfloat16()
    s = ((x.double().amax(-1, keepdim=True) - lo.double()) / 15).clamp_min(0).float().bfloat16()
    c = ((x.double() - lo.double()) / torch.where(s > 0, s, torch.ones_like(s)).double()).round()
    c = torch.where(s > 0, c, torch.zeros_like(c)).clamp(0, 15)
    return c.to(torch.uint8), s.float(), lo.float()


def _pack(codes):
    """Two channels a byte, the even one in the low half."""
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 11)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    t = TYPES[case["dtype"]]
    b, h_q, h_kv, d = case["batch"], case["h_q"], case["h_kv"], case["d"]
    sizes = _lengths(case)
    starts = [0]
    for n, _ in sizes:
        starts.append(starts[-1] + n)
    total = starts[-1]
    longest = max(n for _, n in sizes)
    st = {"case": case, "q_start": ints(starts), "kv_len": ints([n for _, n in sizes]),
          "rows": max(n for n, _ in sizes), "longest": longest, "total": total}
    if case["op"] != "attend4":
        # one projection's output holds the rows' queries, keys and values side by side
        qkv = normal(total, h_q + 2 * h_kv, d)
        qkv[:, h_q:h_q + h_kv] *= 1 + 3 * (torch.rand(d, generator=g, device="cuda") < 0.05)
        qkv = qkv.to(t)
        st |= {"q": qkv[:, :h_q], "k": qkv[:, h_q:h_q + h_kv], "v": qkv[:, h_q + h_kv:],
               "rope": _rope(case)}
    else:
        st["q"] = normal(total, h_q, d).to(t)
    # the cache: contiguous with spare room, or pages in random order of which an append needs
    # those that its rows fall into
    if case["paged"]:
        table = torch.full((b, -(-longest // PAGE)), -1, dtype=torch.int64)
        first = [0 if case["op"] == "attend4" else (n - r) // PAGE for r, n in sizes]
        used = [-(-n // PAGE) - f for f, (_, n) in zip(first, sizes)]
        pages = sum(used) + 2
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))
        at = 0
        for i in range(b):
            table[i, first[i]:first[i] + used[i]] = order[at:at + used[i]]
            at += used[i]
        st["table"] = table.to(torch.int32).cuda()
        shape = (pages, h_kv, PAGE)
    else:
        shape = (b, h_kv, -(-(longest + 7) // 8) * 8)
    if case["op"] == "append":
        st["k_cache"] = torch.zeros(*shape, d, dtype=t, device="cuda")
        st["v_cache"] = torch.zeros(*shape, d, dtype=t, device="cuda")
    elif case["op"] == "append4":
        for n in ("k", "v"):
            st[n + "_codes"] = torch.zeros(*shape, d // 2, dtype=torch.uint8, device="cuda")
            st[n + "_param"] = torch.zeros(*shape, 2, dtype=torch.bfloat16, device="cuda")
    else:
        # a filled cache; about 1% of the keys point where the queries do
        for n in ("k", "v"):
            codes = torch.empty(*shape, d // 2, dtype=torch.uint8, device="cuda")
            param = torch.empty(*shape, 2, dtype=torch.bfloat16, device="cuda")
            step = 8192 if case["paged"] else 4
            for i in range(0, shape[0], step):
                part = slice(i, min(shape[0], i + step))
                x = normal(part.stop - part.start, *shape[1:], d)
                if n == "k":
                    to = st["q"][-1].float().view(h_kv, -1, d).mean(1)
                    hit = torch.rand(x.shape[:3], generator=g, device="cuda") < 0.01
                    x = torch.where(hit[..., None], 4 * to[None, :, None], x)
                c, s, lo = _quantise(x.to(torch.bfloat16))
                codes[part], param[part] = _pack(c), torch.cat([s, lo], -1).bfloat16()
            st[n + "_codes"], st[n + "_param"] = codes, param
        # what lies behind a sequence's end was never written: it may hold anything
        j = torch.arange(shape[2], device="cuda")
        if case["paged"]:
            at = torch.zeros(shape[0], dtype=torch.int64, device="cuda")
            for i, (_, n) in enumerate(sizes):
                at[st["table"][i, :-(-n // PAGE)].long()] = \
                    (n - PAGE * torch.arange(-(-n // PAGE), device="cuda")).clamp(max=PAGE)
            free = j[None] >= at[:, None]
        else:
            free = j[None] >= st["kv_len"][:, None]
        free = free[:, None, :, None].expand(*shape, 2)
        for n in ("k", "v"):
            st[n + "_param"][free] = float("nan")
    return st


# -------------------------------------------------------------------------- plain form ----

def _positions(st):
    """Sequence and cache position of every row."""
    rows = torch.arange(st["total"], device="cuda")
    seq = torch.searchsorted(st["q_start"][1:].long(), rows, right=True)
    return seq, (st["kv_len"][seq] - st["q_start"][seq + 1]).long() + rows


def _turn(x, pos, case, rope):
    """x [rows][heads][d] rotated, in the precision of x."""
    f, gain = rope
    r = case["rotary"]
    angle = pos.double()[:, None] * torch.tensor(f, dtype=torch.float64, device="cuda")
    c, s = (gain * angle.cos()).to(x.dtype)[:, None], (gain * angle.sin()).to(x.dtype)[:, None]
    if case["layout"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat([a * c - b * s, b * c + a * s], -1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    return torch.cat([y, x[..., r:]], -1)


def _slots(st, seq, pos):
    """First and third index of the rows' places in the cache."""
    if "table" in st:
        return st["table"][seq, pos // PAGE].long(), pos % PAGE
    return seq, pos


def _plain(st):
    case = st["case"]
    t = TYPES[case["dtype"]]
    if case["op"] == "attend4":
        return _plain_attention(st)
    seq, pos = _positions(st)
    q_out = _turn(st["q"].float(), pos, case, st["rope"]).to(t)
    a, j = _slots(st, seq, pos)
    if case["op"] == "append":
        st["k_cache"][a, :, j] = _turn(st["k"].float(), pos, case, st["rope"]).to(t)
        st["v_cache"][a, :, j] = st["v"]
        return {"q": q_out, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    # (64 bits: the rounded keys decide the codes)
    got = {"q": q_out}
    for n, x in (("k", _turn(st["k"].double(), pos, case, st["rope"]).to(t)), ("v", st["v"])):
        c, s, lo = _quantise(x)
        st[n + "_codes"][a, :, j] = _pack(c)
        st[n + "_param"][a, :, j] = torch.cat([s, lo], -1).bfloat16()
        got[n] = (lo + s * c.float()).to(t)
        got[n + "_param"] = st[n + "_param"]
    return got


def _plain_attention(st):
    case = st["case"]
    b, h_q, h_kv, d = case["batch"], case["h_q"], case["h_kv"], case["d"]
    n, m = st["longest"], st["rows"]
    j = torch.arange(n, device="cuda")
    used = j[None] < st["kv_len"][:, None]

    def values(name):
        codes, param = st[name + "_codes"], st[name + "_param"]
        if case["paged"]:
            at = st["table"].long().clamp_min(0)
            codes = codes[at].transpose(1, 2).flatten(2, 3)
            param = param[at].transpose(1, 2).flatten(2, 3)
        codes, param = codes[:, :, :n], param[:, :, :n].float()
        x = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
        x = param[..., 1:] + param[..., :1] * x
        return torch.where(used[:, None, :, None], x, torch.zeros((), device="cuda"))

    i = torch.arange(m, device="cuda")
    count = (st["q_start"][1:] - st["q_start"][:-1]).long()
    at = (st["q_start"][:-1, None].long() + i).clamp(max=st["total"] - 1)
    q = st["q"].float()[at].view(b, m, h_kv, h_q // h_kv, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    s = q @ values("k").transpose(2, 3)
    s *= 1 / math.sqrt(d)
    sees = j[None, None] <= (st["kv_len"].long() - count)[:, None, None] + i[None, :, None]
    s = s.view(b, h_kv, h_q // h_kv, m, n).masked_fill_(~(sees & used[:, None])[:, None, None],
                                                        float("-inf"))
    s -= s.amax(-1, keepdim=True)
    p = s.exp_()
    o = p.flatten(2, 3) @ values("v")
    o = o.view(b, h_kv, h_q // h_kv, m, d) / p.sum(-1, keepdim=True)
    o = o.permute(0, 3, 1, 2, 4).reshape(b, m, h_q, d)
    return o[i[None] < count[:, None]].to(TYPES[case["dtype"]])


# ------------------------------------------------------------------------ library form ----

def _handles(st):
    """What a program keeps beside its tensors: descriptors, workspace and output buffers."""
    from speculative_decoding_attention_verify_b200 import sdattn as sd
    case = st["case"]
    h = {"sd": sd}
    if case["op"] == "append":
        h["cache"] = sd.KVCache(st["k_cache"], st["v_cache"], st["kv_len"], st.get("table"))
    else:
        h["cache"] = sd.KV4Cache(st["k_codes"], st["v_codes"], st["k_param"], st["v_param"],
                                 st["kv_len"], st.get("table"), dtype=TYPES[case["dtype"]])
    if case["op"] == "attend4":
        h["q"] = sd.Queries(st["q"], st["q_start"], st["rows"], st["longest"])
        n = sd.sd_kv4_attention_workspace_size(h["q"], h["cache"])
        h["workspace"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
        h["out"] = torch.empty_like(st["q"])
        return h
    kind = {"none": sd.SD_ROPE_UNSCALED, "linear": sd.SD_ROPE_LINEAR, "ntk": sd.SD_ROPE_NTK,
            "yarn": sd.SD_ROPE_YARN}[case["scaling"]]
    h["rope"] = sd.Rope(case["rotary"], theta=THETA, scaling=kind,
                        layout=sd.SD_ROPE_HALF if case["layout"] == "half"
                        else sd.SD_ROPE_INTERLEAVED,
                        factor=1.0 if case["scaling"] == "none" else 4.0, original_len=ORIGINAL)
    h["rows"] = sd.NewRows(st["k"], st["v"], st["q_start"], st["longest"], q=st["q"])
    h["q_out"] = torch.empty(st["q"].shape, dtype=st["q"].dtype, device="cuda")
    if case["op"] == "append4":
        h["k_out"], h["v_out"] = (torch.empty(st["k"].shape, dtype=st["k"].dtype, device="cuda")
                                  for _ in range(2))
    return h


def _call(st):
    if "handles" not in st:
        st["handles"] = _handles(st)
    h, op = st["handles"], st["case"]["op"]
    sd = h["sd"]
    if op == "attend4":
        return sd.sd_kv4_verify_attention(h["q"], h["cache"], out=h["out"],
                                          workspace=h["workspace"])
    if op == "append":
        q = sd.sd_kv_append(h["rope"], h["rows"], h["cache"], q_out=h["q_out"])
        return {"q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    q = sd.sd_kv4_append(h["rope"], h["rows"], h["cache"], q_out=h["q_out"], k_out=h["k_out"],
                         v_out=h["v_out"])
    return {"q": q, "k": h["k_out"], "v": h["v_out"], "k_param": st["k_param"],
            "v_param": st["v_param"]}


def run(state):
    if own:
        return _call(state)
    return _plain(state)


def work(case):
    sizes = _lengths(case)
    e = 2 if case["dtype"] == "bf16" else 4
    rows, d, h_q, h_kv = sum(n for n, _ in sizes), case["d"], case["h_q"], case["h_kv"]
    row4 = d // 2 + 4
    if case["op"] == "attend4":
        seen = sum(sum(n - r + i + 1 for i in range(r)) for r, n in sizes)
        return {"bytes": 2 * rows * h_q * d * e + sum(n for _, n in sizes) * h_kv * 2 * row4,
                "flops": 4 * h_q * d * seen}
    turns = 3 * rows * case["rotary"] * (h_q + h_kv)
    if case["op"] == "append":
        return {"bytes": 2 * rows * (h_q + 2 * h_kv) * d * e, "flops": turns}
    return {"bytes": 2 * rows * (h_q + 2 * h_kv) * d * e + rows * h_kv * 2 * row4,
            "flops": turns + 8 * rows * h_kv * d}


# ------------------------------------------------------------------------------- exact ----

def exact(case, seed):
    st = prepare(case, seed)
    sizes = _lengths(case)
    d, h_q, h_kv = case["d"], case["h_q"], case["h_kv"]
    if case["op"] == "attend4":
        out = torch.empty(st["total"], h_q, d, dtype=torch.float64, device="cuda")
        at = 0
        for i, (r, n) in enumerate(sizes):
            kv = []
            for name in ("k", "v"):
                if case["paged"]:
                    ids = st["table"][i, :-(-n // PAGE)].long()
                    c = st[name + "_codes"][ids].permute(1, 0, 2, 3).reshape(h_kv, -1, d // 2)[:, :n]
                    p = st[name + "_param"][ids].permute(1, 0, 2, 3).reshape(h_kv, -1, 2)[:, :n]
                else:
                    c, p = st[name + "_codes"][i, :, :n], st[name + "_param"][i, :, :n]
                x = torch.empty(h_kv, n, d, dtype=torch.float64, device="cuda")
                x[..., 0::2], x[..., 1::2] = (c % 16).double(), (c // 16).double()
                kv.append(x.mul_(p[..., 0:1].double()).add_(p[..., 1:2].double()))
            limit = torch.arange(n - r, n, device="cuda")[:, None]
            hide = torch.arange(n, device="cuda")[None] > limit
            for h in range(h_q):
                k, v = kv[0][h // (h_q // h_kv)], kv[1][h // (h_q // h_kv)]
                s = (st["q"][at:at + r, h].double() @ k.T) / math.sqrt(d)
                out[at:at + r, h] = torch.softmax(s.masked_fill(hide, -math.inf), -1) @ v
            at += r
        return out
    f, gain = st["rope"]
    freq = torch.tensor(f, dtype=torch.float64, device="cuda")
    half, r2 = case["layout"] == "half", case["rotary"] // 2
    first = torch.arange(r2, device="cuda") * (1 if half else 2)
    second = first + (r2 if half else 1)

    def rotated(x, pos):
        y = x.double().clone()
        z = torch.polar(torch.full((1,), gain, dtype=torch.float64, device="cuda"),
                        pos.double()[:, None] * freq)
        w = torch.complex(x[..., first].double(), x[..., second].double()) * z[:, None]
        y[..., first], y[..., second] = w.real, w.imag
        return y

    pos = torch.cat([torch.arange(n - r, n, device="cuda") for r, n in sizes])
    seq = [i for i, (r, _) in enumerate(sizes) for _ in range(r)]
    if case["paged"]:
        table = st["table"].tolist()
        where = [(table[i][j // PAGE], j % PAGE) for i, j in zip(seq, pos.tolist())]
    else:
        where = list(zip(seq, pos.tolist()))
    a, j = (torch.tensor(x, device="cuda") for x in zip(*where))
    got = {"q": rotated(st["q"], pos)}
    if case["op"] == "append":
        for n, x in (("k", rotated(st["k"], pos)), ("v", st["v"].double())):
            got[n + "_cache"] = st[n + "_cache"].double()
            got[n + "_cache"][a, :, j] = x
        return got
    t = TYPES[case["dtype"]]
    for n, x in (("k", rotated(st["k"], pos).to(t).double()), ("v", st["v"].double())):
        top, lo = x.max(-1).values, x.min(-1).values.bfloat16().double()
        s = ((top - lo) / 15).clamp(min=0).float().bfloat16().double()
        c = ((x - lo[..., None]) / s[..., None]).round().clamp(0, 15)
        got[n] = lo[..., None] + s[..., None] * torch.where(s[..., None] > 0, c, 0.0)
        got[n + "_param"] = st[n + "_param"].double()
        got[n + "_param"][a, :, j] = torch.stack([s, lo], -1)
    return got
