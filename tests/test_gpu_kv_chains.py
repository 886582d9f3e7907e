"""Appends and attention enqueued far ahead of the GPU, so that each kernel may be resident before
the one whose rows it reads has run: the same bits as with a pause after every call."""
import pytest
import torch

from speculative_decoding_attention_verify_b200 import sdattn as sd

from .test_gpu_kv4_attention import BF, i32

pytestmark = pytest.mark.gpu
STEPS = 60


@pytest.mark.parametrize("kv4", [True, False])
@pytest.mark.parametrize("heads,rows,lens", [((4, 1, 64), 1, [[325]]), ((4, 1, 64), 5, [[325]]),
                                             ((28, 4, 128), 1, [[3000, 50], [60, 2500]]),
                                             ((28, 4, 128), 1, [[3000, 700]]),
                                             ((28, 4, 128), 9, [[700]])])
def test_calls_that_follow_at_once(heads, rows, lens, kv4):
    """One buffer for the rotated queries and one workspace, as a decoding loop keeps them; the lengths
    change between steps where there are two sets of them."""
    h_q, h_kv, d = heads
    g = torch.Generator(device="cuda").manual_seed(rows)
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
    batch, cap = len(lens[0]), max(map(max, lens)) + 8
    mk = lambda w, t: torch.zeros(batch, h_kv, cap, w, dtype=t, device="cuda")  # noqa: E731
    kv_len = i32([cap] * batch)
    if kv4:
        cache = sd.KV4Cache(mk(d // 2, torch.uint8), mk(d // 2, torch.uint8), mk(2, BF), mk(2, BF), kv_len)
        append, attend, size = sd.sd_kv4_append, sd.sd_kv4_verify_attention, sd.sd_kv4_attention_workspace_size
        parts = (cache.k, cache.v, cache.k_param, cache.v_param)
    else:
        cache = sd.KVCache(mk(d, BF), mk(d, BF), kv_len)
        append, attend = sd.sd_kv_append, sd.sd_verify_attention
        size = lambda q, kv: sd.sd_attention_workspace_size(sd.SD_ATTN_VERIFY, q, kv)  # noqa: E731
        parts = (cache.k, cache.v)
    fill = [normal(batch * cap, h_kv, d) for _ in range(2)]
    append(None, sd.NewRows(*fill, i32([cap * i for i in range(batch + 1)]), cap), cache)
    kept = [t.clone() for t in parts]
    starts = i32([rows * i for i in range(batch + 1)])
    steps = []
    for _ in range(STEPS):
        x = normal(batch * rows, h_q + 2 * h_kv, d)
        steps.append(sd.NewRows(x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:], starts, cap, q=x[:, :h_q]))
    rope, on_gpu = sd.Rope(d), [i32(x) for x in lens]
    q_out = torch.empty(batch * rows, h_q, d, dtype=BF, device="cuda")
    queries = sd.Queries(q_out, starts, rows, cap)
    ws = torch.empty(max(size(queries, cache), 16), dtype=torch.uint8, device="cuda")
    busy = torch.empty(1 << 28, device="cuda")

    def run(pause):
        for t, x in zip(parts, kept):
            t.copy_(x)
        kv_len.copy_(on_gpu[0])
        outs = [torch.empty_like(q_out) for _ in range(STEPS)]
        torch.cuda.synchronize()
        if not pause:  # (some milliseconds, in which the calls line up)
            for _ in range(60):
                busy.fill_(1.0)
        for i in range(STEPS):
            if len(lens) > 1:
                kv_len.copy_(on_gpu[i % len(lens)])
            for call in (lambda: append(rope, steps[i], cache, q_out=q_out),
                         lambda: attend(queries, cache, out=outs[i], workspace=ws)):
                if pause:
                    torch.cuda.synchronize()
                call()
        torch.cuda.synchronize()
        return outs

    want = run(True)
    for _ in range(3):
        for i, (a, b) in enumerate(zip(run(False), want)):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16)), i
