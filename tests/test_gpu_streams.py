"""Calls on a stream that is not the current one: what they allocate belongs to that stream."""
import pytest
import torch

from speculative_decoding_attention_verify_b200 import sdattn as sd

from .test_gpu_kv4_attention import Call
from .test_gpu_kv_append import BF, Case

pytestmark = pytest.mark.gpu


def not_handed_out(ptr, nbytes):
    """Memory freed for another stream is not given to the current one."""
    kept = [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(4)]
    return ptr not in [t.data_ptr() for t in kept]


@pytest.mark.parametrize("what", ["kv4", "dense"])
def test_workspaces_and_outputs_of_attention(what, monkeypatch):
    c = Call([3000], [9], 14, 2, 128, False, seed=2)
    want, _ = c.run()
    cap = c.kv.k.shape[2]
    if what == "dense":
        kv = sd.KVCache(*(torch.randn(1, 2, cap, 128, device="cuda").to(BF) for _ in range(2)), c.kv.kv_len)
        call = lambda **kw: sd.sd_verify_attention(c.queries, kv, **kw)  # noqa: E731
        want = call().cpu()
    else:
        call = lambda **kw: sd.sd_kv4_verify_attention(c.queries, c.kv, **kw)  # noqa: E731
    seen = []
    real = sd._ptr
    monkeypatch.setattr(sd, "_ptr", lambda t: (seen.append((t.data_ptr(), t.numel())) if t is not None and
                                               t.dtype == torch.uint8 else None, real(t))[1])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = call(stream=side)
    assert len(seen) == 1 and not_handed_out(*seen[0])
    side.synchronize()
    assert torch.equal(out.cpu(), want)
    ptr, n = out.data_ptr(), out.numel() * 2
    del out
    assert not_handed_out(ptr, n)


@pytest.mark.parametrize("kv4", [False, True])
def test_rotated_queries_of_appends(kv4):
    c = Case([30], [700], 4, 2, 64, False, BF, kv4=kv4)
    call = sd.sd_kv4_append if kv4 else sd.sd_kv_append
    rows, rope = c.new_rows(), sd.Rope(64)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    q = call(rope, rows, c.cache, stream=side)
    side.synchronize()
    assert torch.equal(q, call(rope, rows, c.cache))
    ptr, n = q.data_ptr(), q.numel() * 2
    del q
    assert not_handed_out(ptr, n)


def test_streams_of_other_makers():
    """Anything with a cuda_stream handle serves."""
    c = Call([300], [2], 4, 1, 64, False)
    want, _ = c.run()
    side = torch.cuda.Stream()

    class Handle:
        cuda_stream = side.cuda_stream

    out = sd.sd_kv4_verify_attention(c.queries, c.kv, stream=Handle())
    side.synchronize()
    assert torch.equal(out.cpu(), want)


def test_tokens_of_acceptance():
    """The -1 behind the emitted tokens are written on the call's own stream, before the tokens."""
    logits = torch.randn(6, 500, device="cuda")
    want = logits.argmax(1)
    draft = torch.cat([want[:2], want[3:5]]).int()
    gamma = torch.tensor([2, 2], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.empty(1 << 28, device="cuda")
    for _ in range(300):
        busy.fill_(1.0)  # (keeps the current stream behind for some tens of milliseconds)
    n, tok = sd.sd_accept_greedy(logits, draft, gamma, 2, stream=side)
    side.synchronize()
    got = torch.empty_like(tok)
    with torch.cuda.stream(side):
        got.copy_(tok)
    torch.cuda.synchronize()
    assert n.tolist() == [2, 2] and got.flatten().tolist() == want.tolist() and torch.equal(tok, got)
