"""Refusals of the cache appends and of attention over a 4-bit cache, without a GPU: a wrong
argument returns a status before anything is launched (the pointers are never dereferenced)."""
import ctypes

import pytest

from speculative_decoding_attention_verify_b200 import sdattn as sd

FAKE = ctypes.c_void_p(0x7f0000001000)
ODD = ctypes.c_void_p(0x7f0000001001)
OFF2 = ctypes.c_void_p(0x7f0000001002)


def _kv4(**kw):
    d = sd.sd_kv4_desc()
    d.dtype, d.h_kv, d.head_dim = sd.SD_BF16, 4, 128
    d.k = d.v = d.k_param = d.v_param = d.kv_len = FAKE
    d.stride_b, d.stride_h = 4 * 4096, 4096
    for n, x in kw.items():
        setattr(d, n, x)
    return d


def _kv(**kw):
    d = sd.sd_kv_desc()
    d.dtype, d.h_kv, d.head_dim = sd.SD_BF16, 4, 128
    d.k = d.v = d.kv_len = FAKE
    d.stride_b, d.stride_h, d.stride_pos = 4 * 4096 * 128, 4096 * 128, 128
    for n, x in kw.items():
        setattr(d, n, x)
    return d


def _rows(**kw):
    d = sd.sd_rows_desc()
    d.h_q, d.n_rows, d.max_kv_len = 28, 9, 4096
    d.q_start = d.q = d.k = d.v = FAKE
    d.q_stride, d.k_stride, d.v_stride = 28 * 128, 4 * 128, 4 * 128
    for n, x in kw.items():
        setattr(d, n, x)
    return d


def _rope(**kw):
    d = sd.sd_rope_desc()
    d.rotary_dim, d.theta, d.factor, d.original_len = 128, 1e6, 4.0, 32768
    for n, x in kw.items():
        setattr(d, n, x)
    return d


def _q(**kw):
    d = sd.sd_q_desc()
    d.h_q, d.max_q_rows, d.max_kv_len, d.q_start = 28, 9, 4096, FAKE
    for n, x in kw.items():
        setattr(d, n, x)
    return d


def _append(rope=None, rows=None, cache=None, batch=2, q_out=FAKE, kv4=False, k_out=None):
    r = ctypes.byref
    rope, rows = rope or _rope(), rows or _rows()
    if kv4:
        return sd.lib().sd_kv4_append(r(rope), r(rows), r(cache or _kv4()), batch, q_out, k_out, None,
                                      None, None)
    return sd.lib().sd_kv_append(r(rope), r(rows), r(cache or _kv()), batch, q_out, None, None)


BAD_ROPE = [dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=130), dict(layout=2),
            dict(scaling=4), dict(theta=0.0), dict(theta=float("nan")), dict(theta=float("inf")),
            dict(gain=-1.0), dict(gain=float("inf")),
            dict(scaling=sd.SD_ROPE_LINEAR, factor=0.5),
            dict(scaling=sd.SD_ROPE_NTK, rotary_dim=2),
            dict(scaling=sd.SD_ROPE_YARN, original_len=0),
            dict(scaling=sd.SD_ROPE_YARN, theta=1.0)]
BAD_ROWS = [dict(k=None), dict(v=None), dict(q_start=None), dict(n_rows=-1), dict(max_kv_len=0),
            dict(h_q=-1), dict(q=None), dict(h_q=0), dict(k_stride=511), dict(q_stride=3583),
            dict(v_stride=-512), dict(k=ODD)]


@pytest.mark.parametrize("kv4", [False, True])
def test_bad_rotations_and_rows_are_refused(kv4):
    for kw in BAD_ROPE:
        assert _append(rope=_rope(**kw), kv4=kv4) == sd.SD_ERR_INVALID_ARG, kw
    for kw in BAD_ROWS:
        assert _append(rows=_rows(**kw), kv4=kv4) == sd.SD_ERR_INVALID_ARG, kw
    assert _append(q_out=None, kv4=kv4) == sd.SD_ERR_INVALID_ARG
    assert _append(q_out=ODD, kv4=kv4) == sd.SD_ERR_INVALID_ARG
    assert _append(batch=0, kv4=kv4) == sd.SD_ERR_INVALID_ARG
    assert _append(batch=65536, kv4=kv4) == sd.SD_ERR_INVALID_ARG
    # q_out over q needs dense rows
    assert _append(rows=_rows(q_stride=28 * 128 + 8), q_out=FAKE, kv4=kv4) == sd.SD_ERR_INVALID_ARG


def test_frequencies_are_checked():
    table = (ctypes.c_float * 64)(*([float("nan")] * 64))
    assert _append(rope=_rope(inv_freq=ctypes.cast(table, ctypes.c_void_p))) == sd.SD_ERR_INVALID_ARG


def test_no_rows_is_a_no_op():
    assert _append(rows=_rows(n_rows=0)) == sd.SD_OK
    assert _append(rows=_rows(n_rows=0), kv4=True) == sd.SD_OK


def test_bad_caches_are_refused():
    for kw in (dict(k=None), dict(v=OFF2), dict(dtype=5), dict(h_kv=0), dict(kv_len=None),
               dict(page_size=8), dict(page_size=16), dict(stride_pos=256), dict(stride_h=4),
               dict(stride_b=-8)):
        assert _append(cache=_kv(**kw)) == sd.SD_ERR_INVALID_ARG, kw
    assert _append(cache=_kv(head_dim=96, stride_pos=96)) == sd.SD_ERR_UNSUPPORTED
    for kw in BAD_KV4:
        assert _append(cache=_kv4(**kw), kv4=True) == sd.SD_ERR_INVALID_ARG, kw
    assert _append(cache=_kv4(head_dim=32), kv4=True) == sd.SD_ERR_UNSUPPORTED
    assert _append(kv4=True, k_out=ODD) == sd.SD_ERR_INVALID_ARG


BAD_KV4 = [dict(k=None), dict(v=OFF2), dict(k_param=None), dict(v_param=OFF2), dict(dtype=5),
           dict(h_kv=0), dict(kv_len=None), dict(page_size=8), dict(page_size=16),
           dict(page_size=16, block_table=FAKE, max_pages_per_seq=4, num_pages=0),
           dict(stride_h=-1)]


def _attend(q=None, kv=None, batch=2, data=FAKE, out=FAKE, ws=FAKE, nbytes=1 << 40):
    return sd.lib().sd_kv4_verify_attention(ctypes.byref(q or _q()), data,
                                            ctypes.byref(kv or _kv4()), batch, out, ws, nbytes,
                                            None, None)


def test_bad_attention_calls_are_refused():
    n = ctypes.c_size_t(0)
    size = lambda q, kv, batch=2: sd.lib().sd_kv4_attention_workspace_size(  # noqa: E731
        ctypes.byref(q), ctypes.byref(kv), batch, ctypes.byref(n))
    for kw in BAD_KV4:
        assert _attend(kv=_kv4(**kw)) == sd.SD_ERR_INVALID_ARG, kw
        assert size(_q(), _kv4(**kw)) == sd.SD_ERR_INVALID_ARG, kw
    for kw in (dict(h_q=27), dict(h_q=0), dict(max_q_rows=0), dict(max_kv_len=0), dict(q_start=None),
               dict(softmax_scale=-1.0), dict(softmax_scale=float("nan")),
               dict(max_q_rows=1 << 30)):
        assert _attend(q=_q(**kw)) == sd.SD_ERR_INVALID_ARG, kw
        assert size(_q(**kw), _kv4()) == sd.SD_ERR_INVALID_ARG, kw
    assert _attend(kv=_kv4(head_dim=96)) == sd.SD_ERR_UNSUPPORTED
    assert size(_q(), _kv4(head_dim=96)) == sd.SD_ERR_UNSUPPORTED
    assert _attend(data=None) == sd.SD_ERR_INVALID_ARG
    assert _attend(out=None) == sd.SD_ERR_INVALID_ARG
    assert _attend(data=ODD) == sd.SD_ERR_INVALID_ARG
    assert _attend(batch=0) == sd.SD_ERR_INVALID_ARG
    # the workspace of the query is asked for, 16-byte aligned
    assert size(_q(), _kv4()) == sd.SD_OK and n.value > 0
    assert _attend(nbytes=n.value - 1) == sd.SD_ERR_WORKSPACE
    assert _attend(ws=None) == sd.SD_ERR_WORKSPACE
    assert _attend(ws=ctypes.c_void_p(0x7f0000001008)) == sd.SD_ERR_WORKSPACE


def test_workspace_does_not_grow_with_the_context():
    """The partial results are a share of the GPU's CTAs, not of the positions."""
    n = [ctypes.c_size_t(0), ctypes.c_size_t(0)]
    for x, length in zip(n, (100_000, 1_000_000)):
        assert sd.lib().sd_kv4_attention_workspace_size(
            ctypes.byref(_q(max_q_rows=1, max_kv_len=length)), ctypes.byref(_kv4(stride_h=10**6)),
            28, ctypes.byref(x)) == sd.SD_OK
    assert n[0].value == n[1].value
