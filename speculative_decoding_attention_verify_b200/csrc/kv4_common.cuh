// Shared by the kernels that read a 4-bit cache: sequences, row numbers, and the division of a
// call's tiles over its CTAs.
//
// Tensor-core engines.  A unit is a (sequence, KV head); its positions are tiles of kKv4Tile.
// All units' tiles, in (sequence, KV head) order, form one list of T tiles, counted on the device
// from the actual lengths, and CTA c of G takes tiles [c T / G, (c+1) T / G) of it, so a ragged
// batch is spread as evenly as an equal one whatever the hints say.  A unit inside one CTA's
// range gets its output directly.  Otherwise the CTA that starts it writes partial slot 2c + 1
// and each CTA that continues it slot 2c (of one CTA's units only the first can be continued and
// only the last left open), and kv4_merge_kernel joins them in CTA order.
#pragma once

#include "sd_internal.h"

namespace sd {

constexpr int kKv4Tile = 128;

// Sequence b of a 4-bit attention call: its rows and length; false (and *bad for a violated
// hint) when it has no work.
__device__ __forceinline__ bool kv4_sequence(const Kv4Params &p, int b, int &q0, int &n_q,
                                             int &kv_len, bool &bad) {
    q0 = __ldg(p.q_start + b);
    n_q = __ldg(p.q_start + b + 1) - q0;
    kv_len = __ldg(p.kv_len + b);
    bad = false;
    if (n_q == 0) return false;
    bad = n_q < 0 || n_q > p.max_q_rows || q0 < 0 || q0 + n_q > p.rows_cap || kv_len < n_q ||
          kv_len > p.max_kv_len || (p.page_size && kv_len > (int64_t)p.max_pages * kPageSize);
    return !bad;
}

__device__ __forceinline__ int kv4_tiles(const Kv4Params &p, int b) {
    int q0, n_q, kv_len;
    bool bad;
    return kv4_sequence(p, b, q0, n_q, kv_len, bad) ? (kv_len + kKv4Tile - 1) / kKv4Tile : 0;
}

// Row number of position j of (b, h), or -1 when its page is outside the pool.
__device__ __forceinline__ int64_t kv4_row(const Kv4Params &p, int b, int h, int j) {
    if (p.page_size == 0)
        return (int64_t)b * p.stride_b + (int64_t)h * p.stride_h + j;
    const int page = __ldg(p.block_table + (int64_t)b * p.max_pages + (j >> 4));
    if (page < 0 || page >= p.num_pages) {
        set_dev_err(p.dev_err, SD_DEVERR_PAGE);
        return -1;
    }
    return ((int64_t)page * p.h_kv + h) * kPageSize + (j & 15);
}

__device__ __forceinline__ float param_scale(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float param_low(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ long long warp_sum_ll(long long x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

// Tiles (of one KV head) of all sequences and of those before sequence b.  Every thread of the
// block calls it; s_red holds 2 * NT / 32 values.
template <int NT>
__device__ __forceinline__ void kv4_count(const Kv4Params &p, int b, long long *s_red,
                                          long long &total, long long &before) {
    long long t = 0, u = 0;
    for (int i = threadIdx.x; i < p.batch; i += NT) {
        const int n = kv4_tiles(p, i);
        t += n;
        if (i < b) u += n;
    }
    t = warp_sum_ll(t);
    u = warp_sum_ll(u);
    if ((threadIdx.x & 31) == 0) {
        s_red[2 * (threadIdx.x >> 5)] = t;
        s_red[2 * (threadIdx.x >> 5) + 1] = u;
    }
    __syncthreads();
    total = before = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        total += s_red[2 * w];
        before += s_red[2 * w + 1];
    }
}

// CTA of G that holds tile x of T.
__device__ __forceinline__ int kv4_cta_of(long long x, long long total, int ctas) {
    return (int)(((x + 1) * ctas - 1) / total);
}

// Where partial slot `slot` keeps local row lr: its outputs, and its (maximum in log2 units, sum).
__device__ __forceinline__ float *kv4_slot_o(const Kv4Params &p, int64_t slot, int lr) {
    return p.ws + (slot * (p.group * p.max_q_rows) + lr) * p.head_dim;
}
__device__ __forceinline__ float *kv4_slot_ml(const Kv4Params &p, int64_t slot, int lr) {
    const int64_t rows = p.group * p.max_q_rows;
    return p.ws + (int64_t)p.n_slots * rows * p.head_dim + (slot * rows + lr) * 2;
}

}  // namespace sd
