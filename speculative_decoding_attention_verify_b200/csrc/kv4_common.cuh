// Shared by the kernels that read a 4-bit cache: sequences, row numbers, and the division of a
// call's tiles over its CTAs.
//
// Tensor-core engines.  A unit is a (sequence, KV head); its positions are tiles of p.tile.
// All units' tiles, in (sequence, KV head) order, form one list of T tiles, counted on the device
// from the actual lengths, and CTA c of G takes tiles [c T / G, (c+1) T / G) of it, so a ragged
// batch is spread as evenly as an equal one whatever the hints say.  A unit inside one CTA's
// range gets its output directly.  Otherwise the CTA that starts it writes partial slot 2c + 1
// and each CTA that continues it slot 2c (of one CTA's units only the first can be continued and
// only the last left open), and kv4_merge_kernel joins them in CTA order.  With p.whole the CTAs
// share the units instead, each a range of whole ones: nothing is left to join.
#pragma once

#include <cuda_fp16.h>

#include "sd_internal.h"

namespace sd {

// Sequence b of a 4-bit attention call: its rows and length; false (and *bad for a violated
// hint) when it has no work.
__device__ __forceinline__ bool kv4_sequence(const Kv4Params &p, int b, int &q0, int &n_q,
                                             int &kv_len, bool &bad) {
    q0 = ld_dep(p.q_start + b);
    n_q = ld_dep(p.q_start + b + 1) - q0;
    kv_len = ld_dep(p.kv_len + b);
    bad = false;
    if (n_q == 0) return false;
    bad = n_q < 0 || n_q > p.max_q_rows || q0 < 0 || q0 + n_q > p.rows_cap || kv_len < n_q ||
          kv_len > p.max_kv_len || (p.page_size && kv_len > (int64_t)p.max_pages * kPageSize);
    return !bad;
}

// Row number of position j of (b, h), or -1 when its page is outside the pool.
__device__ __forceinline__ int64_t kv4_row(const Kv4Params &p, int b, int h, int j) {
    if (p.page_size == 0)
        return (int64_t)b * p.stride_b + (int64_t)h * p.stride_h + j;
    const int page = ld_dep(p.block_table + (int64_t)b * p.max_pages + (j >> 4));
    if (page < 0 || page >= p.num_pages) {
        set_dev_err(p.dev_err, SD_DEVERR_PAGE);
        return -1;
    }
    return ((int64_t)page * p.h_kv + h) * kPageSize + (j & 15);
}

__device__ __forceinline__ float param_scale(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float param_low(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// CTAs that take part: no more than there are tiles, so that each has one at least.
__device__ __forceinline__ int kv4_ctas(const Kv4Params &p, long long total) {
    return (int)(total < p.ctas ? total : p.ctas);
}

// ---- what the tensor-core kernels share of the mathematics (kv4_mma.cu) ----

__device__ __forceinline__ void cp_async16z(uint32_t dst, const void *src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void cp_async4z(uint32_t dst, const void *src, int n) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
}

// Exponents of the weights.  A maximum is set so that the largest weight becomes 2^kTopLog2 (or up to
// twice that, in whole steps), and moves only when one would exceed 2^kGrowLog2 (fp16 ends below
// 2^16).  fp16's smallest step is 2^-24,
// so a weight is off by 2^-11 of itself or by 2^-35 of its row's largest, whichever is more: 140,000
// positions of next to no weight lose 2^-18 together, where a largest weight of 1 would lose 2^-8.
constexpr float kTopLog2 = 10.f, kGrowLog2 = 15.f;

// A scale below this is taken for it: 1 / s stays in range, and codes of such rows are worth less
// than 1e-26.
constexpr float kMinScale = 8.0779357e-28f;  // 2^-90

// The scale that a row of V counts with.  A row of one value (s = 0) has codes 0, so any serves: one
// well below the row's value, or the weight of a sink of zeros would set the scale of all others'
// weights, and -8 and + 8 times it (codes taken as c - 8) would not cancel to 2^-17 of the value.
__device__ __forceinline__ float value_scale(uint32_t w) {
    const float s = param_scale(w);
    return fmaxf(s == 0.f ? fabsf(param_low(w)) * 0.00390625f : s, kMinScale);
}

// Codes at nibble P (0..3) of both halves of w as a pair of fp16 numbers: c 2^-24 (P even) or
// 16 c 2^-24 (P odd).  w8 is w >> 8.
template <int P>
__device__ __forceinline__ uint32_t codes_at(uint32_t w, uint32_t w8) {
    return (P < 2 ? w : w8) & (P & 1 ? 0x00f000f0u : 0x000f000fu);
}

// The same codes as whole numbers around zero: c - 8 (P even) or 16 (c - 8) (P odd), from the
// fp16 numbers 1024 + c and 1024 + 16 c.
template <int P>
__device__ __forceinline__ uint32_t centred_at(uint32_t w, uint32_t w8) {
    const uint32_t x = codes_at<P>(w, w8) | 0x64006400u;
    const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&x),
                              __float2half2_rn(P & 1 ? 1152.f : 1032.f));
    return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 p = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Power of two that brings a row's largest query element below 2^14, and 2^24 over it (codes_at's
// scale).
__device__ __forceinline__ float query_scale(float top, float &unscale) {
    const int e = (int)(__float_as_uint(top) >> 23);  // biased; 255: not finite
    // (rows of zeros, and elements beyond 2^114 or not finite, keep a scale that is in range)
    const int k = e == 0 || e == 255 ? 0 : min(max(127 + 13 - e, -100), 126);
    unscale = __uint_as_float((uint32_t)(127 + 24 - k) << 23);
    return __uint_as_float((uint32_t)(127 + k) << 23);
}

// The CTAs that hold a unit's first and last tile, written by those CTAs for the merge.
__device__ __forceinline__ int2 *kv4_unit_ctas(const Kv4Params &p) {
    return reinterpret_cast<int2 *>(p.ws + (int64_t)p.n_slots * p.group * p.max_q_rows *
                                               (p.head_dim + 2));
}

// Where partial slot `slot` keeps local row lr: its outputs, and its (maximum in log2 units, sum).
__device__ __forceinline__ float *kv4_slot_o(const Kv4Params &p, int64_t slot, int lr) {
    return p.ws + (slot * (p.group * p.max_q_rows) + lr) * p.head_dim;
}
__device__ __forceinline__ float *kv4_slot_ml(const Kv4Params &p, int64_t slot, int lr) {
    const int64_t rows = p.group * p.max_q_rows;
    return p.ws + (int64_t)p.n_slots * rows * p.head_dim + (slot * rows + lr) * 2;
}

// Sequence b or the next one with work (batch at the end).  Out of line: cursors move to another
// sequence rarely, and the tile loops have to stay small.
static __device__ __noinline__ int kv4_next_sequence(const Kv4Params &p, int b) {
    for (; b < p.batch; ++b) {
        int q0, n_q, kv_len;
        bool bad;
        if (kv4_sequence(p, b, q0, n_q, kv_len, bad)) break;
    }
    return b;
}

// A position in the list of tiles: tile t of unit (b, g), with the sequence's row data.
struct Kv4Cursor {
    int b, g, t, tiles;
    int q0, n_q, kv_len;
    // Sequence b at head g, or the next one with work (b = batch at the end).
    __device__ __forceinline__ void load(const Kv4Params &p) {
        const int from = b;
        b = kv4_next_sequence(p, b);
        if (b != from) g = 0;
        tiles = 1;
        kv_len = 0;
        if (b >= p.batch) return;
        q0 = ld_dep(p.q_start + b);
        n_q = ld_dep(p.q_start + b + 1) - q0;
        kv_len = ld_dep(p.kv_len + b);
        tiles = (kv_len + p.tile - 1) / p.tile;
    }
    // n tiles on, within the unit or to the start of the next one.
    __device__ __forceinline__ void skip(const Kv4Params &p, int n) {
        t += n;
        if (t < tiles) return;
        t = 0;
        if (++g < p.h_kv) return;
        g = 0;
        ++b;
        load(p);
    }
    __device__ __forceinline__ void next(const Kv4Params &p) { skip(p, 1); }
};

struct Kv4Start {
    Kv4Cursor c;       // at tile 0 of KV head 0 of its sequence
    long long before;  // tiles of one KV head before that sequence
};

// The CTA's tiles: [lo, hi) of the list (p.whole: hi - lo of its own units), and the cursor at the
// first.  Every thread of the block calls it; s_red holds NT / 32 values.  The sequences are read
// once, NT at a time (one round of loads for up to NT of them), and CTA 0 reports violated hints.
template <int NT>
__device__ __forceinline__ Kv4Cursor kv4_first(const Kv4Params &p, long long *s_red,
                                               Kv4Start *s_start, long long &lo, long long &hi) {
    constexpr int W = NT / 32;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long units = (long long)p.batch * p.h_kv;
    const long long u0 = units * blockIdx.x / p.ctas, u1 = units * (blockIdx.x + 1) / p.ctas;
    // pass 0: the total (p.whole: the tiles of units [u0, u1)); pass 1: the sequence of tile lo.
    // One chunk of sequences needs one pass: every thread keeps its own.
    Kv4Cursor mine{};
    long long total = 0;
    int n = 0;
    for (int i0 = 0; i0 < p.batch; i0 += NT) {
        const int i = i0 + tid;
        n = 0;
        if (i < p.batch) {
            bool bad;
            if (kv4_sequence(p, i, mine.q0, mine.n_q, mine.kv_len, bad))
                n = (mine.kv_len + p.tile - 1) / p.tile;
            if (bad && blockIdx.x == 0) set_dev_err(p.dev_err, SD_DEVERR_SHAPE);
        }
        mine.b = i;
        mine.tiles = n;
        long long x = n;
        if (p.whole) {
            const long long a = (long long)i * p.h_kv, b = a + p.h_kv;
            const long long in = (u1 < b ? u1 : b) - (u0 > a ? u0 : a);
            x = in > 0 ? x * in : 0;
        }
        total += x;
    }
    // sums before this thread's sequence within the last chunk, and the total
    auto scan = [&](long long x, long long &sum) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        __syncthreads();  // (the last use of s_red)
        if (lane == 31) s_red[warp] = x;
        __syncthreads();
        sum = 0;
        long long before = x;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            if (w < warp) before += s_red[w];
            sum += s_red[w];
        }
        return before;
    };
    long long sum;
    long long upto = scan(total, sum);
    Kv4Cursor c{};
    lo = hi = 0;
    if (p.whole) {
        hi = sum;
        if (hi == 0) return c;
        c.b = (int)(u0 / p.h_kv);
        c.g = (int)(u0 % p.h_kv);
        if (p.batch <= NT) {  // the thread that read the sequence hands it over
            if (tid == c.b) s_start->c = mine;
            __syncthreads();
            const int g = c.g;
            c = s_start->c;
            c.g = g;
            if (c.tiles == 0) c.load(p);
        } else {
            c.load(p);
        }
        return c;
    }
    const long long all = sum * p.h_kv;
    const int ctas = kv4_ctas(p, all);
    if ((int)blockIdx.x >= ctas) return c;
    lo = all * blockIdx.x / ctas;
    hi = all * (blockIdx.x + 1) / ctas;
    const long long want = lo / p.h_kv;  // (before b) <= want < (before b + 1)
    if (p.batch <= NT) {
        if (n > 0 && upto - n <= want && want < upto) {
            s_start->c = mine;
            s_start->before = upto - n;
        }
    } else {
        long long base = 0;
        for (int i0 = 0; i0 < p.batch && base <= want; i0 += NT) {
            const int i = i0 + tid;
            bool bad;
            n = 0;
            if (i < p.batch && kv4_sequence(p, i, mine.q0, mine.n_q, mine.kv_len, bad))
                n = (mine.kv_len + p.tile - 1) / p.tile;
            mine.b = i;
            mine.tiles = n;
            long long chunk;
            const long long end = base + scan(n, chunk);
            if (n > 0 && end - n <= want && want < end) {
                s_start->c = mine;
                s_start->before = end - n;
            }
            base += chunk;
        }
    }
    __syncthreads();
    c = s_start->c;
    const long long in = lo - s_start->before * p.h_kv;
    c.g = (int)(in / c.tiles);
    c.t = (int)(in % c.tiles);
    return c;
}

}  // namespace sd
