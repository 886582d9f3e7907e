// Appending rotated key / value rows to a cache, dense (fp32, bf16) or in 4 bits.
//
// Per row r of sequence b (position j = kv_len[b] - n + i): every query and key head turns by the
// row's angles and is rounded once; keys and values go to the row's slot of the cache, queries to
// q_out.  All of it is one pass over the rows, bound by their bytes (each read once and written
// once) for a prompt and by launch and load latency for a decode step.
//
// append_kernel (16-byte aligned rows): a block of 8 warps takes 1 or 4 rows, 8 or 2 warps each.  A
// thread handles a unit of two VEC-element chunks of a head, chosen so that both elements of every
// pair are its own (half layout: chunks rotary/2 apart; q_out may so overwrite q), and goes with it
// through the row's heads, loading two heads ahead.  It asks for the first ones at once, since
// their place depends on nothing looked up.  Then its warp finds the row's sequence (a 32-way
// search of q_start, one round of loads for up to 32 sequences) and slot, and the row's warps form
// its cosines and sines, each once: position * f_m is taken in turns and reduced to [-1/2, 1/2] in
// fp64 (positions reach 1e6, where an fp32 angle is off by 0.06 rad), so the fp32 sine and cosine
// see a small argument.  A thread's own pairs' then stay in registers for all heads.
// append_narrow_kernel takes the rest (odd strides and alignments, rotated parts that cut a
// 16-byte chunk) one pair at a time.
//
// 4-bit rows: the D/(2 VEC) neighbouring lanes of a head share its minimum and maximum by
// shuffles, and each writes its chunks' codes as one word per 8 channels.  A key's rotation is in
// fp64 here: its rounded value decides codes, and a code is a whole step.  A code is the rounded
// quotient (x - lo) / s: fp32 with one reciprocal per row, rounded by adding and subtracting
// 1.5 2^23 (the sum's low bits are then the code), and in fp64 when the fp32 quotient is within
// 1e-4 of a border (its own error is below 5e-6), which gives the fp64 quotient's code every time
// at fp32 cost.
//
// Measured (28 query and 4 KV heads of 128, bf16): 8 ragged prompts of up to 4,096 rows into pages
// 81 us, 4.8 TB/s; a prompt of 26,024 rows into a 4-bit cache 127 us, 3.9 TB/s.  Neither is at a
// limit of the chip: HBM is busy for 55 and 46%, issue slots for 64 and 66%, the ALU pipe for 47 and
// 43%, fp64 for 4% (4 bits).  Warps wait for global loads (2.4 and 2.2 of 10 per issue): a block
// looks up, forms its cosines and meets a barrier before it turns anything, and the 4-bit keys' and
// values' loads come after the queries'.  At 64 registers (4 blocks per SM) the bf16 kernels spill
// 36 bytes, with 4-bit caches 160, which is 4% of the instructions.  (With the chunks in a structure
// that the compiler kept in local memory as a whole: 115 and 170 us.)  13,012 fp32 rows: 80 us (0.91
// of the copy rate), into 4 bits 88.  append_narrow_kernel: the prompt of 26,024 bf16 rows with a
// rotated part of 24 channels 175 us, into 4 bits 333.  A decode step's row 6.2 us (4 bits: 8.1), of
// which the kernel has 3.5 (5.2): launch and the loads that depend on one another.
#include <math.h>

#include <cuda_bf16.h>

#include "sd_internal.h"

namespace sd {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 4;  // rows per block, at most

struct RowInfo {
    int b, j;      // sequence and position
    int page;      // paged caches: the row's page
    int flags;     // bit 0: the row is valid (query), bit 1: its slot is (key, value)
};

// count of entries of q_start[1..batch] that are <= r: the row's sequence (all lanes)
__device__ __forceinline__ int find_sequence(const int32_t *q_start, int batch, int r, int lane) {
    int lo = 0, n = batch;
    while (n > 0) {
        const int step = (n + 31) / 32, idx = lo + step * (lane + 1);
        const bool le = idx <= lo + n && ld_dep(q_start + idx) <= r;
        const int cnt = __popc(__ballot_sync(0xffffffffu, le));
        const int hi = lo + n;
        lo += step * cnt;
        n = min(step - 1, hi - lo);
    }
    return lo;
}

template <typename T>
__device__ __forceinline__ float to_f(T x) {
    if constexpr (sizeof(T) == 4)
        return x;
    else
        return __uint_as_float((uint32_t)x << 16);
}
template <typename T>
__device__ __forceinline__ T from_f(float x) {
    if constexpr (sizeof(T) == 4)
        return x;
    else
        return (T)f32_to_bf16_bits(x);
}

// 16 bytes of the rows' type as floats (8 for bf16, 4 for fp32), and back with one rounding.
template <typename T, int VEC>
__device__ __forceinline__ void unpack(const uint4 &w, float (&f)[VEC]) {
    Chunk<sizeof(T) == 2>::to_float(w, f);
}
template <typename T, int VEC>
__device__ __forceinline__ uint4 pack(const float (&f)[VEC]) {
    if constexpr (sizeof(T) == 4) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
    } else {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t *>(&p);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

__device__ __forceinline__ float bf16_round(float x) {
    return __uint_as_float(f32_to_bf16_bits(x) << 16);
}

// Scale and low value of a row with extremes mn, mx (bad: it holds a non-finite element).
template <typename T>
__device__ __forceinline__ void row_params(float mn, float mx, bool bad, float &s, float &lo) {
    lo = bf16_round(mn);
    // (bf16 rows: the fp32 difference and quotient round to the same bf16 as fp64 ones, since a
    // fifteenth of a difference of two bf16 values is never next to the middle of two)
    s = sizeof(T) == 4 ? (float)(((double)mx - (double)lo) / 15.0) : __fdiv_rn(mx - lo, 15.f);
    s = mx > lo ? bf16_round(s) : 0.f;
    if (bad || !isfinite(mx - lo)) {  // (an infinite lo included)
        s = 0.f;
        lo = __uint_as_float(0x7fc00000u);
    }
}

constexpr float kRoundMagic = 12582912.f;  // 1.5 2^23: adding it rounds to a whole number, ties to even

// Code of x as a whole float; inv is 1 / s, or 0 for s == 0.
template <typename T>
__device__ __forceinline__ float code_of(float x, float s, float lo, float inv) {
    const float q = (x - lo) * inv;
    float c = (q + kRoundMagic) - kRoundMagic;
    if (!(fabsf(q - c) < 0.4999f))
        c = s > 0.f ? (float)rint(((double)x - (double)lo) / (double)s) : 0.f;
    // (bf16 rows: lo is the minimum itself, and (max - lo) / s is below 15.04)
    return sizeof(T) == 4 || !(c <= 15.f) ? fminf(fmaxf(c, 0.f), 15.f) : c;
}

__device__ __forceinline__ uint32_t param_bits(float s, float lo) {
    return (__float_as_uint(s) >> 16) | (__float_as_uint(lo) & 0xffff0000u);
}

// Sequence, position and slot of row r (every lane of the warp gets them).
__device__ __forceinline__ RowInfo find_row(const AppendParams &p, int r, int lane) {
    RowInfo f{0, 0, 0, 0};
    const int b = find_sequence(p.q_start, p.batch, r, lane);
    if (b >= p.batch) return f;
    const int q0 = ld_dep(p.q_start + b), q1 = ld_dep(p.q_start + b + 1), n = q1 - q0;
    const int len = ld_dep(p.kv_len + b);
    if (q0 < 0 || q0 > r || r >= q1) return f;
    if (q1 > p.n_rows || len < n || len > p.max_kv_len ||
        (p.page_size && len > (int64_t)p.max_pages * kPageSize)) {
        if (lane == 0) set_dev_err(p.dev_err, SD_DEVERR_SHAPE);
        return f;
    }
    f.b = b;
    f.j = len - n + (r - q0);
    f.flags = 3;
    if (p.page_size) {
        f.page = ld_dep(p.block_table + (int64_t)b * p.max_pages + (f.j >> 4));
        if (f.page < 0 || f.page >= p.num_pages) {
            if (lane == 0) set_dev_err(p.dev_err, SD_DEVERR_PAGE);
            f.flags = 1;
        }
    }
    return f;
}

// Block 0 reports the row starts that no row of the launch meets: negative or decreasing ones, and
// rows that begin at or behind n_rows.  (The blocks read q_start for their rows anyway.)
__device__ __forceinline__ void check_starts(const AppendParams &p) {
    if (blockIdx.x != 0) return;
    for (int b = threadIdx.x; b < p.batch; b += kThreads) {
        const int q0 = ld_dep(p.q_start + b), q1 = ld_dep(p.q_start + b + 1);
        if (q0 < 0 || q1 < q0 || q1 > p.n_rows) set_dev_err(p.dev_err, SD_DEVERR_SHAPE);
    }
}

// Position of row r, in turns of pair m, reduced to [-1/2, 1/2].
__device__ __forceinline__ double turn_of(const AppendParams &p, const RowInfo &f, int r, int m) {
    const int pos = p.pos ? ld_dep(p.pos + r) : f.j;
    const double t = (double)pos * p.rope.turns[m];
    return t - rint(t);
}

__device__ __forceinline__ float2 cos_sin(const AppendParams &p, double t) {
    float sn, cs;
    sincospif((float)(2.0 * t), &sn, &cs);
    const float g = (float)p.rope.gain;
    return make_float2(g * cs, g * sn);
}

__device__ __forceinline__ double2 cos_sin_d(const AppendParams &p, double t) {
    double sn, cs;
    sincospi(2.0 * t, &sn, &cs);
    return make_double2(p.rope.gain * cs, p.rope.gain * sn);
}

// Row number of head h at the row's slot (paged, and 4-bit caches), and its element offset.
__device__ __forceinline__ int64_t slot_row(const AppendParams &p, const RowInfo &f, int h) {
    return p.page_size ? ((int64_t)f.page * p.h_kv + h) * kPageSize + (f.j & 15)
                       : (int64_t)f.b * p.stride_b + (int64_t)h * p.stride_h + f.j;
}
__device__ __forceinline__ int64_t slot_element(const AppendParams &p, const RowInfo &f, int h) {
    return p.page_size ? slot_row(p, f, h) * p.head_dim
                       : (int64_t)f.b * p.stride_b + (int64_t)h * p.stride_h +
                             (int64_t)f.j * p.head_dim;
}

template <typename T, int D, int VEC, bool KV4>
__global__ void __launch_bounds__(kThreads, 4)
append_kernel(const __grid_constant__ AppendParams p) {
    pdl_trigger();  // (see launch_pdl)
    pdl_wait();
    constexpr int UH = D / (2 * VEC);  // units (lanes) of a head
    // cosine and sine of pair u VEC + e at [e][u]
    __shared__ float2 s_cs[kMaxRows][VEC][UH];
    __shared__ double2 s_csd[KV4 ? kMaxRows : 1][KV4 ? VEC : 1][KV4 ? UH : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int wpr = kThreads / 32 / p.rows_per_block;  // warps of a row
    const int row = warp / wpr, r = blockIdx.x * p.rows_per_block + row;
    const bool here = r < p.n_rows;
    const int slots = wpr * (32 / UH), slot = (warp % wpr) * (32 / UH) + lane / UH;
    const int rot = p.rope.rotary_dim, half_rot = rot >> 1;
    const bool half = p.rope.layout == SD_ROPE_HALF;
    const int u = lane % UH;  // this thread's unit of every head it handles
    // Channels of the unit's two chunks in a head that is rotated, and in one that is copied.
    const bool turns = u * 2 * VEC < rot;
    const int ra = turns && half ? u * VEC : u * 2 * VEC;
    const int rb = turns && half ? ra + half_rot : ra + VEC;
    const int ca = u * 2 * VEC;

    // heads: queries, keys, values (4-bit caches: queries here, the others below)
    const int heads = p.h_q + (KV4 ? 0 : 2 * p.h_kv);
    auto is_value = [&](int hd) { return hd >= p.h_q + p.h_kv; };
    auto source = [&](int hd) {
        return hd < p.h_q ? static_cast<const T *>(p.q) + (int64_t)r * p.q_stride + hd * D
               : !is_value(hd)
                   ? static_cast<const T *>(p.k) + (int64_t)r * p.k_stride + (hd - p.h_q) * D
                   : static_cast<const T *>(p.v) + (int64_t)r * p.v_stride +
                         (hd - p.h_q - p.h_kv) * D;
    };
    uint4 a0, b0, a1, b1;  // the next two heads' chunks
    a0 = b0 = a1 = b1 = make_uint4(0u, 0u, 0u, 0u);
    auto fetch = [&](uint4 &a, uint4 &b, int hd, int end) {
        if (here && hd < end) {
            const T *src = source(hd);
            const bool v = is_value(hd);
            a = *reinterpret_cast<const uint4 *>(src + (v ? ca : ra));
            b = *reinterpret_cast<const uint4 *>(src + (v ? ca + VEC : rb));
        }
    };
    fetch(a0, b0, slot, heads);
    fetch(a1, b1, slot + slots, heads);

    RowInfo f{0, 0, 0, 0};
    if (here) f = find_row(p, r, lane);
    if (f.flags & 1)
        for (int m = (warp % wpr) * 32 + lane; m < half_rot; m += wpr * 32) {
            const double t = turn_of(p, f, r, m);
            if constexpr (KV4) {
                const double2 cs = cos_sin_d(p, t);
                s_csd[row][m % VEC][m / VEC] = cs;
                s_cs[row][m % VEC][m / VEC] = make_float2((float)cs.x, (float)cs.y);
            } else {
                s_cs[row][m % VEC][m / VEC] = cos_sin(p, t);
            }
        }
    check_starts(p);
    __syncthreads();
    if (!(f.flags & 1)) return;
    float2 cs[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) cs[e] = turns ? s_cs[row][e][u] : make_float2(1.f, 0.f);
    // Turns the unit's pairs: g(index of the first and second element in a / b, e of the table).
    auto pairs = [&](auto &&g) {
        if (half) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) g(e, VEC + e, e);
        } else {
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                if (ra + 2 * e < rot) g(2 * e, 2 * e + 1, e);
        }
    };
#pragma unroll 1
    for (int hd = slot; hd < heads; hd += slots) {
        uint4 xa = a0, xb = b0;
        a0 = a1;
        b0 = b1;
        fetch(a1, b1, hd + 2 * slots, heads);
        const bool is_q = hd < p.h_q, is_v = is_value(hd);
        if (!(f.flags & (is_q ? 1 : 2))) continue;
        if (turns && !is_v) {
            float v[2][VEC];
            unpack<T, VEC>(xa, v[0]);
            unpack<T, VEC>(xb, v[1]);
            pairs([&](int ea, int eb, int e) {
                float &x = v[ea / VEC][ea % VEC], &y = v[eb / VEC][eb % VEC];
                const float c = x, d = y;
                x = c * cs[e].x - d * cs[e].y;
                y = d * cs[e].x + c * cs[e].y;
            });
            xa = pack<T, VEC>(v[0]);
            xb = pack<T, VEC>(v[1]);
        }
        T *dst = is_q   ? static_cast<T *>(p.q_out) + ((int64_t)r * p.h_q + hd) * D
                 : is_v ? static_cast<T *>(p.v_cache) + slot_element(p, f, hd - p.h_q - p.h_kv)
                        : static_cast<T *>(p.k_cache) + slot_element(p, f, hd - p.h_q);
        *reinterpret_cast<uint4 *>(dst + (is_v ? ca : ra)) = xa;
        *reinterpret_cast<uint4 *>(dst + (is_v ? ca + VEC : rb)) = xb;
    }
    if constexpr (KV4) {
        if (!(f.flags & 2)) return;
        const int end = p.h_q + 2 * p.h_kv;
        fetch(a0, b0, p.h_q + slot, end);
#pragma unroll 1
        for (int hd = p.h_q + slot; hd < end; hd += slots) {
            const bool is_k = !is_value(hd);
            const int h = is_k ? hd - p.h_q : hd - p.h_q - p.h_kv;
            const int oa = is_k ? ra : ca, ob = is_k ? rb : ca + VEC;
            float v[2][VEC];
            unpack<T, VEC>(a0, v[0]);
            unpack<T, VEC>(b0, v[1]);
            fetch(a0, b0, hd + slots, end);
            if (is_k && turns) {
                pairs([&](int ea, int eb, int e) {
                    const double2 cd = s_csd[row][e][u];
                    float &x = v[ea / VEC][ea % VEC], &y = v[eb / VEC][eb % VEC];
                    const double c = x, d = y;
                    x = (float)(c * cd.x - d * cd.y);
                    y = (float)(d * cd.x + c * cd.y);
                });
                // (the key as the rows' type holds it)
                unpack<T, VEC>(pack<T, VEC>(v[0]), v[0]);
                unpack<T, VEC>(pack<T, VEC>(v[1]), v[1]);
            }
            float mn = INFINITY, mx = -INFINITY, zero = 0.f;
#pragma unroll
            for (int e = 0; e < 2 * VEC; ++e) {
                const float w = v[e / VEC][e % VEC];
                mn = fminf(mn, w);
                mx = fmaxf(mx, w);
                zero = fmaf(w, 0.f, zero);  // NaN once any element is not finite
            }
            // the UH lanes of the head (a head's lanes go through the loop together)
            const unsigned group = UH == 32 ? 0xffffffffu : ((1u << UH) - 1u) << (lane & ~(UH - 1));
#pragma unroll
            for (int o = UH / 2; o > 0; o >>= 1) {
                mn = fminf(mn, __shfl_xor_sync(group, mn, o));
                mx = fmaxf(mx, __shfl_xor_sync(group, mx, o));
            }
            const bool bad = (__ballot_sync(group, zero != 0.f) & group) != 0u;
            float s, lo;
            row_params<T>(mn, mx, bad, s, lo);
            const float inv = s > 0.f ? 1.f / s : 0.f;
            // codes as whole floats; quotients near a border are taken again in fp64
            float code[2][VEC], edge = 0.f;
#pragma unroll
            for (int e = 0; e < 2 * VEC; ++e) {
                const float q = (v[e / VEC][e % VEC] - lo) * inv;
                const float c = (q + kRoundMagic) - kRoundMagic;
                code[e / VEC][e % VEC] = c;
                edge = fmaxf(edge, fabsf(q - c));
                if (!(q < 16.f)) edge = 1.f;  // (also NaN)
            }
            if (!(edge < 0.4999f) || sizeof(T) == 4) {
#pragma unroll
                for (int e = 0; e < 2 * VEC; ++e)
                    code[e / VEC][e % VEC] = code_of<T>(v[e / VEC][e % VEC], s, lo, inv);
            }
            const int64_t rw = slot_row(p, f, h);
            unsigned char *codes = static_cast<unsigned char *>(is_k ? p.k_cache : p.v_cache);
            T *vals = static_cast<T *>(is_k ? p.k_out : p.v_out);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                // the sum of code_e 16^e from the floats' bits: each is the magic's plus the code
                uint32_t w = 0u;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    w += (__float_as_uint(code[c][e] + kRoundMagic) - __float_as_uint(kRoundMagic))
                         << (4 * e);
                    v[c][e] = fmaf(s, code[c][e], lo);
                }
                const int o = c ? ob : oa;
                unsigned char *cp = codes + rw * (D / 2) + o / 2;
                if constexpr (VEC == 8)
                    *reinterpret_cast<uint32_t *>(cp) = w;
                else
                    *reinterpret_cast<unsigned short *>(cp) = (unsigned short)w;
                if (vals)
                    *reinterpret_cast<uint4 *>(vals + ((int64_t)r * p.h_kv + h) * D + o) =
                        pack<T, VEC>(v[c]);
            }
            if (u == 0) {
                (is_k ? p.k_param : p.v_param)[rw] = param_bits(s, lo);
                if (lo != lo) set_dev_err(p.dev_err, SD_DEVERR_NUMERIC);
            }
        }
    }
}

// One row per block, one pair of channels at a time.
template <typename T, int D, bool KV4>
__global__ void __launch_bounds__(kThreads) append_narrow_kernel(const __grid_constant__ AppendParams p) {
    pdl_trigger();  // (see launch_pdl)
    pdl_wait();
    __shared__ float2 s_cs[D / 2];
    __shared__ double2 s_csd[KV4 ? D / 2 : 1];
    __shared__ float s_val[KV4 ? kThreads / 32 : 1][KV4 ? D : 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = blockIdx.x;
    const RowInfo f = find_row(p, r, lane);
    check_starts(p);
    if (!(f.flags & 1)) return;
    const int rot = p.rope.rotary_dim, half_rot = rot >> 1;
    const bool half = p.rope.layout == SD_ROPE_HALF;
    if (tid < half_rot) {
        const double t = turn_of(p, f, r, tid);
        if constexpr (KV4) {
            s_csd[tid] = cos_sin_d(p, t);
            s_cs[tid] = make_float2((float)s_csd[tid].x, (float)s_csd[tid].y);
        } else {
            s_cs[tid] = cos_sin(p, t);
        }
    }
    __syncthreads();
    const T *kin = static_cast<const T *>(p.k) + (int64_t)r * p.k_stride;
    const T *vin = static_cast<const T *>(p.v) + (int64_t)r * p.v_stride;
    // channels of pair x of a head: rotated pairs first, then neighbours
    auto channels = [&](int x, bool turned, int &a, int &b) {
        a = turned && half ? x : 2 * x;
        b = turned && half ? x + half_rot : a + 1;
    };
    for (int x = tid; x < p.h_q * (D / 2); x += kThreads) {
        const int h = x / (D / 2), m = x % (D / 2);
        const T *src = static_cast<const T *>(p.q) + (int64_t)r * p.q_stride + h * D;
        T *dst = static_cast<T *>(p.q_out) + ((int64_t)r * p.h_q + h) * D;
        int ia, ib;
        channels(m, 2 * m < rot, ia, ib);
        T a = src[ia], b = src[ib];
        if (2 * m < rot) {
            const float fa = to_f<T>(a), fb = to_f<T>(b);
            a = from_f<T>(fa * s_cs[m].x - fb * s_cs[m].y);
            b = from_f<T>(fb * s_cs[m].x + fa * s_cs[m].y);
        }
        dst[ia] = a;
        dst[ib] = b;
    }
    if (!(f.flags & 2)) return;
    if constexpr (!KV4) {
        for (int x = tid; x < p.h_kv * (D / 2); x += kThreads) {
            const int h = x / (D / 2), m = x % (D / 2);
            const int64_t o = slot_element(p, f, h);
            T *kd = static_cast<T *>(p.k_cache) + o, *vd = static_cast<T *>(p.v_cache) + o;
            int ia, ib;
            channels(m, 2 * m < rot, ia, ib);
            T a = kin[h * D + ia], b = kin[h * D + ib];
            if (2 * m < rot) {
                const float fa = to_f<T>(a), fb = to_f<T>(b);
                a = from_f<T>(fa * s_cs[m].x - fb * s_cs[m].y);
                b = from_f<T>(fb * s_cs[m].x + fa * s_cs[m].y);
            }
            kd[ia] = a;
            kd[ib] = b;
            vd[2 * m] = vin[h * D + 2 * m];
            vd[2 * m + 1] = vin[h * D + 2 * m + 1];
        }
    } else {
        // One warp per (K or V, head), the row's values through shared memory so that each lane
        // holds neighbouring channels when it packs codes.
        float *val = s_val[warp];
        constexpr int EL = D / 32;
        for (int y = warp; y < 2 * p.h_kv; y += kThreads / 32) {
            const bool is_k = y < p.h_kv;
            const int h = is_k ? y : y - p.h_kv;
            const T *src = (is_k ? kin : vin) + h * D;
            for (int m = lane; m < D / 2; m += 32) {
                const bool turned = is_k && 2 * m < rot;
                int ia, ib;
                channels(m, turned, ia, ib);
                float a = to_f<T>(src[ia]), c = to_f<T>(src[ib]);
                if (turned) {
                    const double2 cs = s_csd[m];
                    const double da = a, dc = c;
                    a = to_f<T>(from_f<T>((float)(da * cs.x - dc * cs.y)));
                    c = to_f<T>(from_f<T>((float)(dc * cs.x + da * cs.y)));
                }
                val[ia] = a;
                val[ib] = c;
            }
            __syncwarp();
            float v[EL], mn = INFINITY, mx = -INFINITY, zero = 0.f;
#pragma unroll
            for (int e = 0; e < EL; ++e) {
                v[e] = val[lane * EL + e];
                mn = fminf(mn, v[e]);
                mx = fmaxf(mx, v[e]);
                zero = fmaf(v[e], 0.f, zero);
            }
            __syncwarp();  // (the buffer's next row)
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            }
            const bool bad = __any_sync(0xffffffffu, zero != 0.f);
            float s, lo;
            row_params<T>(mn, mx, bad, s, lo);
            const float inv = s > 0.f ? 1.f / s : 0.f;
            const int64_t rw = slot_row(p, f, h);
            uint32_t w = 0;
            T *vals = static_cast<T *>(is_k ? p.k_out : p.v_out);
#pragma unroll
            for (int e = 0; e < EL; ++e) {
                const float k = code_of<T>(v[e], s, lo, inv);
                w |= (uint32_t)(int)k << (4 * e);
                if (vals) vals[((int64_t)r * p.h_kv + h) * D + lane * EL + e] = from_f<T>(fmaf(s, k, lo));
            }
            unsigned char *cp =
                static_cast<unsigned char *>(is_k ? p.k_cache : p.v_cache) + rw * (D / 2) + lane * (EL / 2);
            if constexpr (EL == 4)
                *reinterpret_cast<unsigned short *>(cp) = (unsigned short)w;
            else
                *cp = (unsigned char)w;
            if (lane == 0) {
                (is_k ? p.k_param : p.v_param)[rw] = param_bits(s, lo);
                if (lo != lo) set_dev_err(p.dev_err, SD_DEVERR_NUMERIC);
            }
        }
    }
}

template <typename T, int D, bool KV4>
cudaError_t launch_t(const AppendParams &p, bool wide, cudaStream_t s) {
    constexpr int VEC = 16 / (int)sizeof(T);
    if (!wide)
        return launch_pdl(append_narrow_kernel<T, D, KV4>, dim3(p.n_rows), dim3(kThreads), 0, s, p);
    const int blocks = (p.n_rows + p.rows_per_block - 1) / p.rows_per_block;
    return launch_pdl(append_kernel<T, D, VEC, KV4>, dim3(blocks), dim3(kThreads), 0, s, p);
}

template <typename T, int D>
cudaError_t launch_d(const AppendParams &p, bool wide, cudaStream_t s) {
    return p.kv4 ? launch_t<T, D, true>(p, wide, s) : launch_t<T, D, false>(p, wide, s);
}

}  // namespace

cudaError_t launch_append(AppendParams p, bool wide, cudaStream_t s) {
    // one row per block while that leaves SMs free, else four (two warps then form a row's 64
    // cosines and sines at once)
    p.rows_per_block = p.n_rows <= 2 * device_sm_count() ? 1 : kMaxRows;
    const bool bf = p.dtype == SD_BF16;
    // 16-byte chunks need both chunks of a rotated unit aligned
    if (p.rope.layout == SD_ROPE_HALF && p.rope.rotary_dim % (bf ? 16 : 8) != 0) wide = false;
    if (bf)
        return p.head_dim == 128 ? launch_d<unsigned short, 128>(p, wide, s)
                                 : launch_d<unsigned short, 64>(p, wide, s);
    return p.head_dim == 128 ? launch_d<float, 128>(p, wide, s) : launch_d<float, 64>(p, wide, s);
}

}  // namespace sd
