// Appending rotated key / value rows to a cache, dense (fp32, bf16) or in 4 bits.
//
// Per row r of sequence b (position j = kv_len[b] - n + i): every query and key head turns by the
// row's angles and is rounded once; keys and values go to the row's slot of the cache, queries to
// q_out.  All of it is one pass over the rows, bound by their bytes (each read once and written
// once) for a prompt and by launch and load latency for a decode step.
//
// A block takes 1 or 4 rows.  One warp per row finds the row's sequence (a 32-way search of
// q_start, one round of loads for up to 32 sequences) and slot; the block then forms the row's
// cosines and sines once for all heads: position * f_m is taken in turns and reduced to
// [-1/2, 1/2] in fp64 (positions reach 1e6, where an fp32 angle is off by 0.06 rad), so the fp32
// sine and cosine see a small argument.  A thread handles a unit of two VEC-element chunks of a
// head, chosen so that both elements of every pair are its own (half layout: chunks rotary/2
// apart), and so q_out may overwrite q.
//
// 4-bit rows: the D/(2 VEC) neighbouring lanes of a head share its minimum and maximum by
// shuffles, and each writes its chunks' codes as one word per 8 channels.  A key's rotation is in
// fp64 here: its rounded value decides codes, and a code is a whole step.  A code is the rounded
// quotient (x - lo) / s: fp32 with one reciprocal per row, and in fp64 when the fp32 quotient is
// within 1e-4 of a border (its own error is below 5e-6), which gives the fp64 quotient's code
// every time at fp32 cost.
#include <math.h>

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
        const bool le = idx <= lo + n && __ldg(q_start + idx) <= r;
        const int cnt = __popc(__ballot_sync(0xffffffffu, le));
        const int hi = lo + n;
        lo += step * cnt;
        n = min(step - 1, hi - lo);
    }
    return lo;
}

template <typename T>
__device__ __forceinline__ float to_f(T x);
template <>
__device__ __forceinline__ float to_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f<unsigned short>(unsigned short x) {
    return __uint_as_float((uint32_t)x << 16);
}
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ unsigned short from_f<unsigned short>(float x) {
    return (unsigned short)f32_to_bf16_bits(x);
}

// VEC elements, moved as one 16-byte access when VEC > 1
template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Pack {
    T x[VEC];
};

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

__device__ __forceinline__ float code_of(float x, float s, float lo, float inv) {
    if (!(s > 0.f)) return 0.f;
    const float q = (x - lo) * inv;
    float c = rintf(q);
    if (!(fabsf(q - c) < 0.4999f)) c = (float)rint(((double)x - (double)lo) / (double)s);
    return fminf(fmaxf(c, 0.f), 15.f);
}

__device__ __forceinline__ uint32_t param_bits(float s, float lo) {
    return (__float_as_uint(s) >> 16) | (__float_as_uint(lo) & 0xffff0000u);
}

template <typename T, int D, int VEC, bool KV4>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendParams p) {
    pdl_trigger();  // (see launch_pdl)
    pdl_wait();
    constexpr int UH = D / (2 * VEC);  // units of a head
    using P = Pack<T, VEC>;
    __shared__ RowInfo s_row[kMaxRows];
    __shared__ float2 s_cs[kMaxRows][D / 2];
    __shared__ double2 s_csd[KV4 ? kMaxRows : 1][KV4 ? D / 2 : 1];
    __shared__ float s_val[(KV4 && VEC == 1) ? kThreads / 32 : 1][(KV4 && VEC == 1) ? D : 1];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r0 = blockIdx.x * p.rows_per_block;
    const int nr = min(p.rows_per_block, p.n_rows - r0);
    if (warp < nr) {
        const int r = r0 + warp;
        const int b = find_sequence(p.q_start, p.batch, r, lane);
        if (lane == 0) {
            RowInfo f{0, 0, 0, 0};
            if (b < p.batch) {
                const int q0 = __ldg(p.q_start + b), q1 = __ldg(p.q_start + b + 1), n = q1 - q0;
                const int len = __ldg(p.kv_len + b);
                if (q0 >= 0 && q0 <= r && r < q1) {
                    if (q1 > p.n_rows || len < n || len > p.max_kv_len ||
                        (p.page_size && len > (int64_t)p.max_pages * kPageSize)) {
                        set_dev_err(p.dev_err, SD_DEVERR_SHAPE);
                    } else {
                        f.b = b;
                        f.j = len - n + (r - q0);
                        f.flags = 3;
                        if (p.page_size) {
                            f.page = __ldg(p.block_table + (int64_t)b * p.max_pages + (f.j >> 4));
                            if (f.page < 0 || f.page >= p.num_pages) {
                                set_dev_err(p.dev_err, SD_DEVERR_PAGE);
                                f.flags = 1;
                            }
                        }
                    }
                }
            }
            s_row[warp] = f;
        }
    }
    __syncthreads();
    const int rot = p.rope.rotary_dim, half_rot = rot >> 1;
    for (int x = tid; x < nr * half_rot; x += kThreads) {
        const int row = x / half_rot, m = x - row * half_rot;
        const RowInfo f = s_row[row];
        if (!(f.flags & 1)) continue;
        const int pos = p.pos ? __ldg(p.pos + r0 + row) : f.j;
        double t = (double)pos * p.rope.turns[m];
        t -= rint(t);
        if constexpr (KV4) {
            double sn, cs;
            sincospi(2.0 * t, &sn, &cs);
            s_csd[row][m] = make_double2((double)p.rope.gain * cs, (double)p.rope.gain * sn);
            s_cs[row][m] = make_float2((float)(p.rope.gain * cs), (float)(p.rope.gain * sn));
        } else {
            float sn, cs;
            sincospif((float)(2.0 * t), &sn, &cs);
            const float g = (float)p.rope.gain;
            s_cs[row][m] = make_float2(g * cs, g * sn);
        }
    }
    __syncthreads();

    const bool half = p.rope.layout == SD_ROPE_HALF;
    const T *qin = static_cast<const T *>(p.q), *kin = static_cast<const T *>(p.k),
            *vin = static_cast<const T *>(p.v);
    // Channels of the two chunks of unit u: both elements of every pair of a rotated unit.
    auto chunks = [&](int u, bool rotated, int &oa, int &ob) {
        if (rotated && half) {
            if (u * 2 * VEC < rot) {
                oa = u * VEC;
                ob = oa + half_rot;
            } else {
                oa = u * 2 * VEC;
                ob = oa + VEC;
            }
        } else {
            oa = u * 2 * VEC;
            ob = oa + VEC;
        }
    };
    // Pair m of unit u in a / b: element indexes through f(a, b, m)
    auto turn = [&](int u, int oa, auto &&f) {
        if (half || VEC == 1) {
            if (u * 2 * VEC < rot)
#pragma unroll
                for (int e = 0; e < VEC; ++e) f(e, VEC + e, half ? oa + e : u);
        } else {
#pragma unroll
            for (int e = 0; e < 2 * VEC; e += 2)
                if (oa + e < rot) f(e, e + 1, (oa + e) >> 1);
        }
    };
    // heads handled by units: queries, then (dense caches, or wide chunks) keys and values
    constexpr bool kKvUnits = !(KV4 && VEC == 1);
    const int heads = p.h_q + (kKvUnits ? 2 * p.h_kv : 0);
    const int per_row = heads * UH;
    for (int x = tid; x < nr * per_row; x += kThreads) {
        const int row = x / per_row, y = x - row * per_row;
        const int hd = y / UH, u = y % UH;
        const RowInfo f = s_row[row];
        const int64_t r = r0 + row;
        const bool is_q = hd < p.h_q, is_k = !is_q && hd < p.h_q + p.h_kv;
        if (!(f.flags & (is_q ? 1 : 2))) continue;
        const int h = is_q ? hd : is_k ? hd - p.h_q : hd - p.h_q - p.h_kv;
        const T *src = is_q   ? qin + r * p.q_stride + (int64_t)h * D
                       : is_k ? kin + r * p.k_stride + (int64_t)h * D
                              : vin + r * p.v_stride + (int64_t)h * D;
        int oa, ob;
        chunks(u, is_q || is_k, oa, ob);
        P ab[2];
        ab[0] = *reinterpret_cast<const P *>(src + oa);
        ab[1] = *reinterpret_cast<const P *>(src + ob);
        auto at = [&](int e) -> T & { return ab[e / VEC].x[e % VEC]; };
        if (is_q || (is_k && !KV4)) {
            turn(u, oa, [&](int ea, int eb, int m) {
                const float2 cs = s_cs[row][m];
                const float a = to_f<T>(at(ea)), c = to_f<T>(at(eb));
                at(ea) = from_f<T>(a * cs.x - c * cs.y);
                at(eb) = from_f<T>(c * cs.x + a * cs.y);
            });
        }
        if (is_q || !KV4) {
            T *dst;
            if (is_q) {
                dst = static_cast<T *>(p.q_out) + (r * p.h_q + h) * D;
            } else {
                const int64_t o = p.page_size
                                      ? (((int64_t)f.page * p.h_kv + h) * kPageSize + (f.j & 15)) * D
                                      : (int64_t)f.b * p.stride_b + (int64_t)h * p.stride_h +
                                            (int64_t)f.j * D;
                dst = static_cast<T *>(is_k ? p.k_cache : p.v_cache) + o;
            }
            *reinterpret_cast<P *>(dst + oa) = ab[0];
            *reinterpret_cast<P *>(dst + ob) = ab[1];
        } else if constexpr (KV4 && VEC > 1) {
            if (is_k) {
                turn(u, oa, [&](int ea, int eb, int m) {
                    const double2 cs = s_csd[row][m];
                    const double a = to_f<T>(at(ea)), c = to_f<T>(at(eb));
                    at(ea) = from_f<T>((float)(a * cs.x - c * cs.y));
                    at(eb) = from_f<T>((float)(c * cs.x + a * cs.y));
                });
            }
            float mn = INFINITY, mx = -INFINITY, zero = 0.f;
#pragma unroll
            for (int e = 0; e < 2 * VEC; ++e) {
                const float v = to_f<T>(at(e));
                mn = fminf(mn, v);
                mx = fmaxf(mx, v);
                zero += v * 0.f;  // NaN once any element is not finite
            }
            // the UH lanes of the head (aligned groups: every loop count is a multiple of UH)
            const unsigned group = (UH == 32 ? 0xffffffffu : ((1u << UH) - 1u) << (lane & ~(UH - 1)));
#pragma unroll
            for (int o = UH / 2; o > 0; o >>= 1) {
                mn = fminf(mn, __shfl_xor_sync(group, mn, o));
                mx = fmaxf(mx, __shfl_xor_sync(group, mx, o));
            }
            const bool bad = (__ballot_sync(group, zero != 0.f) & group) != 0u;
            float s, lo;
            row_params<T>(mn, mx, bad, s, lo);
            const float inv = 1.f / s;
            const int64_t rw = p.page_size ? ((int64_t)f.page * p.h_kv + h) * kPageSize + (f.j & 15)
                                           : (int64_t)f.b * p.stride_b + (int64_t)h * p.stride_h + f.j;
            unsigned char *codes = static_cast<unsigned char *>(is_k ? p.k_cache : p.v_cache);
            T *vals = static_cast<T *>(is_k ? p.k_out : p.v_out);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t w = 0;
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    const float k = code_of(to_f<T>(ab[c].x[e]), s, lo, inv);
                    w |= (uint32_t)(int)k << (4 * e);
                    ab[c].x[e] = from_f<T>(fmaf(s, k, lo));
                }
                const int o = c ? ob : oa;
                unsigned char *cp = codes + rw * (D / 2) + o / 2;
                if constexpr (VEC == 8)
                    *reinterpret_cast<uint32_t *>(cp) = w;
                else
                    *reinterpret_cast<unsigned short *>(cp) = (unsigned short)w;
                if (vals) *reinterpret_cast<P *>(vals + (r * p.h_kv + h) * D + o) = ab[c];
            }
            if (u == 0) {
                (is_k ? p.k_param : p.v_param)[rw] = param_bits(s, lo);
                if (lo != lo) set_dev_err(p.dev_err, SD_DEVERR_NUMERIC);
            }
        }
    }
    if constexpr (KV4 && VEC == 1) {
        // Element-wise access: one warp per (row, K or V, head), the row's values through shared
        // memory so that each lane holds neighbouring channels when it packs codes.
        float *val = s_val[warp];
        constexpr int EL = D / 32;
        for (int x = warp; x < nr * 2 * p.h_kv; x += kThreads / 32) {
            const int row = x / (2 * p.h_kv), y = x - row * 2 * p.h_kv;
            const bool is_k = y < p.h_kv;
            const int h = is_k ? y : y - p.h_kv;
            const RowInfo f = s_row[row];
            if (!(f.flags & 2)) continue;
            const int64_t r = r0 + row;
            const T *src = is_k ? kin + r * p.k_stride + (int64_t)h * D
                                : vin + r * p.v_stride + (int64_t)h * D;
            for (int u = lane; u < UH; u += 32) {
                int oa, ob;
                chunks(u, is_k, oa, ob);
                float a = to_f<T>(src[oa]), c = to_f<T>(src[ob]);
                if (is_k && 2 * u < rot) {
                    const double2 cs = s_csd[row][u];
                    const double da = a, dc = c;
                    a = to_f<T>(from_f<T>((float)(da * cs.x - dc * cs.y)));
                    c = to_f<T>(from_f<T>((float)(dc * cs.x + da * cs.y)));
                }
                val[oa] = a;
                val[ob] = c;
            }
            __syncwarp();
            float v[EL], mn = INFINITY, mx = -INFINITY, zero = 0.f;
#pragma unroll
            for (int e = 0; e < EL; ++e) {
                v[e] = val[lane * EL + e];
                mn = fminf(mn, v[e]);
                mx = fmaxf(mx, v[e]);
                zero += v[e] * 0.f;
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
            const float inv = 1.f / s;
            const int64_t rw = p.page_size ? ((int64_t)f.page * p.h_kv + h) * kPageSize + (f.j & 15)
                                           : (int64_t)f.b * p.stride_b + (int64_t)h * p.stride_h + f.j;
            uint32_t w = 0;
            T *vals = static_cast<T *>(is_k ? p.k_out : p.v_out);
#pragma unroll
            for (int e = 0; e < EL; ++e) {
                const float k = code_of(v[e], s, lo, inv);
                w |= (uint32_t)(int)k << (4 * e);
                if (vals) vals[(r * p.h_kv + h) * D + lane * EL + e] = from_f<T>(fmaf(s, k, lo));
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

template <typename T, int D, int VEC>
cudaError_t launch_t(const AppendParams &p, cudaStream_t s) {
    const int blocks = (p.n_rows + p.rows_per_block - 1) / p.rows_per_block;
    return p.kv4 ? launch_pdl(append_kernel<T, D, VEC, true>, dim3(blocks), dim3(kThreads), 0, s, p)
                 : launch_pdl(append_kernel<T, D, VEC, false>, dim3(blocks), dim3(kThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_append(AppendParams p, bool wide, cudaStream_t s) {
    // one row per block while that leaves SMs free, else four (their cosines and sines then fill
    // a block's threads once)
    p.rows_per_block = p.n_rows <= 2 * device_sm_count() ? 1 : kMaxRows;
    const bool bf = p.dtype == SD_BF16;
    // 16-byte chunks need both chunks of a rotated unit aligned
    const int vec = bf ? 8 : 4;
    if (p.rope.layout == SD_ROPE_HALF && p.rope.rotary_dim % (2 * vec) != 0) wide = false;
    if (bf) {
        if (p.head_dim == 128)
            return wide ? launch_t<unsigned short, 128, 8>(p, s) : launch_t<unsigned short, 128, 1>(p, s);
        return wide ? launch_t<unsigned short, 64, 8>(p, s) : launch_t<unsigned short, 64, 1>(p, s);
    }
    if (p.head_dim == 128) return wide ? launch_t<float, 128, 4>(p, s) : launch_t<float, 128, 1>(p, s);
    return wide ? launch_t<float, 64, 4>(p, s) : launch_t<float, 64, 1>(p, s);
}

}  // namespace sd
