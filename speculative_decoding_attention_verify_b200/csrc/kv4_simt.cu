// CUDA-core attention over a 4-bit cache: fp32 rows, and the shapes that the tensor-core kernels
// do not take (more than 128 rows per KV head, rows that are not 16-byte aligned).
//
// One CTA per (split of the positions, block of 8 rows, KV head, sequence).  Tiles of 64
// positions are expanded once to fp32 in shared memory and used by the 8 rows: a thread forms
// the scores of one position with 4 rows, the warps keep a running maximum and sum of 2 rows
// each, and a thread owns one channel of the output.  Everything is fp32.  Bound by its shared
// memory reads (a K and a V value each serve 4 or 8 rows); the splits are joined by
// kv4_merge_kernel.
// Far slower than the tensor-core kernels: 4 sequences of 10,000 positions, 4 KV heads, fp32: 7 rows
// 110 us, 63 rows 814; 2 sequences of 26,043 positions and 133 bf16 rows 2.0 ms.
#include "kv4_common.cuh"

namespace sd {
namespace {

constexpr int kThreads = 128;
constexpr int kTile = 64;
constexpr int kRB = 8;  // rows per block

template <typename T>
__device__ __forceinline__ float row_value(const void *p, int64_t i) {
    if constexpr (sizeof(T) == 4) return static_cast<const float *>(p)[i];
    return __uint_as_float((uint32_t) static_cast<const unsigned short *>(p)[i] << 16);
}

template <int D>
struct SimtSmem {
    float q[kRB][D];
    float k[kTile][D + 1];  // (+1: neighbouring positions in different banks)
    float v[kTile][D];
    float p[kRB][kTile];
    float m[kRB], l[kRB], corr[kRB];
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_simt_kernel(const Kv4Params p, int row_blocks) {
    pdl_trigger();  // (see launch_pdl)
    pdl_wait();
    extern __shared__ float4 smem_raw[];
    SimtSmem<D> &s = *reinterpret_cast<SimtSmem<D> *>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int split = blockIdx.x / row_blocks, rb = blockIdx.x % row_blocks;
    const int g = blockIdx.y, b = blockIdx.z, G = p.group;
    int q0, n_q, kv_len;
    bool bad;
    if (!kv4_sequence(p, b, q0, n_q, kv_len, bad)) {
        if (bad && tid == 0) set_dev_err(p.dev_err, SD_DEVERR_SHAPE);
        return;
    }
    const int R = n_q * G;
    if (rb * kRB >= R) return;
    const int tiles = (kv_len + kTile - 1) / kTile;
    const int t_lo = (int)((int64_t)tiles * split / p.n_splits);
    const int t_hi = (int)((int64_t)tiles * (split + 1) / p.n_splits);
    for (int x = tid; x < kRB * D; x += kThreads) {
        const int r = rb * kRB + x / D;
        s.q[x / D][x % D] =
            r < R ? row_value<T>(p.q, ((int64_t)(q0 + r / G) * p.h_q + g * G + r % G) * D + x % D)
                  : 0.f;
    }
    if (tid < kRB) {
        s.m[tid] = -INFINITY;
        s.l[tid] = 0.f;
    }
    constexpr int kCols = kThreads / D;  // threads per channel (each a share of the rows)
    constexpr int kOwn = kRB / kCols;    // rows of one thread's channel
    const int col = tid % D, r_own = (tid / D) * kOwn;
    float acc[kOwn];
    int limit_own[kOwn];  // the rows' last visible positions; rows past R see nothing
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const int r = rb * kRB + r_own + i;
        acc[i] = 0.f;
        limit_own[i] = r < R ? kv_len - n_q + r / G : -1;
    }
    for (int t = t_lo; t < t_hi; ++t) {
        const int base = t * kTile, n = min(kTile, kv_len - base);
        __syncthreads();  // the last tile's reads
        // expand: a thread takes 16 channels (8 bytes) of a position of K, then of V
        for (int x = tid; x < kTile * (D / 16); x += kThreads) {
            const int j = x / (D / 16), c = x % (D / 16);
            const int64_t row = j < n ? kv4_row(p, b, g, base + j) : -1;
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                float *dst = w ? &s.v[j][c * 16] : &s.k[j][c * 16];
                uint2 q = make_uint2(0u, 0u);
                uint32_t par = 0u;
                if (row >= 0) {
                    q = ld_dep(reinterpret_cast<const uint2 *>((w ? p.v : p.k) + row * (D / 2)) + c);
                    par = ld_dep((w ? p.vp : p.kp) + row);
                }
                const float sc = param_scale(par), lo = param_low(par);
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const uint32_t code = ((e < 8 ? q.x : q.y) >> (4 * (e & 7))) & 15u;
                    dst[e] = fmaf(sc, (float)code, lo);
                }
            }
        }
        __syncthreads();
        {
            const int j = tid % kTile, r4 = (tid / kTile) * 4;
            float d[4] = {0.f, 0.f, 0.f, 0.f};
            for (int e = 0; e < D; ++e) {
                const float k = s.k[j][e];
#pragma unroll
                for (int i = 0; i < 4; ++i) d[i] = fmaf(s.q[r4 + i][e], k, d[i]);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = rb * kRB + r4 + i;
                // (the row's last visible position; rows past R see nothing)
                const int limit = r < R ? kv_len - n_q + r / G : -1;
                s.p[r4 + i][j] = base + j <= limit ? d[i] * p.scale_log2 : -INFINITY;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRB / 4; ++i) {
            const int r = warp * (kRB / 4) + i;
            const float x0 = s.p[r][lane], x1 = s.p[r][lane + 32];
            const float m0 = s.m[r], m = fmaxf(m0, warp_max(fmaxf(x0, x1)));
            // A row that has seen nothing but NaN keeps m = -inf: its exponents stay NaN.
            const float base_m = m == -INFINITY ? 0.f : m;
            const float p0 = exp2f(x0 - base_m), p1 = exp2f(x1 - base_m);
            const float c = m0 == -INFINITY ? (m == -INFINITY ? 1.f : 0.f) : exp2f(m0 - base_m);
            s.p[r][lane] = p0;
            s.p[r][lane + 32] = p1;
            const float sum = warp_sum(p0 + p1);
            __syncwarp();
            if (lane == 0) {
                const float l0 = s.l[r];
                s.l[r] = (l0 == 0.f ? 0.f : l0 * c) + sum;
                s.m[r] = m;
                s.corr[r] = c;
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kOwn; ++i) acc[i] *= s.corr[r_own + i];
        // (a row that does not see a position must not see its NaN either)
        for (int j = 0; j < n; ++j) {
            const float v = s.v[j][col];
#pragma unroll
            for (int i = 0; i < kOwn; ++i)
                if (base + j <= limit_own[i]) acc[i] = fmaf(s.p[r_own + i][j], v, acc[i]);
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
        const int r = rb * kRB + r_own + i;
        if (r >= R) break;
        const int row = q0 + r / G, h = g * G + r % G;
        const float l = s.l[r_own + i], m = s.m[r_own + i];
        if (p.n_splits == 1) {
            const float o = l == 0.f ? 0.f : acc[i] / l;
            const int64_t at = ((int64_t)row * p.h_q + h) * D + col;
            if constexpr (sizeof(T) == 4)
                static_cast<float *>(p.out)[at] = o;
            else
                static_cast<unsigned short *>(p.out)[at] = (unsigned short)f32_to_bf16_bits(o);
        } else {
            const int64_t slot = ((int64_t)b * p.h_kv + g) * p.n_splits + split;
            kv4_slot_o(p, slot, r)[col] = acc[i];
            if (col == 0) {
                float *ml = kv4_slot_ml(p, slot, r);
                // (NaN sums need a finite maximum to survive the merge)
                ml[0] = l != l && m == -INFINITY ? 0.f : m;
                ml[1] = l;
            }
        }
    }
}

template <typename T, int D>
cudaError_t launch_t(const Kv4Params &p, cudaStream_t s) {
    const int bytes = (int)sizeof(SimtSmem<D>);
    cudaError_t e = set_max_dynamic_smem<kv4_simt_kernel<T, D>>(bytes);
    if (e != cudaSuccess) return e;
    const int row_blocks = (p.group * p.max_q_rows + kRB - 1) / kRB;
    e = launch_pdl(kv4_simt_kernel<T, D>, dim3(p.n_splits * row_blocks, p.h_kv, p.batch),
                   dim3(kThreads), bytes, s, p, row_blocks);
    if (e != cudaSuccess || p.n_splits == 1) return e;
    return launch_kv4_merge(p, s);
}

}  // namespace

// Splits of the CUDA-core engine: two CTAs of 128 threads per SM over the units (sequence, KV
// head, block of rows), at least two tiles each, at most 64.
int kv4_simt_splits(int batch, int h_kv, int rows, int max_kv_len) {
    const long long units = (long long)batch * h_kv * ((rows + kRB - 1) / kRB);
    const long long tiles = ((long long)max_kv_len + kTile - 1) / kTile;
    long long s = 2LL * device_sm_count() / units;
    if (s > tiles / 2) s = tiles / 2;
    return (int)(s < 1 ? 1 : s > 64 ? 64 : s);
}

cudaError_t launch_kv4_simt(const Kv4Params &p, cudaStream_t s) {
    if (p.dtype == SD_BF16)
        return p.head_dim == 128 ? launch_t<unsigned short, 128>(p, s)
                                 : launch_t<unsigned short, 64>(p, s);
    return p.head_dim == 128 ? launch_t<float, 128>(p, s) : launch_t<float, 64>(p, s);
}

}  // namespace sd
