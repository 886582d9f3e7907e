// Tensor-core attention over a 4-bit cache for few rows per KV head (decoding, short drafts):
// up to 16 rows (heads of the group x query rows), bf16.
//
// Mathematics.  A key is lo + s c with codes c = 0..15, so
//     q . k = s (sum_e q_e (16 + c_e)) + (lo - 16 s) sum_e q_e
// and the sum over channels is one bf16 product of the query with 16 + c, which a code becomes by
// one shift and one and-or: bf16 16.0 has its four highest mantissa bits free, 0x4180 | c << 3.
// No multiplication and no rounding (q and 16 + c are exact in bf16).  For the values
//     sum_j p_j v_j = sum_j bf16(p_j s_j) (c_j - 8) + sum_j p_j (lo_j + 8 s_j)
// with 16 + c - 24 = c - 8 exact too; V's scale is folded into the softmax weight, which is
// rounded to bf16 for the product (a rounding that the bf16 cache's kernels make as well), and
// codes are centred so that the weight's rounding acts on values no larger than v itself.
//
// Layout.  Everything is transposed: S^T = K Q^T and O^T = V^T P^T by mma.sync m16n8k16 with 16
// positions (S) or 16 channels (O) as M and 8 rows as N, because few rows would leave most of an
// M = 128 tcgen05 tile (or an M = 16 row tile) empty, and because the operand that has to be
// expanded from codes is then A, whose fragments are expanded in registers straight from the
// codes' 16-byte chunks: nothing is ever written back to shared memory.  A head's channels are
// assigned to k indexes, and positions to m indexes, so that a lane's codes are neighbours in
// memory: lane (g, t) holds channels [D/4 t, D/4 (t+1)) of two positions for S, and channels
// [D/8 g, D/8 (g+1)) of four positions for O.  P^T moves from accumulator to operand layout by
// one 8x8 transpose per 8 positions.  (mma.sync runs at 1,024 products per cycle per SM here, a
// quarter of tcgen05's rate; at 8 rows that is a third of the time that a tile takes from HBM.)
//
// Work.  Two CTAs of 8 warps per SM; the CTAs share all units' tiles evenly (kv4_common.cuh) and
// of a tile every warp takes 16 positions, one page.  Each warp streams its own positions through
// its own ring of cp.async stages, with its page numbers looked up one stage further ahead, and
// keeps its own running maximum, sums and O^T; there is no block-wide step until a unit ends,
// where the warps are merged pairwise through shared memory.  The maximum moves only when a score
// exceeds it by more than 2^8 (one vote per 16 positions; the weights stay below 256).
#include "kv4_common.cuh"
#include "tc_ptx.cuh"

namespace sd {
namespace {

using tc::ex2;
using tc::pack_bf16;
using tc::saddr;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kCtasPerSm = 2;
constexpr float kGrow = 8.0f;
static_assert(kWarps * kPageSize == kKv4Tile, "a tile is one page per warp");

template <int D, int NT>
struct MmaCfg {
    static constexpr int kRow = D / 2;                    // bytes of a row's codes
    static constexpr int kBlock = kPageSize * kRow;       // codes of one warp's positions
    static constexpr int kStageBytes = 2 * kBlock + 128;  // K, V, parameters
    static constexpr int kStages = 4;
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    static constexpr int kMt = D / 16;                    // channel tiles of O^T
    static constexpr int kOFloats = kMt * NT * 4;         // O^T values of a lane
    static constexpr int kPart = (kOFloats + 6 * NT) * 32;  // floats of one warp's partial
    static constexpr int kSmem = kRing + kWarps / 2 * kPart * 4;
};

__device__ __forceinline__ void cp_async16z(uint32_t dst, const void *src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
}
__device__ __forceinline__ void cp_async4z(uint32_t dst, const void *src, int n) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n)
                 : "memory");
}

// (x & 0x00780078) | 0x41804180: a pair of codes at bits 3..6 of both halves to bf16 16 + c
__device__ __forceinline__ uint32_t code_pair(uint32_t x) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(x), "r"(0x00780078u), "r"(0x41804180u));
    return r;
}
// codes at nibble p (0..3) of both halves of w
template <int P>
__device__ __forceinline__ uint32_t codes_at(uint32_t w) {
    return code_pair(P == 0 ? w << 3 : w >> (P == 0 ? 0 : 4 * P - 3));
}
__device__ __forceinline__ uint32_t sub24(uint32_t x) {
    const __nv_bfloat162 c = __floats2bfloat162_rn(24.f, 24.f);
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&x), c);
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// m index of position r of a warp's 16: rows t, 4+t, 8+t, 12+t are m = 2t, 2t+1, 2t+8, 2t+9, so
// that the four positions of a V fragment are rows apart by 4 and a quarter-warp reads whole rows
__device__ __forceinline__ int m_of(int r) { return (r & 8) | ((r & 3) << 1) | ((r >> 2) & 1); }
__device__ __forceinline__ int pos_of(int m) { return (m & 8) | ((m & 1) << 2) | ((m >> 1) & 3); }

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) kv4_mma_kernel(const __grid_constant__ Kv4Params p) {
    pdl_trigger();  // (see launch_pdl)
    pdl_wait();
    using C = MmaCfg<D, NT>;
    constexpr unsigned FULL = 0xffffffffu;
    constexpr int kS = C::kStages;
    constexpr int kKs = D / 16;  // k steps of S^T, and channel tiles of O^T
    constexpr int kW = D / 32;   // 8-code words of a lane's share of a key
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long s_red[2 * kThreads / 32];
    __shared__ Kv4Start s_start;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gq = lane >> 2, t4 = lane & 3;

    long long lo, hi;
    Kv4Cursor cc = kv4_first<kThreads>(p, s_red, &s_start, lo, hi);  // next tile to compute
    if (hi <= lo) return;
    Kv4Cursor pc = cc;  // next tile to copy
    const int n_my = (int)(hi - lo);

    const uint32_t ring = saddr(smem) + warp * kS * C::kStageBytes;
    // Page of the warp's positions of cursor c (contiguous caches: 0); -1: nothing to read.
    auto page_of = [&](const Kv4Cursor &c) {
        const int j0 = c.t * kKv4Tile + warp * kPageSize;
        if (j0 >= c.kv_len) return -1;
        return p.page_size ? __ldg(p.block_table + (int64_t)c.b * p.max_pages + (j0 >> 4)) : 0;
    };
    int page = page_of(pc);
    int copied = 0;
    auto copy_next = [&]() {
        if (copied < n_my) {
            const int j0 = pc.t * kKv4Tile + warp * kPageSize;
            int n = pc.kv_len - j0;  // positions of this block
            if (n > 0) {
                int64_t row0 = (int64_t)pc.b * p.stride_b + (int64_t)pc.g * p.stride_h + j0;
                if (p.page_size) {
                    row0 = ((int64_t)page * p.h_kv + pc.g) * kPageSize;
                    if (page < 0 || page >= p.num_pages) {
                        if (lane == 0) set_dev_err(p.dev_err, SD_DEVERR_PAGE);
                        n = 0;  // (zeros, as the bf16 kernels' out-of-range boxes)
                        row0 = 0;
                    }
                }
                const uint32_t dst = ring + (copied % kS) * C::kStageBytes;
#pragma unroll
                for (int i = 0; i < C::kBlock / 512; ++i) {
                    const int x = lane + 32 * i;
                    const int r = x / (C::kRow / 16), q = x % (C::kRow / 16);
                    const bool in = r < n;
                    const int64_t off = (row0 + (in ? r : 0)) * C::kRow + q * 16;
                    cp_async16z(dst + m_of(r) * C::kRow + q * 16, p.k + off, in ? 16 : 0);
                    const int qv = D == 128 ? q ^ (r & 2) : q;
                    cp_async16z(dst + C::kBlock + r * C::kRow + qv * 16, p.v + off, in ? 16 : 0);
                }
                const int r = lane & 15;
                const bool in = r < n;
                cp_async4z(dst + 2 * C::kBlock + (lane & 16) * 4 + m_of(r) * 4,
                           (lane < 16 ? p.kp : p.vp) + row0 + (in ? r : 0), in ? 4 : 0);
            }
            ++copied;
            pc.next(p);
            if (copied < n_my) page = page_of(pc);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kS - 1; ++i) copy_next();

    int done = 0;
    while (done < n_my) {
        // ---- a unit's share: tiles [cc.t, cc.t + n_seg) of unit (cc.b, cc.g) ----
        const int n_seg = min(cc.tiles - cc.t, n_my - done);
        const bool starts = cc.t == 0, ends = cc.t + n_seg == cc.tiles;
        const int G = p.group, R = cc.n_q * G, kv_len = cc.kv_len;
        // the last position that query row 0 sees: blocks up to it need no mask
        const int first_limit = kv_len - cc.n_q;
        uint32_t qb[NT][kKs][2];
        float qs[NT][2];   // sum of a column's query channels
        int limit[NT][2];  // last visible position of columns 2t, 2t + 1
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = nt * 8 + gq;
            const uint4 *src = reinterpret_cast<const uint4 *>(
                static_cast<const unsigned short *>(p.q) +
                ((int64_t)(cc.q0 + (r < R ? r / G : 0)) * p.h_q + cc.g * G + (r < R ? r % G : 0)) * D +
                t4 * (D / 4));
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                const uint4 x = r < R ? __ldg(src + w) : make_uint4(0u, 0u, 0u, 0u);
                qb[nt][2 * w][0] = __byte_perm(x.x, x.z, 0x5410);
                qb[nt][2 * w][1] = __byte_perm(x.x, x.z, 0x7632);
                qb[nt][2 * w + 1][0] = __byte_perm(x.y, x.w, 0x5410);
                qb[nt][2 * w + 1][1] = __byte_perm(x.y, x.w, 0x7632);
                sum += bf16_lo(x.x) + bf16_hi(x.x) + bf16_lo(x.y) + bf16_hi(x.y) + bf16_lo(x.z) +
                       bf16_hi(x.z) + bf16_lo(x.w) + bf16_hi(x.w);
            }
            sum += __shfl_xor_sync(FULL, sum, 1);
            sum += __shfl_xor_sync(FULL, sum, 2);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                qs[nt][c] = __shfl_sync(FULL, sum, (2 * t4 + c) * 4);
                const int n = nt * 8 + 2 * t4 + c;
                limit[nt][c] = n < R ? first_limit + n / G : -1;
            }
        }
        float o[kKs][NT][4], m[NT][2], l[NT][2], cr[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int mt = 0; mt < kKs; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                m[nt][c] = -INFINITY;
                l[nt][c] = cr[nt][c] = 0.f;
            }
        }
        for (int it = 0; it < n_seg; ++it, ++done) {
            copy_next();
            cp_async_wait<kS - 1>();
            __syncwarp();
            const int j0 = (cc.t + it) * kKv4Tile + warp * kPageSize;
            if (j0 < kv_len) {
                const uint8_t *st = smem + (warp * kS + done % kS) * C::kStageBytes;
                // ---- S^T = K Q^T ----
                uint32_t kw[2][kW];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint8_t *src = st + (gq + 8 * i) * C::kRow + t4 * (C::kRow / 4);
                    if constexpr (D == 128) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(src);
                        kw[i][0] = x.x;
                        kw[i][1] = x.y;
                        kw[i][kW - 2] = x.z;
                        kw[i][kW - 1] = x.w;
                    } else {
                        const uint2 x = *reinterpret_cast<const uint2 *>(src);
                        kw[i][0] = x.x;
                        kw[i][1] = x.y;
                    }
                }
                float s[NT][4], s2[NT][4];  // two chains of products
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[nt][e] = s2[nt][e] = 0.f;
#pragma unroll
                for (int w = 0; w < kW; ++w) {
                    const uint32_t a0 = codes_at<0>(kw[0][w]), a1 = codes_at<0>(kw[1][w]);
                    const uint32_t a2 = codes_at<1>(kw[0][w]), a3 = codes_at<1>(kw[1][w]);
                    const uint32_t b0 = codes_at<2>(kw[0][w]), b1 = codes_at<2>(kw[1][w]);
                    const uint32_t b2 = codes_at<3>(kw[0][w]), b3 = codes_at<3>(kw[1][w]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma16816(s[nt], a0, a1, a2, a3, qb[nt][2 * w][0], qb[nt][2 * w][1]);
                        mma16816(s2[nt], b0, b1, b2, b3, qb[nt][2 * w + 1][0], qb[nt][2 * w + 1][1]);
                    }
                }
                const uint32_t *par = reinterpret_cast<const uint32_t *>(st + 2 * C::kBlock);
                const uint32_t kp0 = par[gq], kp1 = par[gq + 8];
                const uint32_t vp0 = par[16 + gq], vp1 = par[24 + gq];
                // scores in log2 units: s[0], s[1] at position pos_of(g), s[2], s[3] at g + 8
                const float ks0 = param_scale(kp0) * p.scale_log2, ks1 = param_scale(kp1) * p.scale_log2;
                const float kl0 = fmaf(param_low(kp0), p.scale_log2, -16.f * ks0);
                const float kl1 = fmaf(param_low(kp1), p.scale_log2, -16.f * ks1);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        s[nt][c] = fmaf(ks0, s[nt][c] + s2[nt][c], kl0 * qs[nt][c]);
                        s[nt][2 + c] = fmaf(ks1, s[nt][2 + c] + s2[nt][2 + c], kl1 * qs[nt][c]);
                    }
                const bool whole = j0 + kPageSize - 1 <= first_limit;
                const int pa = j0 + pos_of(gq), pb = pa + 8;
                if (!whole) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            if (pa > limit[nt][c]) s[nt][c] = -INFINITY;
                            if (pb > limit[nt][c]) s[nt][2 + c] = -INFINITY;
                        }
                }
                bool grow = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        grow |= fmaxf(s[nt][c], s[nt][2 + c]) > m[nt][c] + kGrow;
                if (__any_sync(FULL, grow)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float f[2];
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float x = fmaxf(s[nt][c], s[nt][2 + c]);
                            x = fmaxf(x, __shfl_xor_sync(FULL, x, 4));
                            x = fmaxf(x, __shfl_xor_sync(FULL, x, 8));
                            x = fmaxf(x, __shfl_xor_sync(FULL, x, 16));
                            x = fmaxf(x, m[nt][c]);
                            f[c] = x == -INFINITY ? 1.f : ex2(m[nt][c] - x);
                            m[nt][c] = x;
                            l[nt][c] *= f[c];
                            cr[nt][c] *= f[c];
                        }
#pragma unroll
                        for (int mt = 0; mt < kKs; ++mt)
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[mt][nt][e] *= f[e & 1];
                    }
                }
                // ---- weights, and P^T in operand layout ----
                const float vs0 = param_scale(vp0), vs1 = param_scale(vp1);
                const float vl0 = fmaf(8.f, vs0, param_low(vp0)), vl1 = fmaf(8.f, vs1, param_low(vp1));
                uint32_t pt[NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float w0[2], w1[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float base = m[nt][c] == -INFINITY ? 0.f : m[nt][c];
                        const float e0 = ex2(s[nt][c] - base), e1 = ex2(s[nt][2 + c] - base);
                        l[nt][c] += e0 + e1;
                        w0[c] = e0 * vs0;
                        w1[c] = e1 * vs1;
                        float k0 = e0 * vl0, k1 = e1 * vl1;
                        if (!whole) {  // a hidden position's NaN must not get through
                            if (pa > limit[nt][c]) w0[c] = k0 = 0.f;
                            if (pb > limit[nt][c]) w1[c] = k1 = 0.f;
                        }
                        cr[nt][c] += k0 + k1;
                    }
                    pt[nt][0] = transpose8(pack_bf16(w0[0], w0[1]));
                    pt[nt][1] = transpose8(pack_bf16(w1[0], w1[1]));
                }
                // ---- O^T += V^T P^T ----
                constexpr int kVw = D / 64;  // words of a lane's 8-channel groups per position
                uint32_t vw[4][kVw];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = t4 + 4 * i;
                    if constexpr (D == 128) {
                        const int q = (gq >> 1) ^ (r & 2);
                        const uint2 x = *reinterpret_cast<const uint2 *>(
                            st + C::kBlock + r * C::kRow + q * 16 + (gq & 1) * 8);
                        vw[i][0] = x.x;
                        vw[i][kVw - 1] = x.y;
                    } else {
                        vw[i][0] = *reinterpret_cast<const uint32_t *>(st + C::kBlock +
                                                                       r * C::kRow + gq * 4);
                    }
                }
                // channel D/8 g + 8 w + 4 h + c: tile 4 w + 2 h + c / 2, row g + 8 (c & 1)
#pragma unroll
                for (int w = 0; w < kVw; ++w)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t x = __byte_perm(vw[0][w], vw[1][w], h ? 0x7632 : 0x5410);
                        const uint32_t y = __byte_perm(vw[2][w], vw[3][w], h ? 0x7632 : 0x5410);
                        const uint32_t a0 = sub24(codes_at<0>(x)), a1 = sub24(codes_at<1>(x));
                        const uint32_t a2 = sub24(codes_at<0>(y)), a3 = sub24(codes_at<1>(y));
                        const uint32_t b0 = sub24(codes_at<2>(x)), b1 = sub24(codes_at<3>(x));
                        const uint32_t b2 = sub24(codes_at<2>(y)), b3 = sub24(codes_at<3>(y));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma16816(o[4 * w + 2 * h][nt], a0, a1, a2, a3, pt[nt][0], pt[nt][1]);
                            mma16816(o[4 * w + 2 * h + 1][nt], b0, b1, b2, b3, pt[nt][0], pt[nt][1]);
                        }
                    }
            }
            __syncwarp();  // (the stage's next copies)
        }
        // ---- end of the share: merge the warps ----
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) {
                    l[nt][c] += __shfl_xor_sync(FULL, l[nt][c], x);
                    cr[nt][c] += __shfl_xor_sync(FULL, cr[nt][c], x);
                }
                // (a sum that is NaN needs a finite maximum to survive a merge)
                if (l[nt][c] != l[nt][c] && m[nt][c] == -INFINITY) m[nt][c] = 0.f;
            }
        float *part = reinterpret_cast<float *>(smem + C::kRing);
#pragma unroll
        for (int half = kWarps / 2; half > 0; half >>= 1) {
            if (warp >= half && warp < 2 * half) {
                float *d = part + (warp - half) * C::kPart + lane;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                    for (int mt = 0; mt < kKs; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) d[((mt * NT + nt) * 4 + e) * 32] = o[mt][nt][e];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        d[(C::kOFloats + nt * 6 + c) * 32] = m[nt][c];
                        d[(C::kOFloats + nt * 6 + 2 + c) * 32] = l[nt][c];
                        d[(C::kOFloats + nt * 6 + 4 + c) * 32] = cr[nt][c];
                    }
                }
            }
            __syncthreads();
            if (warp < half) {
                const float *d = part + warp * C::kPart + lane;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float f0[2], f1[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const float m1 = d[(C::kOFloats + nt * 6 + c) * 32];
                        const float M = fmaxf(m[nt][c], m1);
                        f0[c] = m[nt][c] == -INFINITY ? 0.f : ex2(m[nt][c] - M);
                        f1[c] = m1 == -INFINITY ? 0.f : ex2(m1 - M);
                        m[nt][c] = M;
                        l[nt][c] = f0[c] * l[nt][c] + f1[c] * d[(C::kOFloats + nt * 6 + 2 + c) * 32];
                        cr[nt][c] = f0[c] * cr[nt][c] + f1[c] * d[(C::kOFloats + nt * 6 + 4 + c) * 32];
                    }
#pragma unroll
                    for (int mt = 0; mt < kKs; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[mt][nt][e] = f0[e & 1] * o[mt][nt][e] +
                                           f1[e & 1] * d[((mt * NT + nt) * 4 + e) * 32];
                }
            }
            __syncthreads();
        }
        if (warp == 0) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int n = nt * 8 + 2 * t4 + c;
                    if (n >= R) continue;
                    // this lane's channels [D/8 g, D/8 (g + 1)) of column n, in order
                    float x[D / 8];
#pragma unroll
                    for (int mt = 0; mt < kKs; ++mt) {
                        x[2 * mt] = o[mt][nt][c] + cr[nt][c];
                        x[2 * mt + 1] = o[mt][nt][2 + c] + cr[nt][c];
                    }
                    if (starts && ends) {
                        const float inv = l[nt][c] == 0.f ? 0.f : 1.f / l[nt][c];
                        uint4 *dst = reinterpret_cast<uint4 *>(
                            static_cast<unsigned short *>(p.out) +
                            ((int64_t)(cc.q0 + n / G) * p.h_q + cc.g * G + n % G) * D + gq * (D / 8));
#pragma unroll
                        for (int i = 0; i < D / 64; ++i)
                            dst[i] = make_uint4(pack_bf16(x[8 * i] * inv, x[8 * i + 1] * inv),
                                                pack_bf16(x[8 * i + 2] * inv, x[8 * i + 3] * inv),
                                                pack_bf16(x[8 * i + 4] * inv, x[8 * i + 5] * inv),
                                                pack_bf16(x[8 * i + 6] * inv, x[8 * i + 7] * inv));
                    } else {
                        const int64_t slot = 2 * (int64_t)blockIdx.x + (starts ? 1 : 0);
                        float4 *dst = reinterpret_cast<float4 *>(kv4_slot_o(p, slot, n) + gq * (D / 8));
#pragma unroll
                        for (int i = 0; i < D / 32; ++i)
                            dst[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                        if (gq == 0) {
                            float *ml = kv4_slot_ml(p, slot, n);
                            ml[0] = m[nt][c];
                            ml[1] = l[nt][c];
                        }
                    }
                }
        }
        cc.skip(p, n_seg);
    }
    cp_async_wait<0>();
}

template <int D, int NT>
cudaError_t launch_t(const Kv4Params &p, cudaStream_t s) {
    constexpr int bytes = MmaCfg<D, NT>::kSmem;
    cudaError_t e = set_max_dynamic_smem<kv4_mma_kernel<D, NT>>(bytes);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kv4_mma_kernel<D, NT>, dim3(p.ctas), dim3(kThreads), bytes, s, p);
    return e != cudaSuccess ? e : launch_kv4_merge(p, s);
}

}  // namespace

int kv4_mma_max_rows() { return 16; }

// CTAs of a launch: no more than the tiles that the hints allow.
int kv4_mma_ctas(int batch, int h_kv, int max_kv_len) {
    const long long tiles = (long long)batch * h_kv * (((long long)max_kv_len + kKv4Tile - 1) / kKv4Tile);
    const long long g = (long long)device_sm_count() * kCtasPerSm;
    return (int)(tiles < g ? tiles : g);
}

cudaError_t launch_kv4_mma(const Kv4Params &p, cudaStream_t s) {
    const bool one = p.group * p.max_q_rows <= 8;
    if (p.head_dim == 128) return one ? launch_t<128, 1>(p, s) : launch_t<128, 2>(p, s);
    return one ? launch_t<64, 1>(p, s) : launch_t<64, 2>(p, s);
}

}  // namespace sd
