// Tensor-core attention over a 4-bit cache for few rows per KV head (decoding, short drafts):
// up to 16 rows (heads of the group x query rows), bf16.
//
// Mathematics.  A key is lo + s c with codes c = 0..15, so
//     q . k = s (sum_e q_e c_e) + lo (sum_e q_e)
// and the sum over channels is one fp16 product of the query with the codes themselves: a code in
// the low bits of an fp16 word IS the number c 2^-24 (a subnormal; the tensor cores take those
// exactly), one in bits 4-7 is 16 c 2^-24.  So a pair of codes becomes an operand by one AND, after
// one shift by 8 for every second byte, with no conversion, no rounding and no offset to take away
// again.  The queries are scaled by a power of two per row (their largest to 2^13; bf16's 8 bits
// fit fp16's 11, and an element has to be 2^-27 of the row's largest to lose any) and the odd
// channels, whose codes sit in bits 4-7, by 1/16.  For the values
//     sum_j p_j v_j = sum_j (p_j s_j) (c_j - 8) + sum_j p_j (lo_j + 8 s_j)
// with w_j = p_j s_j taken as one exponential, w_j = 2^(x_j + log2 s_j - m), x_j the score in log2
// units and m a running maximum of the whole exponent.  w is rounded to fp16 (2^-11 of itself; see
// kTopLog2 for the smallest ones) and p = w / s is not rounded: it enters the sums of the
// softmax and of p lo in fp32.  Rows of one value (s = 0, codes 0) count with s = |lo| / 256 there,
// and no row with less than 2^-90: a sink of zeros, however large its p, then leaves the others'
// weights the whole range of fp16.  The products are with c, and 8 times the sum of the step's
// rounded weights (one more product, with ones) is taken from the accumulators after each step:
// the tensor core cuts towards zero as it accumulates, and the sum of w c would grow to hundreds
// of times what is left once lo's part is added (140,000 random positions: odd channels off by
// 6.7e-4 of themselves without, 1.7e-4 with).  Taking 8 from each code cost twice as much.  All of
// V's codes are moved to bits 4-7: the tensor core aligns a product by its factors' exponent fields,
// which for a subnormal say 2^-14, and cuts what lies 24 bits below the largest, so that codes in
// bits 0-3 lose four bits more than those in bits 4-7 (even channels off by 1.9e-3, now 1.9e-4; the
// scores' products, of factors that differ less, lose nothing that shows).
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
// Work.  The CTAs share all units' tiles evenly (kv4_common.cuh); of every tile each of a CTA's 8
// warps takes 32 positions (two pages) for all rows.  Each warp streams its positions through its
// own two cp.async stages, with its page numbers looked up a stage further ahead, and keeps its own
// running maxima, sums and O^T; there is no block-wide step until a unit ends, where the warps'
// shares are merged pairwise through shared memory.  Whether a maximum moves is one vote per 32
// positions.
// Query fragments are registers for up to 8 rows; for more they are read from shared memory, once
// for both pages.
// Measured: 28 sequences of 26,025 positions, 4 KV heads, 7 rows: 101 us, 3.9 TB/s (in pages 107); one
// sequence of 140,001 31.5 us.  With 16 warps per SM the ALU pipe is busy for 55% and issue slots
// for 57% (half the sequences: 315 instructions per page of a warp); warps wait for the pipe and for
// results in turn.  14 rows take 197 us: at 128 registers that kernel spills 524 bytes, and half of
// what its warps wait for is local memory (issue slots 40%).
#include <type_traits>

#include "kv4_common.cuh"
#include "tc_ptx.cuh"

namespace sd {
namespace {

using tc::ex2;
using tc::pack_bf16;
using tc::saddr;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kPos = 32;       // positions of a warp per tile
constexpr int kStages = 2;

constexpr int kTile = kWarps * kPos;
constexpr int kCtasPerSm = 2;  // registers of O^T decide
constexpr uint32_t kOnes = 0x3c003c00u;  // a pair of fp16 ones

template <int D, int NT>
struct MmaCfg {
    static constexpr int kRow = D / 2;                     // bytes of a row's codes
    static constexpr int kPage = kPageSize * kRow;         // codes of a page
    static constexpr int kPageBytes = 2 * kPage + 128;     // K, V, parameters
    static constexpr int kStageBytes = 2 * kPageBytes;
    static constexpr int kRing = kWarps * kStages * kStageBytes;
    static constexpr int kMt = D / 16;                     // channel tiles of O^T, k steps of S^T
    static constexpr int kOFloats = kMt * NT * 4;          // O^T values of a lane
    static constexpr int kPart = (kOFloats + 6 * NT) * 32;  // floats of one warp's partial
    // query fragments: registers for NT = 1
    static constexpr int kQ = kRing + kWarps / 2 * kPart * 4;
    static constexpr int kSmem = kQ + (NT == 1 ? 0 : NT * kMt * 256);
};
static_assert(kCtasPerSm * (MmaCfg<128, 2>::kSmem + 1024) <= 227 * 1024, "shared memory");

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Codes at nibble P (0..3) of both halves of w as a pair of fp16 numbers c / kVOne, all four at bits
// 4-7 of an operand.
constexpr float kVOne = 1048576.f;  // 2^20
template <int P>
__device__ __forceinline__ uint32_t high_codes_at(uint32_t w) {
    return (P == 0 ? w << 4 : P == 1 ? w : P == 2 ? w >> 4 : w >> 8) & 0x00f000f0u;
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
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
kv4_mma_kernel(const __grid_constant__ Kv4Params p) {
    pdl_trigger();  // (see launch_pdl)
    pdl_wait();
    using C = MmaCfg<D, NT>;
    constexpr unsigned FULL = 0xffffffffu;
    constexpr int kKs = C::kMt;
    constexpr int kW = D / 32;  // 8-code words of a lane's share of a key
    constexpr bool kQRegs = NT == 1;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long s_red[kThreads / 32];
    __shared__ Kv4Start s_start;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gq = lane >> 2, t4 = lane & 3;

    long long lo, hi;
    Kv4Cursor cc = kv4_first<kThreads>(p, s_red, &s_start, lo, hi);  // next tile to compute
    if (hi <= lo) return;
    Kv4Cursor pc = cc;  // next tile to copy
    const int n_my = (int)(hi - lo);

    // ---- copies ----
    const uint8_t *ring_p = smem + warp * kStages * C::kStageBytes;
    const uint32_t ring = saddr(ring_p);
    constexpr int Q = C::kRow / 16;  // 16-byte chunks of a row
    // Where 16-byte chunk x of a page's codes goes: K rows in fragment order; V rows in place, the
    // chunks of every second pair of rows swapped pairwise (a fragment's four rows then differ in
    // banks).
    auto k_at = [](int x) { return m_of(x / Q) * C::kRow + (x % Q) * 16; };
    auto v_at = [](int x) {
        const int r = x / Q;
        return C::kPage + r * C::kRow + (D == 128 ? (x % Q) ^ (r & 2) : x % Q) * 16;
    };
    const uint32_t par_at = 2 * C::kPage + (lane & 16) * 4 + m_of(lane & 15) * 4;
    const uint32_t *par_src = (lane < 16 ? p.kp : p.vp) + (lane & 15);
    int pages[2];
    auto look_up = [&]() {  // pages of the next tile to copy
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int j = pc.t * kTile + warp * kPos + i * kPageSize;
            pages[i] = p.page_size && j < pc.kv_len
                           ? ld_dep(p.block_table + (int64_t)pc.b * p.max_pages + (j >> 4))
                           : 0;
        }
    };
    look_up();
    int copied = 0;
    int64_t unit_row = (int64_t)pc.b * p.stride_b + (int64_t)pc.g * p.stride_h;  // (contiguous)
    auto copy_next = [&]() {
        if (copied < n_my) {
            const int j0 = pc.t * kTile + warp * kPos;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int j = j0 + i * kPageSize;
                int n = pc.kv_len - j;  // positions of this page
                if (n > 0) {
                    int64_t row0 = unit_row + j;
                    if (p.page_size) {
                        row0 = ((int64_t)pages[i] * p.h_kv + pc.g) * kPageSize;
                        if (pages[i] < 0 || pages[i] >= p.num_pages) {
                            if (lane == 0) set_dev_err(p.dev_err, SD_DEVERR_PAGE);
                            n = 0;  // (zeros, as the bf16 kernels' out-of-range boxes)
                            row0 = 0;
                        }
                    }
                    const uint32_t dst =
                        ring + (copied % kStages) * C::kStageBytes + i * C::kPageBytes;
                    if (n >= kPageSize) {
                        const int64_t off = row0 * C::kRow + lane * 16;
#pragma unroll
                        for (int k = 0; k < C::kPage / 512; ++k) {
                            cp_async16(dst + k_at(lane + 32 * k), p.k + off + 512 * k);
                            cp_async16(dst + v_at(lane + 32 * k), p.v + off + 512 * k);
                        }
                        cp_async4z(dst + par_at, par_src + row0, 4);
                    } else {  // the end of the sequence: zeros past it
#pragma unroll
                        for (int k = 0; k < C::kPage / 512; ++k) {
                            const int x = lane + 32 * k;
                            const bool in = x / Q < n;
                            const int64_t off = row0 * C::kRow + (in ? x : 0) * 16;
                            cp_async16z(dst + k_at(x), p.k + off, in ? 16 : 0);
                            cp_async16z(dst + v_at(x), p.v + off, in ? 16 : 0);
                        }
                        const bool in = (lane & 15) < n;
                        cp_async4z(dst + par_at, in ? par_src + row0 : par_src - (lane & 15),
                                   in ? 4 : 0);
                    }
                }
            }
            ++copied;
            pc.next(p);
            if (pc.t == 0) unit_row = (int64_t)pc.b * p.stride_b + (int64_t)pc.g * p.stride_h;
            if (copied < n_my) look_up();
        }
        cp_async_commit();
    };
#pragma unroll 1
    for (int i = 0; i < kStages - 1; ++i) copy_next();

    uint2 *s_q = reinterpret_cast<uint2 *>(smem + C::kQ);
    int done = 0;
#pragma unroll 1
    while (done < n_my) {
        // ---- a unit's share: tiles [cc.t, cc.t + n_seg) of unit (cc.b, cc.g) ----
        const int n_seg = min(cc.tiles - cc.t, n_my - done);
        const bool starts = cc.t == 0, ends = cc.t + n_seg == cc.tiles;
        const int G = p.group, R = cc.n_q * G, kv_len = cc.kv_len;
        // the last position that query row 0 sees: positions up to it need no mask
        const int first_limit = kv_len - cc.n_q;
        uint32_t qb[kQRegs ? kKs : 1][2];
        float2 qs[NT], qe[NT];  // of columns 2t, 2t + 1: sums of the query, 2^24 / its scale
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = nt * 8 + gq;
            const bool has = r < R;
            const uint4 *src = reinterpret_cast<const uint4 *>(
                static_cast<const unsigned short *>(p.q) +
                ((int64_t)(cc.q0 + (has ? r / G : 0)) * p.h_q + cc.g * G + (has ? r % G : 0)) * D +
                t4 * (D / 4));
            uint4 x[kW];
            float sum = 0.f, top = 0.f;
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                x[w] = has ? ld_dep(src + w) : make_uint4(0u, 0u, 0u, 0u);
                float f[8];
                Chunk<true>::to_float(x[w], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    sum += f[e];
                    top = fmaxf(top, fabsf(f[e]));
                }
            }
            sum += __shfl_xor_sync(FULL, sum, 1);
            sum += __shfl_xor_sync(FULL, sum, 2);
            top = fmaxf(top, __shfl_xor_sync(FULL, top, 1));
            top = fmaxf(top, __shfl_xor_sync(FULL, top, 2));
            float unscale;
            const float scale = query_scale(top, unscale);
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                float f[8];
                Chunk<true>::to_float(x[w], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] *= e & 1 ? scale * 0.0625f : scale;
                const uint32_t f0 = pack_f16(f[0], f[4]), f1 = pack_f16(f[1], f[5]);
                const uint32_t f2 = pack_f16(f[2], f[6]), f3 = pack_f16(f[3], f[7]);
                if constexpr (kQRegs) {
                    qb[2 * w][0] = f0;
                    qb[2 * w][1] = f1;
                    qb[2 * w + 1][0] = f2;
                    qb[2 * w + 1][1] = f3;
                } else if (warp == 0) {
                    s_q[((2 * w) * NT + nt) * 32 + lane] = make_uint2(f0, f1);
                    s_q[((2 * w + 1) * NT + nt) * 32 + lane] = make_uint2(f2, f3);
                }
            }
            qs[nt] = make_float2(__shfl_sync(FULL, sum, 8 * t4), __shfl_sync(FULL, sum, 8 * t4 + 4));
            qe[nt] = make_float2(__shfl_sync(FULL, unscale, 8 * t4),
                                 __shfl_sync(FULL, unscale, 8 * t4 + 4));
        }
        // (the merge's barriers at the end of a share keep the fragments until all have read them)
        if (!kQRegs) __syncthreads();
        float o[kKs][NT][4], m[NT][2];
        float2 l2[NT], cr2[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int mt = 0; mt < kKs; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
            m[nt][0] = m[nt][1] = -INFINITY;
            l2[nt] = cr2[nt] = make_float2(0.f, 0.f);
        }
        // One page pair at j0 (instantiated apart for positions that need no mask).
        auto step = [&](const uint8_t *st, int j0, auto masked) {
            constexpr bool kMasked = decltype(masked)::value;
            // ---- S^T = K Q^T: s[page][nt] holds positions pos_of(g), pos_of(g) + 8 ----
            float s[2][NT][4];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[i][nt][e] = 0.f;
            uint32_t kw[2][2][kW];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint8_t *src =
                        st + i * C::kPageBytes + (gq + 8 * h) * C::kRow + t4 * (C::kRow / 4);
                    if constexpr (D == 128) {
                        const uint4 x = *reinterpret_cast<const uint4 *>(src);
                        kw[i][h][0] = x.x;
                        kw[i][h][1] = x.y;
                        kw[i][h][kW - 2] = x.z;
                        kw[i][h][kW - 1] = x.w;
                    } else {
                        const uint2 x = *reinterpret_cast<const uint2 *>(src);
                        kw[i][h][0] = x.x;
                        kw[i][h][1] = x.y;
                    }
                }
#pragma unroll
            for (int w = 0; w < kW; ++w) {
                uint2 f[2][NT];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if constexpr (kQRegs)
                            f[h][nt] = make_uint2(qb[2 * w + h][0], qb[2 * w + h][1]);
                        else
                            f[h][nt] = s_q[((2 * w + h) * NT + nt) * 32 + lane];
                    }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t x = kw[i][0][w], y = kw[i][1][w], x8 = x >> 8, y8 = y >> 8;
                    const uint32_t a0 = codes_at<0>(x, x8), a1 = codes_at<0>(y, y8);
                    const uint32_t a2 = codes_at<1>(x, x8), a3 = codes_at<1>(y, y8);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma16816(s[i][nt], a0, a1, a2, a3, f[0][nt].x, f[0][nt].y);
                    const uint32_t b0 = codes_at<2>(x, x8), b1 = codes_at<2>(y, y8);
                    const uint32_t b2 = codes_at<3>(x, x8), b3 = codes_at<3>(y, y8);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma16816(s[i][nt], b0, b1, b2, b3, f[1][nt].x, f[1][nt].y);
                }
            }
            // ---- exponents of the weights: x + log2 s - m ----
            float2 nm[NT];  // (before a column's first visible position its maximum counts as 0)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                nm[nt] = make_float2(m[nt][0] == -INFINITY ? 0.f : -m[nt][0],
                                     m[nt][1] == -INFINITY ? 0.f : -m[nt][1]);
            bool grow = false;
            float is[2][2], vl[2][2];  // 1 / s and lo / s + 8 of the values
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t *par =
                    reinterpret_cast<const uint32_t *>(st + i * C::kPageBytes + 2 * C::kPage);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t kp = par[gq + 8 * h], vp = par[16 + gq + 8 * h];
                    const float ks = param_scale(kp) * p.scale_log2;
                    const float kl = param_low(kp) * p.scale_log2;
                    const float sc = value_scale(vp);
                    is[i][h] = rcp(sc);
                    vl[i][h] = fmaf(param_low(vp), is[i][h], 8.f);
                    const float ls = lg2(sc);
                    const float2 ks2 = make_float2(ks, ks), kl2 = make_float2(kl, kl);
                    const float2 ls2 = make_float2(ls, ls);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float2 x = __ffma2_rn(
                            __fmul2_rn(make_float2(s[i][nt][2 * h], s[i][nt][2 * h + 1]), qe[nt]), ks2,
                            __ffma2_rn(kl2, qs[nt], __fadd2_rn(ls2, nm[nt])));
                        s[i][nt][2 * h] = x.x;
                        s[i][nt][2 * h + 1] = x.y;
                    }
                }
            }
            if constexpr (kMasked) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        // last visible position of the column (those past R see nothing)
                        const int n = nt * 8 + 2 * t4 + c;
                        const int limit = n < R ? first_limit + n / G : -1;
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (j0 + i * kPageSize + pos_of(gq) + 8 * h > limit)
                                    s[i][nt][2 * h + c] = -INFINITY;
                    }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    grow |= fmaxf(fmaxf(s[0][nt][c], s[0][nt][2 + c]),
                                  fmaxf(s[1][nt][c], s[1][nt][2 + c])) >
                            (m[nt][c] == -INFINITY ? -INFINITY : kGrowLog2);
            if (__any_sync(FULL, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float f[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        float x = fmaxf(fmaxf(s[0][nt][c], s[0][nt][2 + c]),
                                        fmaxf(s[1][nt][c], s[1][nt][2 + c]));
                        x = fmaxf(x, __shfl_xor_sync(FULL, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(FULL, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(FULL, x, 16));
                        const bool up = x > (m[nt][c] == -INFINITY ? -INFINITY : kGrowLog2);
                        x -= kTopLog2;
                        f[c] = up && m[nt][c] != -INFINITY ? ex2(-x) : 1.f;
                        if (up) {
                            m[nt][c] = (m[nt][c] == -INFINITY ? 0.f : m[nt][c]) + x;
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                s[i][nt][c] -= x;
                                s[i][nt][2 + c] -= x;
                            }
                        }
                    }
                    l2[nt] = __fmul2_rn(l2[nt], make_float2(f[0], f[1]));
                    cr2[nt] = __fmul2_rn(cr2[nt], make_float2(f[0], f[1]));
#pragma unroll
                    for (int mt = 0; mt < kKs; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[mt][nt][e] *= f[e & 1];
                }
            }
            uint32_t pts[2][NT][2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint8_t *pg = st + i * C::kPageBytes;
                // ---- weights, and their transpose in operand layout ----
                uint32_t (&pt)[NT][2] = pts[i];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const float a = s[i][nt][2 * h], b = s[i][nt][2 * h + 1];
                        float2 is2 = make_float2(is[i][h], is[i][h]);
                        float2 vl2 = make_float2(vl[i][h], vl[i][h]);
                        if constexpr (kMasked) {  // a hidden position's NaN must not get through
                            if (a == -INFINITY) is2.x = vl2.x = 0.f;
                            if (b == -INFINITY) is2.y = vl2.y = 0.f;
                        }
                        const float2 w = make_float2(ex2(a), ex2(b));
                        l2[nt] = __ffma2_rn(w, is2, l2[nt]);
                        cr2[nt] = __ffma2_rn(w, vl2, cr2[nt]);
                        pt[nt][h] = transpose8(pack_f16(w.x, w.y));
                    }
                }
                // ---- O^T += V^T P^T ----
                constexpr int kVw = D / 64;  // words of a lane's 8-channel groups per position
                uint32_t vw[4][kVw];
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    const int r = t4 + 4 * h;
                    if constexpr (D == 128) {
                        const uint2 x = *reinterpret_cast<const uint2 *>(
                            pg + C::kPage + r * C::kRow + ((gq >> 1) ^ (r & 2)) * 16 + (gq & 1) * 8);
                        vw[h][0] = x.x;
                        vw[h][kVw - 1] = x.y;
                    } else {
                        vw[h][0] = *reinterpret_cast<const uint32_t *>(pg + C::kPage + r * C::kRow +
                                                                       gq * 4);
                    }
                }
                // channel D/8 g + 8 w + 4 h + c: tile 4 w + 2 h + c / 2, row g + 8 (c & 1)
#pragma unroll
                for (int w = 0; w < kVw; ++w)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t x = __byte_perm(vw[0][w], vw[1][w], h ? 0x7632 : 0x5410);
                        const uint32_t y = __byte_perm(vw[2][w], vw[3][w], h ? 0x7632 : 0x5410);
                        const uint32_t a0 = high_codes_at<0>(x), a1 = high_codes_at<1>(x);
                        const uint32_t a2 = high_codes_at<0>(y), a3 = high_codes_at<1>(y);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816(o[4 * w + 2 * h][nt], a0, a1, a2, a3, pt[nt][0], pt[nt][1]);
                        const uint32_t b0 = high_codes_at<2>(x), b1 = high_codes_at<3>(x);
                        const uint32_t b2 = high_codes_at<2>(y), b3 = high_codes_at<3>(y);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816(o[4 * w + 2 * h + 1][nt], b0, b1, b2, b3, pt[nt][0], pt[nt][1]);
                    }
            }
            // ---- 8 times the weights' sums, as rounded, off every channel ----
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float sw[4] = {0.f, 0.f, 0.f, 0.f};  // of columns 2t, 2t + 1, twice
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    mma16816(sw, kOnes, kOnes, kOnes, kOnes, pts[i][nt][0], pts[i][nt][1]);
                const float2 s2 = make_float2(sw[0], sw[1]);
                const float2 by = make_float2(-8.f / kVOne, -8.f / kVOne);
#pragma unroll
                for (int mt = 0; mt < kKs; ++mt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float2 x = __ffma2_rn(
                            s2, by, make_float2(o[mt][nt][2 * h], o[mt][nt][2 * h + 1]));
                        o[mt][nt][2 * h] = x.x;
                        o[mt][nt][2 * h + 1] = x.y;
                    }
            }
        };
#pragma unroll 1
        for (int it = 0; it < n_seg; ++it, ++done) {
            copy_next();
            cp_async_wait<kStages - 1>();
            __syncwarp();
            const int j0 = (cc.t + it) * kTile + warp * kPos;
            const uint8_t *st = ring_p + (done % kStages) * C::kStageBytes;
            if (j0 + kPos - 1 <= first_limit)
                step(st, j0, std::false_type{});
            else if (j0 < kv_len)  // (a second page past the end is masked as a whole)
                step(st, j0, std::true_type{});
            __syncwarp();  // (the stage's next copies)
        }
        // ---- end of the share: merge the warps ----
        float l[NT][2], cr[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            l[nt][0] = l2[nt].x;
            l[nt][1] = l2[nt].y;
            cr[nt][0] = cr2[nt].x;
            cr[nt][1] = cr2[nt].y;
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
        }
        float *part = reinterpret_cast<float *>(smem + C::kRing);
#pragma unroll 1
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
        if (tid == 0 && !p.whole) {
            int *uc = reinterpret_cast<int *>(kv4_unit_ctas(p) + (int64_t)cc.b * p.h_kv + cc.g);
            if (starts) uc[0] = blockIdx.x;
            if (ends) uc[1] = blockIdx.x;
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
                        x[2 * mt] = fmaf(o[mt][nt][c], kVOne, cr[nt][c]);
                        x[2 * mt + 1] = fmaf(o[mt][nt][2 + c], kVOne, cr[nt][c]);
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
                        const int64_t part_slot = 2 * (int64_t)blockIdx.x + (starts ? 1 : 0);
                        float4 *dst =
                            reinterpret_cast<float4 *>(kv4_slot_o(p, part_slot, n) + gq * (D / 8));
#pragma unroll
                        for (int i = 0; i < D / 32; ++i)
                            dst[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
                        if (gq == 0) {
                            float *ml = kv4_slot_ml(p, part_slot, n);
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
    return e != cudaSuccess || p.whole ? e : launch_kv4_merge(p, s);
}

template <int D>
cudaError_t launch_d(const Kv4Params &p, cudaStream_t s) {
    return p.group * p.max_q_rows <= 8 ? launch_t<D, 1>(p, s) : launch_t<D, 2>(p, s);
}

}  // namespace

// From 17 rows on the tcgen05 kernel is faster (28 sequences of 26,027 positions, 4 KV heads: this
// kernel with 32 rows per warp took 228 us for 21 rows and 230 for 28, the tcgen05 one takes 227 and
// 224; one sequence of 8,710 and 28 rows 24.1 against 18.0).  Up to 16 this one is: 197 against 220 us
// for 14 rows, 15.6 against 17.8 for the one sequence.
int kv4_mma_max_rows() { return 16; }

void kv4_mma_plan(int *tile, int *per_sm) {
    *tile = kTile;
    *per_sm = kCtasPerSm;
}

cudaError_t launch_kv4_mma(const Kv4Params &p, cudaStream_t s) {
    return p.head_dim == 128 ? launch_d<128>(p, s) : launch_d<64>(p, s);
}

}  // namespace sd
