// tcgen05 attention over a 4-bit cache for many rows per KV head (verification): 17 to 128 rows,
// bf16.
//
// The mathematics is kv4_mma.cu's: the codes themselves are multiplied, the queries are scaled per
// row, and V's scale is in the weights' exponent.  V's codes are c - 8 here, one more instruction
// per pair than c 2^-24: one accumulator gathers hundreds of tiles, its sum of w c would be far larger
// than the output that is left after lo's part is added, and the tensor core rounds towards zero
// as it accumulates (26,033 random positions: output off by 5e-3 of itself with c, 2e-3, most of
// it the output's own rounding, with c - 8).  With this many rows the products outgrow
// mma.sync (1,024 products per cycle per SM; a tile of 64 rows would need 2,048 cycles, three times
// what it takes from HBM), so the codes are spread to fp16 tiles in shared memory once and used by
// tcgen05.mma (4,096 products per cycle).
//
// One persistent CTA per SM, 11 warps (168 registers a thread); the CTAs share all units'
// tiles evenly (kv4_common.cuh).
//   warps 0-3  softmax: TMEM lane r holds MMA row r.  The unit's R rows are placed NCP times
//              (4 copies up to 32 rows, 2 up to 64, else 1) and each warp handles 128 / NCP
//              columns of its copy, so a tile's exponentials are spread over all four warps
//   warps 4-7  expand: each takes 32 positions of every tile from the ring and writes them as fp16
//              into the K and V tiles (128-byte rows of 64 channels, 128-byte swizzle), with the
//              positions' five factors beside them
//   warp 8     S = Q K^T issuer (Q from TMEM), TMEM owner
//   warp 9     O += P V issuer (P from TMEM)
//   warp 10    copies tiles up to kStages ahead: one bulk copy per page for the codes of K and of V
// A word of 8 codes becomes one 16-byte chunk by 4 logic operations and a shift (V: and 4 additions), its channels in the order
// 0 4 1 5 2 6 3 7; Q is written to TMEM in the same order and O's columns are read back in it, so
// no code is ever moved to its own place.
// The softmax takes 32 columns at a time in one pass: the exponents are taken from the running
// maximum as it stands, and only when one exceeds kGrowLog2 does the maximum move (then O, the sums
// and the tile's earlier weights are rescaled).  A second pass, or more columns unrolled into one
// block of code, costs more than its instructions: the warps' roles together must stay within
// the instruction cache (with 64 columns and 32 positions unrolled, two of three issue slots were
// lost to instruction fetch and a tile took 7,000 cycles).
// K and V tiles, S and P are double-buffered: S of tile t overwrites the buffer of tile t - 2
// once that tile's P V has completed.
// Bound by the chain of those steps: with two buffers a tile's S, its softmax and its P V follow one
// another, about 3,300 cycles a tile for 63 rows and 128 channels (154 tiles per CTA), of which the
// softmax has 2,200; the tensor core is busy for 29% of the kernel's time, issue slots for 42%, shared
// memory for 38%.  (A third buffer beside O needs Q in shared memory, where attn_tc.cu has it, and
// with it a shorter ring; not built.)  28 sequences of 26,033 positions, 4 KV heads, 63 rows: 259 us,
// 1.5 TB/s: no faster than attn_tc.cu over a bf16 cache, 252-260 us, which reads 3.8 times the bytes.
// 70 rows 355 us and 126 rows 372 (one copy: a warp has all 128 columns).
// Measured on the way, with codes not yet centred (then 250 us): every
// expanding warp with its own cp.async ring instead of a copying warp 269; the positions' factors
// loaded where they are used 274; 64 columns at a time 293.  Centred: one code for K's and V's
// expansion 274, the four steps of an expansion unrolled together 275.
// Every wait on an mbarrier is bounded (see sd_set_wait_timeout_ns); on expiry the CTA records
// SD_DEVERR_TIMEOUT, drains its copies and MMAs, frees TMEM and exits.
#include <type_traits>

#include "kv4_common.cuh"
#include "tc_ptx.cuh"

namespace sd {
namespace {

using namespace tc;

constexpr int kRows = 128;           // MMA M
constexpr int kTile = 128;           // positions per tile (p.tile)
constexpr int kExpandWarp = 4;       // first of four
constexpr int kExpandWarps = 4;
constexpr int kSWarp = 8;
constexpr int kPvWarp = 9;
constexpr int kCopyWarp = 10;
constexpr int kThreads = 11 * 32;
constexpr int kWarpRows = kTile / kExpandWarps;  // positions of a tile, per expanding warp
static_assert(kWarpRows == 32, "a lane makes one position's factors");
constexpr int kPages = kTile / kPageSize;
constexpr int kStages = 4;           // ring of tiles in flight
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;      // S / P buffers at 0 and 128
constexpr uint32_t kColQ = 384;
constexpr uint32_t kHalfBytes = kTile * 128;  // 64 channels of a tile
constexpr int kParSlots = 4;         // tiles whose position factors are kept:
// pairs of positions' (s, lo) of K [0, 256), log2 s of V [256, 384), (1 / s, lo / s) [384, 640)
constexpr int kParFloats = 5 * kTile;

template <int D>
struct TcCfg {
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kRow = D / 2;
    static constexpr int kCodes = kTile * kRow;                 // K's codes of a tile
    static constexpr int kStageBytes = 2 * kCodes + 8 * kTile;  // K, V, parameters of K and V
    static constexpr int kRing = 4 * kTileBytes;           // after K0 K1 V0 V1
    static constexpr int kPar = kRing + kStages * kStageBytes;
    static constexpr int kScratch = kPar + kParSlots * kParFloats * 4;
    // maxima and sums of every MMA row, then 32 columns of the copies' outputs
    static constexpr int kScratchBytes = (2 * kRows + 96 * 32) * 4;
    static constexpr int kBars = kScratch + kScratchBytes;
    static constexpr int kSmem = kBars + 256 + 1024;
};
static_assert(TcCfg<128>::kSmem <= 227 * 1024, "shared memory");

// kind::f16 instruction descriptor: fp32 accumulate, fp16 A and B, M = 128.
__host__ __device__ constexpr uint32_t idesc_f16(int n, bool b_mn_major) {
    return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
           ((uint32_t)(128 >> 4) << 24);
}

// 16 consecutive columns of this thread's TMEM lane.  Stores are not waited for: a wait::st comes
// before the columns are loaded again or handed to the tensor core.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// 8 N columns of 32 lanes in the accumulator layout of an m16n8 fragment (N = 4 or 8): lane (g, t)
// of the warp gets rows g + 8 k (k = 0..3), columns 8 i + 2 t and 8 i + 2 t + 1 (i < N) in
// v[k / 2][4 i + 2 (k % 2)] and the element after it.
template <int N>
__device__ __forceinline__ void tmem_ld_frag(uint32_t taddr, float (&v)[2][4 * N]) {
    uint32_t r[2][4 * N];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < 4 * N; b += 16)
            asm volatile(
                "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
                "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                : "=r"(r[h][b]), "=r"(r[h][b + 1]), "=r"(r[h][b + 2]), "=r"(r[h][b + 3]),
                  "=r"(r[h][b + 4]), "=r"(r[h][b + 5]), "=r"(r[h][b + 6]), "=r"(r[h][b + 7]),
                  "=r"(r[h][b + 8]), "=r"(r[h][b + 9]), "=r"(r[h][b + 10]), "=r"(r[h][b + 11]),
                  "=r"(r[h][b + 12]), "=r"(r[h][b + 13]), "=r"(r[h][b + 14]), "=r"(r[h][b + 15])
                : "r"(taddr + ((uint32_t)h << 20) + 2 * b)
                : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    // (the values pass through statements after the wait, so no use can move before it)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4 * N; ++e) {
            asm volatile("" : "+r"(r[h][e])::"memory");
            v[h][e] = __uint_as_float(r[h][e]);
        }
}

// The same layout's pairs of columns, packed to fp16: 4 N columns of 32 lanes (lane (g, t): rows
// g + 8 k, column 4 i + t in w[k / 2][2 i + k % 2]).
template <int N>
__device__ __forceinline__ void tmem_st_frag(uint32_t taddr, const uint32_t (&w)[2][2 * N]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < 2 * N; b += 8)
            asm volatile(
                "tcgen05.st.sync.aligned.16x128b.x4.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(
                    taddr + ((uint32_t)h << 20) + 2 * b),
                "r"(w[h][b]), "r"(w[h][b + 1]), "r"(w[h][b + 2]), "r"(w[h][b + 3]),
                "r"(w[h][b + 4]), "r"(w[h][b + 5]), "r"(w[h][b + 6]), "r"(w[h][b + 7])
                : "memory");
}

// Bounded wait, out of the hot code: plain polls (the hardware suspends each for a while and wakes
// it when the phase completes; a poll with a time of its own sleeps in steps, and the kernel's
// roles hand over to one another several times per tile), the clock and the abort flag every 64.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int *abort_flag,
                                       int32_t *dev_err, unsigned long long limit_ns) {
    const unsigned long long t0 = now_ns();
    for (;;) {
        for (int i = 0; i < 64; ++i)
            if (mbar_try(bar, parity)) return true;
        if (*abort_flag) return false;
        if (now_ns() - t0 > limit_ns) {
            *abort_flag = 1;
            set_dev_err(dev_err, SD_DEVERR_TIMEOUT);
            return false;
        }
    }
}

// Column of channel e (0..7) within its group of 8, and the channel order of a group's columns.
__device__ __forceinline__ constexpr int col_of(int e) { return e < 4 ? 2 * e : 2 * (e - 4) + 1; }

template <int D, int NCP>
__global__ void __launch_bounds__(kThreads, 1) kv4_tc_kernel(const __grid_constant__ Kv4Params p) {
    pdl_trigger();  // (see launch_pdl)
    pdl_wait();
    using C = TcCfg<D>;
    constexpr unsigned FULL = 0xffffffffu;
    constexpr int RPC = kRows / NCP;          // rows per copy
    constexpr int NC = kTile / NCP;           // columns of a softmax warp
    constexpr int CW = NC < 32 ? NC : 32;     // columns that it holds at a time
    constexpr int N8 = CW / 8;
    extern __shared__ uint8_t smem_raw[];
    // (an offset from the array, so that accesses stay shared-memory instructions)
    uint8_t *smem = smem_raw + ((1024u - (saddr(smem_raw) & 1023u)) & 1023u);
    __shared__ long long s_red[kThreads / 32];
    __shared__ Kv4Start s_start;
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    volatile int *abort_flag = &s_abort;
    uint8_t *sK = smem, *sV = smem + 2 * C::kTileBytes;
    float *s_par = reinterpret_cast<float *>(smem + C::kPar);
    const uint32_t bar0 = saddr(smem + C::kBars);
    auto BAR = [&](int i) { return bar0 + 8u * (uint32_t)i; };
    // K written, K read (S computed), V written, S computed, P written, P V computed (V read and
    // the S / P buffer free), per buffer; then a unit's share done, Q written, two drains
    constexpr int KF = 0, KE = 2, VF = 4, SF = 6, PF = 8, PD = 10, SD = 12, QF = 13, DR = 14, DS = 15;
    // a stage of the ring filled, and read
    constexpr int RF = 16, RE = RF + kStages;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = p.group;
    const int n_active = NCP > 1 ? 4 : min(4, (G * p.max_q_rows + 31) / 32);

    long long lo, hi;
    const Kv4Cursor first = kv4_first<kThreads>(p, s_red, &s_start, lo, hi);
    if (hi <= lo) return;
    const int n_my = (int)(hi - lo);
    if (warp == kSWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         saddr(&s_tmem)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(BAR(KF + s), kExpandWarps);
            mbar_init(BAR(KE + s), 1);
            mbar_init(BAR(VF + s), kExpandWarps);
            mbar_init(BAR(SF + s), 2);  // the commit, and the issuer's own arrival
            mbar_init(BAR(PF + s), 32 * n_active);
            mbar_init(BAR(PD + s), 1);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(BAR(RF + i), 64);  // (two arrivals of each lane of the copying warp)
            mbar_init(BAR(RE + i), kExpandWarps);
        }
        mbar_init(BAR(SD), 1);
        mbar_init(BAR(QF), 32 * n_active);
        mbar_init(BAR(DR), 1);
        mbar_init(BAR(DS), 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = s_tmem;
    auto wait = [&](int bar, int parity) {
        return mbar_try(BAR(bar), parity & 1) ||
               wait_slow(BAR(bar), parity & 1, abort_flag, p.dev_err, p.wait_ns);
    };
    // One lane waits; the outcome is the warp's.
    auto wait1 = [&](int bar, int parity) {
        bool ok = true;
        if (lane == 0) ok = wait(bar, parity);
        __syncwarp();  // (orders what lane 0 has seen before the other lanes' accesses)
        return __shfl_sync(FULL, ok ? 1 : 0, 0) != 0;
    };

    if (warp >= kExpandWarp && warp < kExpandWarp + kExpandWarps) {
        // ---------------------------------------------------------- expand --------------------
        const int ew = warp - kExpandWarp;
        constexpr int Q = C::kRow / 16;       // 16-byte chunks of a row
        constexpr int kLoads = kWarpRows * Q / 32;
        // The warp's rows of K (or V) of a stage into a tile.  Load i of the warp is 32 / Q rows in
        // a piece: lane has chunk lane % Q of row lane / Q.  Word c of chunk q is 16-byte chunk
        // 4 (q & 1) + c of the row in half q / 2; lanes of the second half take their words in
        // the order 2 3 0 1, so that 8 lanes' stores fall into different banks.
        const int er = lane / Q, eq = lane % Q;
        const bool swap = eq >= 2;
        const uint32_t at = (uint32_t)((ew * kWarpRows + er) * 128) + (uint32_t)(eq >> 1) * kHalfBytes +
                            (uint32_t)((((eq & 1) * 4) ^ (swap ? 2 : 0) ^ (er & 7)) << 4);
        auto expand = [&](const uint8_t *src, uint8_t *dst, auto is_v) {
            constexpr bool kV = decltype(is_v)::value;
#pragma unroll 2
            for (int i = 0; i < kLoads; ++i) {
                const uint4 x = *reinterpret_cast<const uint4 *>(
                    src + ew * kWarpRows * C::kRow + i * 512 + lane * 16);
                const uint32_t w[4] = {swap ? x.z : x.x, swap ? x.w : x.y,
                                       swap ? x.x : x.z, swap ? x.y : x.w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint32_t w8 = w[c] >> 8;
                    // (32 / Q rows on; the swizzle of row r is r mod 8, and 32 / Q is 8 or 16)
                    *reinterpret_cast<uint4 *>(dst + i * (32 / Q) * 128 +
                                               (at ^ (uint32_t)(c << 4))) =
                        kV ? make_uint4(centred_at<0>(w[c], w8), centred_at<1>(w[c], w8),
                                        centred_at<2>(w[c], w8), centred_at<3>(w[c], w8))
                           : make_uint4(codes_at<0>(w[c], w8), codes_at<1>(w[c], w8),
                                        codes_at<2>(w[c], w8), codes_at<3>(w[c], w8));
                }
            }
            fence_async_smem();
            __syncwarp();
        };
#pragma unroll 1
        for (int t = 0; t < n_my; ++t) {
            const int s = t & 1;
            const uint8_t *st = smem + C::kRing + (t % kStages) * C::kStageBytes;
            if (!wait1(RF + t % kStages, t / kStages)) break;
            if (t >= 2 && !wait1(KE + s, (t - 2) >> 1)) break;
            {
                // Factors of the positions.  (Slot t % 4: the softmax of tile t - 4 is past it,
                // since S of tile t - 2 has completed and that waited for the P V of tile t - 4.)
                const int j = ew * kWarpRows + lane;
                const uint32_t *w = reinterpret_cast<const uint32_t *>(st + 2 * C::kCodes) + j;
                const uint32_t wk = w[0], wv = w[kTile];
                float *f = s_par + (t % kParSlots) * kParFloats;
                float *d = f + (j >> 1) * 4 + (j & 1);
                d[0] = param_scale(wk) * p.scale_log2;
                d[2] = param_low(wk) * p.scale_log2;
                // (a V code stands for c - 8: lo moves by 8 s)
                const float sc = value_scale(wv);
                const float inv = rcp(sc);
                f[2 * kTile + j] = lg2(sc);
                d[3 * kTile] = inv;
                d[3 * kTile + 2] = fmaf(param_low(wv), inv, 8.f);
            }
            expand(st, sK + s * C::kTileBytes, std::false_type{});
            if (lane == 0) mbar_arrive(BAR(KF + s));
            if (t >= 2 && !wait1(PD + s, (t - 2) >> 1)) break;
            expand(st + C::kCodes, sV + s * C::kTileBytes, std::true_type{});
            if (lane == 0) {
                mbar_arrive(BAR(VF + s));
                mbar_arrive(BAR(RE + t % kStages));
            }
        }
    } else if (warp == kCopyWarp) {
        // ---------------------------------------------------------- copy ----------------------
        // Lane: page (lane & 7) of the tile, of K (lanes 0-7) or V (lanes 8-15); then positions
        // lane + 32 k of both for the parameters.  Codes of rows past the end stay as they were
        // (any nibble is a finite number, and the softmax gives it the weight zero); parameters
        // are zeros there.
        Kv4Cursor pc = first;
        int64_t unit_row = (int64_t)pc.b * p.stride_b + (int64_t)pc.g * p.stride_h;  // (contiguous)
        auto look_up = [&]() {  // this lane's page of the next tile
            const int j = pc.t * kTile + (lane & 7) * kPageSize;
            return p.page_size && j < pc.kv_len
                       ? ld_dep(p.block_table + (int64_t)pc.b * p.max_pages + (j >> 4))
                       : 0;
        };
        int page = look_up();
        int issued = 0;
#pragma unroll 1
        for (; issued < n_my; ++issued) {
            const int st = issued % kStages;
            if (issued >= kStages && !wait1(RE + st, issued / kStages - 1)) break;
            uint8_t *stage = smem + C::kRing + st * C::kStageBytes;
            const uint32_t dst = saddr(stage);
            const int j = (lane & 7) * kPageSize;
            const int left = pc.kv_len - pc.t * kTile;  // positions of the tile, 128 or more: all
            int n = min(max(left - j, 0), kPageSize);
            int64_t row0 = unit_row + pc.t * kTile + j;
            bool bad = false;
            if (p.page_size) {
                bad = n > 0 && (page < 0 || page >= p.num_pages);
                row0 = ((int64_t)page * p.h_kv + pc.g) * kPageSize;
            }
            const uint32_t my = dst + (lane >> 3) * C::kCodes + j * C::kRow;
            if (lane < 16 && bad) {  // a page outside the pool reads as zeros
                set_dev_err(p.dev_err, SD_DEVERR_PAGE);
                uint8_t *z = stage + (lane >> 3) * C::kCodes + j * C::kRow;
                for (int i = 0; i < kPageSize * C::kRow; i += 16)
                    *reinterpret_cast<uint4 *>(z + i) = make_uint4(0u, 0u, 0u, 0u);
                fence_async_smem();
            }
            if (bad) n = 0;
            const uint32_t bytes = lane < 16 ? (uint32_t)(n * C::kRow) : 0u;
            mbar_arrive_tx(BAR(RF + st), bytes);
            if (bytes)
                bulk_load(my, (lane < 8 ? p.k : p.v) + row0 * C::kRow, bytes, BAR(RF + st));
#pragma unroll
            for (int k = 0; k < kTile / 32; ++k) {
                const int from = 2 * k + (lane >> 4);  // the page's lane
                const int64_t row = __shfl_sync(FULL, row0, from) + (lane & 15);
                const bool in = (lane & 15) < __shfl_sync(FULL, n, from);
                const uint32_t d = dst + 2 * C::kCodes + (lane + 32 * k) * 4;
                cp_async4z(d, p.kp + (in ? row : 0), in ? 4 : 0);
                cp_async4z(d + 4 * kTile, p.vp + (in ? row : 0), in ? 4 : 0);
            }
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(BAR(RF + st))
                         : "memory");
            pc.next(p);
            if (pc.t == 0) unit_row = (int64_t)pc.b * p.stride_b + (int64_t)pc.g * p.stride_h;
            if (issued + 1 < n_my) page = look_up();
        }
        // the copies in flight
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            const unsigned long long t0 = now_ns();
            for (int i = max(issued - kStages, 0); i < issued; ++i)
                while (!mbar_try(BAR(RF + i % kStages), (i / kStages) & 1) &&
                       now_ns() - t0 < kDrainNs) {
                }
        }
        __syncwarp();
    } else if (warp == kSWarp) {
        // ---------------------------------------------------------- S = Q K^T issuer ---------
        const uint32_t idesc = idesc_f16(kTile, false);
        bool issued = false;
        Kv4Cursor c = first;
        int seg = 0;
        for (int t = 0; t < n_my; ++t) {
            const int s = t & 1;
            // (what comes last is waited for last)
            bool ok = true;
            if (t == 0 || c.t == 0) ok = wait1(QF, seg++);  // a unit's share begins
            ok = ok && wait1(KF + s, t >> 1) && (t < 2 || wait1(PD + s, (t - 2) >> 1));
            if (!ok) break;
            tc_after();
            if (lane == 0) {
                const uint32_t kb = saddr(sK + s * C::kTileBytes);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk)
                    mma_ts(tmem + s * kTile, tmem + kColQ + kk * 8,
                           desc_k_sw128(kb + (kk >> 2) * kHalfBytes + (kk & 3) * 32), idesc,
                           kk > 0 ? 1u : 0u);
                mma_commit(BAR(SF + s));
                mma_commit(BAR(KE + s));
                mbar_arrive(BAR(SF + s));  // (orders the factors before the softmax's reads)
                issued = true;
            }
            __syncwarp();
            c.next(p);
        }
        const bool any = __any_sync(FULL, issued);
        if (lane == 0 && any) {
            mma_commit(BAR(DS));
            const unsigned long long t0 = now_ns();
            while (!mbar_try(BAR(DS), 0) && now_ns() - t0 < kDrainNs) {
            }
        }
        __syncwarp();
    } else if (warp == kPvWarp) {
        // ---------------------------------------------------------- O += P V issuer ----------
        const uint32_t idesc = idesc_f16(D, true);
        bool issued = false;
        Kv4Cursor c = first;
        for (int t = 0; t < n_my; ++t) {
            const int s = t & 1;
            if (!(wait1(VF + s, t >> 1) && wait1(PF + s, t >> 1))) break;
            tc_after();
            const bool fresh = t == 0 || c.t == 0;
            const bool last = t + 1 == n_my || c.t + 1 == c.tiles;
            if (lane == 0) {
                const uint32_t vb = saddr(sV + s * C::kTileBytes);
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk)
                    mma_ts(tmem + kColO, tmem + s * kTile + kk * 8,
                           desc_mn_sw128(vb + kk * 2048, kHalfBytes), idesc,
                           (!fresh || kk > 0) ? 1u : 0u);
                mma_commit(BAR(PD + s));
                if (last) mma_commit(BAR(SD));
                issued = true;
            }
            __syncwarp();
            c.next(p);
        }
        const bool any = __any_sync(FULL, issued);
        if (lane == 0 && any) {
            mma_commit(BAR(DR));
            const unsigned long long t0 = now_ns();
            while (!mbar_try(BAR(DR), 0) && now_ns() - t0 < kDrainNs) {
            }
        }
        __syncwarp();
    } else if (warp < n_active) {
        // ---------------------------------------------------------- softmax -------------------
        // tcgen05.ld / st are warp-collective: every lane executes them and decisions that gate
        // them are made uniform by votes.
        const int cp = NCP > 1 ? warp / (4 / NCP) : 0;  // this warp's row copy
        const int c0 = cp * NC;                         // its first column
        const int r = warp * 32 + lane - cp * RPC;      // its row
        const uint32_t lane_base = tmem + ((uint32_t)(warp * 32) << 16);
        float *s_m = reinterpret_cast<float *>(smem + C::kScratch), *s_l = s_m + kRows;
        float4 *s_o = reinterpret_cast<float4 *>(s_l + kRows);  // [copy - 1][RPC][8]
        // Q of unit u into TMEM (zeros past its rows), channels of each group of 8 in the order of
        // the spread codes.
        float qsum, unscale;  // of this lane's row: sum of the query, 2^24 / its scale
        auto write_q = [&](const Kv4Cursor &u) {
            const bool has = r < u.n_q * G;
            const uint4 *src = reinterpret_cast<const uint4 *>(
                static_cast<const unsigned short *>(p.q) +
                ((int64_t)(u.q0 + (has ? r / G : 0)) * p.h_q + u.g * G + (has ? r % G : 0)) * D);
            auto load = [&](int c) { return has ? ld_dep(src + c) : make_uint4(0u, 0u, 0u, 0u); };
            uint32_t top = 0;  // largest magnitudes of both halves, as bits
            float2 sum = make_float2(0.f, 0.f);
            uint4 x[D / 8];
#pragma unroll
            for (int c = 0; c < D / 8; ++c) x[c] = load(c);
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    top = __vmaxu2(top, w[e] & 0x7fff7fffu);
                    sum = __fadd2_rn(sum, make_float2(__uint_as_float(w[e] << 16),
                                                      __uint_as_float(w[e] & 0xffff0000u)));
                }
            }
            qsum = sum.x + sum.y;
            const float scale =
                query_scale(__uint_as_float(max(top << 16, top & 0xffff0000u)), unscale);
            // (channel 2 i is a word's low half; odd channels' codes are 16 times as large)
            const float2 by = make_float2(scale, scale * 0.0625f);
#pragma unroll 
            for (int c = 0; c < D / 8; c += 4) {
                uint32_t q[16];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 y = x[c + i];
                    const uint32_t w[4] = {y.x, y.y, y.z, y.w};
                    float2 f[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        f[e] = __fmul2_rn(make_float2(__uint_as_float(w[e] << 16),
                                                      __uint_as_float(w[e] & 0xffff0000u)),
                                          by);
                    q[4 * i] = pack_f16(f[0].x, f[2].x);
                    q[4 * i + 1] = pack_f16(f[0].y, f[2].y);
                    q[4 * i + 2] = pack_f16(f[1].x, f[3].x);
                    q[4 * i + 3] = pack_f16(f[1].y, f[3].y);
                }
                tmem_st16(lane_base + kColQ + c * 4, q);
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_before();
            mbar_arrive(BAR(QF));
        };
        Kv4Cursor u = first;
        write_q(u);
        bool ok_run = true;
        int t = 0, seg = 0;
        // The softmax itself works on fragments: lane (g, t4) has rows g + 8 k (k = 0..3) of the
        // warp's 32 and two of every eight columns, so a position's factors are loaded by a
        // quarter of the lanes and used for four rows each.
        const int gq = lane >> 2, t4 = lane & 3;
        while (t < n_my) {
            const int n_seg = min(u.tiles - u.t, n_my - t);
            const bool starts = u.t == 0, ends = u.t + n_seg == u.tiles;
            const int R = u.n_q * G;
            const bool row_ok = r < R;
            const int first_limit = u.kv_len - u.n_q;
            const int seg_lo = u.t;
            float mk[4], nm[4], qs[4], qe[4];
            int limit[4];  // last visible position (rows past R see nothing)
            float2 l2[4], cr2[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int rk = warp * 32 + gq + 8 * k - cp * RPC;
                mk[k] = -INFINITY;
                nm[k] = 0.f;
                qs[k] = __shfl_sync(FULL, qsum, gq + 8 * k);
                qe[k] = __shfl_sync(FULL, unscale, gq + 8 * k);
                limit[k] = rk < R ? first_limit + rk / G : -1;
                l2[k] = cr2[k] = make_float2(0.f, 0.f);
            }
            // value of row `lane` from the lanes that hold it
            auto by_row = [&](const float (&x)[4]) {
                float y = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float z = __shfl_sync(FULL, x[k], (lane & 7) * 4);
                    if ((lane >> 3) == k) y = z;
                }
                return y;
            };
            const int t_end = t + n_seg;
            for (int lt = u.t; ok_run && t < t_end; ++t, ++lt) {
                const int s = t & 1;
                if (!__all_sync(FULL, wait(SF + s, t >> 1))) {
                    ok_run = false;
                    break;
                }
                tc_after();
                const uint32_t s_addr = lane_base + s * kTile;
                const float *par = s_par + (t % kParSlots) * kParFloats;
                const int p0 = lt * kTile;
                // every row sees every position of the tile (rows past R may compute anything)
                const bool interior = p0 + kTile - 1 <= first_limit;
                // CW columns (instantiated apart for tiles that need no mask); false: a wait failed
                auto chunk = [&](int ch, auto masked) {
                    constexpr bool kMasked = decltype(masked)::value;
                    const int cb = c0 + ch * CW;
                    // (all of the positions' factors at once, ahead of their use: one warp per
                    // issue slot has nothing else to cover their latency)
                    float4 kf[N8];
                    float2 ls[N8];
#pragma unroll
                    for (int i = 0; i < N8; ++i) {
                        const int at = cb / 2 + 4 * i + t4;  // the pair of positions
                        kf[i] = reinterpret_cast<const float4 *>(par)[at];
                        ls[i] = reinterpret_cast<const float2 *>(par + 2 * kTile)[at];
                    }
                    float4 vf[N8];
#pragma unroll
                    for (int i = 0; i < N8; ++i)
                        vf[i] = reinterpret_cast<const float4 *>(par + 3 * kTile)[cb / 2 + 4 * i + t4];
                    float v[2][4 * N8];
                    tmem_ld_frag<N8>(s_addr + cb, v);
                    // exponents of the weights: x + log2 s - m
#pragma unroll
                    for (int i = 0; i < N8; ++i) {
                        const float4 f = kf[i];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float &a = v[k >> 1][4 * i + 2 * (k & 1)];
                            float &b = v[k >> 1][4 * i + 2 * (k & 1) + 1];
                            const float2 x = __ffma2_rn(
                                __fmul2_rn(make_float2(a, b), make_float2(qe[k], qe[k])),
                                make_float2(f.x, f.y),
                                __ffma2_rn(make_float2(f.z, f.w), make_float2(qs[k], qs[k]),
                                           __fadd2_rn(ls[i], make_float2(nm[k], nm[k]))));
                            a = x.x;
                            b = x.y;
                        }
                    }
                    if constexpr (kMasked) {
#pragma unroll
                        for (int i = 0; i < N8; ++i)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
#pragma unroll
                                for (int c = 0; c < 2; ++c)
                                    if (p0 + cb + 8 * i + 2 * t4 + c > limit[k])
                                        v[k >> 1][4 * i + 2 * (k & 1) + c] = -INFINITY;
                    }
                    float mx[4];
                    bool grow = false;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        mx[k] = -INFINITY;
#pragma unroll
                        for (int i = 0; i < N8; ++i)
                            mx[k] = max3(mx[k], v[k >> 1][4 * i + 2 * (k & 1)],
                                         v[k >> 1][4 * i + 2 * (k & 1) + 1]);
                        // (before a row's first visible position its maximum is -inf and nm is 0)
                        grow |= mx[k] > (mk[k] == -INFINITY ? -INFINITY : kGrowLog2);
                    }
                    if (__any_sync(FULL, grow)) {
                        float f[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float x = fmaxf(mx[k], __shfl_xor_sync(FULL, mx[k], 1));
                            x = fmaxf(x, __shfl_xor_sync(FULL, x, 2));
                            const bool up = x > (mk[k] == -INFINITY ? -INFINITY : kGrowLog2);
                            // (whole steps: the tile's earlier weights, rounded already, take a
                            // power of two exactly)
                            x = floorf(x - kTopLog2);
                            f[k] = up && mk[k] != -INFINITY ? ex2(-x) : 1.f;
                            if (up) {
                                mk[k] = x - nm[k];
                                nm[k] = -mk[k];
#pragma unroll
                                for (int i = 0; i < N8; ++i)
#pragma unroll
                                    for (int c = 0; c < 2; ++c) v[k >> 1][4 * i + 2 * (k & 1) + c] -= x;
                            }
                            l2[k].x *= f[k];
                            l2[k].y *= f[k];
                            cr2[k].x *= f[k];
                            cr2[k].y *= f[k];
                        }
                        const float fr = by_row(f);
                        if (lt > seg_lo) {
                            // O holds the share's earlier tiles: wait for the P V of tile t - 1.
                            // (Its barrier is in phase t - 3 or t - 1: S of tile t - 1 waited for
                            // the former, and tile t + 1's P V needs this warp's arrival.)
                            if (!__all_sync(FULL, wait(PD + ((t - 1) & 1), (t - 1) >> 1))) {
                                return false;
                            }
                            tc_after();
#pragma unroll 1
                            for (int c = 0; c < D / 16; ++c) {
                                uint32_t o[16];
                                tmem_ld16(lane_base + kColO + c * 16, o);
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    o[e] = __float_as_uint(__uint_as_float(o[e]) * fr);
                                tmem_st16(lane_base + kColO + c * 16, o);
                            }
                        }
                        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
#pragma unroll 1
                        for (int c = 0; c < ch * (CW / 32); ++c) {  // this tile's weights so far
                            uint32_t w[16];
                            tmem_ld16(s_addr + c0 / 2 + c * 16, w);
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                            {
                                const float2 x =
                                    __half22float2(*reinterpret_cast<const __half2 *>(&w[e]));
                                w[e] = pack_f16(x.x * fr, x.y * fr);
                            }
                            tmem_st16(s_addr + c0 / 2 + c * 16, w);
                        }
                    }
                    uint32_t pk[2][2 * N8];
#pragma unroll
                    for (int i = 0; i < N8; ++i) {
                        const float4 f = vf[i];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float a = v[k >> 1][4 * i + 2 * (k & 1)];
                            const float b = v[k >> 1][4 * i + 2 * (k & 1) + 1];
                            float2 is = make_float2(f.x, f.y), vl = make_float2(f.z, f.w);
                            if constexpr (kMasked) {  // a hidden position's NaN must not get through
                                if (a == -INFINITY) is.x = vl.x = 0.f;
                                if (b == -INFINITY) is.y = vl.y = 0.f;
                            }
                            const float2 w = make_float2(ex2(a), ex2(b));
                            l2[k] = __ffma2_rn(w, is, l2[k]);
                            cr2[k] = __ffma2_rn(w, vl, cr2[k]);
                            pk[k >> 1][2 * i + (k & 1)] = pack_f16(w.x, w.y);
                        }
                    }
                    // P over the columns of S that this warp has read
                    tmem_st_frag<N8>(s_addr + cb / 2, pk);
                    return true;
                };
                if (interior) {
#pragma unroll 1
                    for (int ch = 0; ok_run && ch < NC / CW; ++ch)
                        ok_run = chunk(ch, std::false_type{});
                } else {
#pragma unroll 1
                    for (int ch = 0; ok_run && ch < NC / CW; ++ch)
                        ok_run = chunk(ch, std::true_type{});
                }
                if (!ok_run) break;
                if constexpr (NCP > 1) {  // zeros in the other copies' columns
                    uint32_t z[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) z[e] = 0u;
#pragma unroll 1
                    for (int c = 0; c < kTile / 2; c += 16)
                        if (c / (NC / 2) != cp) tmem_st16(s_addr + c, z);
                }
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_before();
                mbar_arrive(BAR(PF + s));
            }
            t = t_end;  // (after a failed wait every warp still passes the barriers below)
            // ---- end of the share: the next one's Q, then this one's output ----
            Kv4Cursor nx = u;
            nx.skip(p, n_seg);
            if (ok_run && t < n_my) write_q(nx);
            bool done = ok_run;
            if (ok_run) done = wait(SD, seg);
            ++seg;
            const bool read_o = __all_sync(FULL, done);
            if (!read_o) ok_run = false;
            tc_after();
            // from here on a lane is one row again
            float lk[4], ck[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                lk[k] = l2[k].x + l2[k].y;
                ck[k] = cr2[k].x + cr2[k].y;
#pragma unroll
                for (int x = 1; x < 4; x <<= 1) {
                    lk[k] += __shfl_xor_sync(FULL, lk[k], x);
                    ck[k] += __shfl_xor_sync(FULL, ck[k], x);
                }
            }
            float m = by_row(mk), l = by_row(lk);
            const float cr = by_row(ck);
            if (l != l && m == -INFINITY) m = 0.f;  // (a NaN sum survives the merges)
            float fq[NCP];
            if constexpr (NCP > 1) {
                asm volatile("bar.sync 1, 128;" ::: "memory");  // the last share's merge is done
                s_m[cp * RPC + r] = m;
                s_l[cp * RPC + r] = l;
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (cp == 0) {
                    float M = -INFINITY;
#pragma unroll
                    for (int q = 0; q < NCP; ++q) M = fmaxf(M, s_m[q * RPC + r]);
                    l = 0.f;
#pragma unroll
                    for (int q = 0; q < NCP; ++q) {
                        const float mq = s_m[q * RPC + r];
                        fq[q] = mq == -INFINITY ? 0.f : ex2(mq - M);
                        l += fq[q] * s_l[q * RPC + r];
                    }
                    m = M;
                }
            }
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const int row = u.q0 + (row_ok ? r / G : 0), h = u.g * G + (row_ok ? r % G : 0);
            const int64_t slot = 2 * (int64_t)blockIdx.x + (starts ? 1 : 0);
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                float o[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0.f;
                if (read_o) tmem_ld32(lane_base + kColO + c * 32, o);
#pragma unroll
                for (int e = 0; e < 32; ++e)  // (codes of odd channels were 16 times as large)
                    o[e] = fmaf(o[e], e & 2 ? 0.0625f : 1.f, cr);
                if constexpr (NCP > 1) {
                    // copies 1.. pass their 32 columns through shared memory (16-byte chunk k of
                    // row r in slot k ^ (r & 7))
                    if (cp > 0) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            s_o[((cp - 1) * RPC + r) * 8 + (k ^ (r & 7))] =
                                make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
                    }
                    asm volatile("bar.sync 1, 128;" ::: "memory");
                    if (cp == 0) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            float4 a = make_float4(fq[0] * o[4 * k], fq[0] * o[4 * k + 1],
                                                   fq[0] * o[4 * k + 2], fq[0] * o[4 * k + 3]);
#pragma unroll
                            for (int q = 1; q < NCP; ++q) {
                                const float4 x = s_o[((q - 1) * RPC + r) * 8 + (k ^ (r & 7))];
                                a.x = fmaf(fq[q], x.x, a.x);
                                a.y = fmaf(fq[q], x.y, a.y);
                                a.z = fmaf(fq[q], x.z, a.z);
                                a.w = fmaf(fq[q], x.w, a.w);
                            }
                            o[4 * k] = a.x;
                            o[4 * k + 1] = a.y;
                            o[4 * k + 2] = a.z;
                            o[4 * k + 3] = a.w;
                        }
                    }
                    asm volatile("bar.sync 1, 128;" ::: "memory");
                }
                if (!row_ok || cp != 0 || !read_o) continue;
                // columns to channels: group of 8 by group of 8
                if (starts && ends) {
                    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<unsigned short *>(p.out) +
                                                           ((int64_t)row * p.h_q + h) * D + c * 32);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float *x = o + 8 * k;
                        dst[k] = make_uint4(
                            pack_bf16(x[col_of(0)] * inv, x[col_of(1)] * inv),
                            pack_bf16(x[col_of(2)] * inv, x[col_of(3)] * inv),
                            pack_bf16(x[col_of(4)] * inv, x[col_of(5)] * inv),
                            pack_bf16(x[col_of(6)] * inv, x[col_of(7)] * inv));
                    }
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(kv4_slot_o(p, slot, r) + c * 32);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float *x = o + 8 * k;
                        dst[2 * k] = make_float4(x[col_of(0)], x[col_of(1)], x[col_of(2)], x[col_of(3)]);
                        dst[2 * k + 1] =
                            make_float4(x[col_of(4)], x[col_of(5)], x[col_of(6)], x[col_of(7)]);
                    }
                    if (c == 0) {
                        float *ml = kv4_slot_ml(p, slot, r);
                        ml[0] = m;
                        ml[1] = l;
                    }
                }
            }
            if (warp == 0 && lane == 0 && !p.whole) {
                int *uc = reinterpret_cast<int *>(kv4_unit_ctas(p) + (int64_t)u.b * p.h_kv + u.g);
                if (starts) uc[0] = blockIdx.x;
                if (ends) uc[1] = blockIdx.x;
            }
            u = nx;
        }
    }
    tc_before();
    __syncthreads();
    tc_after();
    if (warp == kSWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem),
                     "r"(kTmemCols)
                     : "memory");
}

template <int D, int NCP>
cudaError_t launch_t(const Kv4Params &p, cudaStream_t s) {
    constexpr int bytes = TcCfg<D>::kSmem;
    cudaError_t e = set_max_dynamic_smem<kv4_tc_kernel<D, NCP>>(bytes);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kv4_tc_kernel<D, NCP>, dim3(p.ctas), dim3(kThreads), bytes, s, p);
    return e != cudaSuccess || p.whole ? e : launch_kv4_merge(p, s);
}

template <int D>
cudaError_t launch_d(const Kv4Params &p, cudaStream_t s) {
    const int rows = p.group * p.max_q_rows;
    return rows <= 32 ? launch_t<D, 4>(p, s) : rows <= 64 ? launch_t<D, 2>(p, s) : launch_t<D, 1>(p, s);
}

}  // namespace

int kv4_tc_max_rows() { return kRows; }

void kv4_tc_plan(int *tile, int *ctas_per_sm) {
    *tile = kTile;
    *ctas_per_sm = 1;
}

cudaError_t launch_kv4_tc(const Kv4Params &p, cudaStream_t s) {
    return p.head_dim == 128 ? launch_d<128>(p, s) : launch_d<64>(p, s);
}

}  // namespace sd
