// Joins the partial results of units that several CTAs of a 4-bit attention call shared.
//
// One block per (unit, row): O = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i over the unit's
// partial slots, M their largest maximum.  The threads form NT / D groups that take every (NT/D)-th
// slot and are added in group order, so the result does not depend on timing.  Bound by load
// latency, so a thread's first eight outputs are loaded together with the statistics, before their
// weights are known, and a unit of one long sequence, which up to 2 x 148 CTAs share, gets four
// groups (1,024 bytes of a row in flight per slot and group).
#include "kv4_common.cuh"

namespace sd {
namespace {

constexpr int kMaxSlots = 1024;  // of one unit: at most the launch's CTAs, or its splits
constexpr int kPre = 8;          // outputs of a thread loaded with the statistics

template <typename T, int D, int kThreads>
__global__ void __launch_bounds__(kThreads) kv4_merge_kernel(const Kv4Params p) {
    pdl_trigger();  // (see launch_pdl)
    pdl_wait();
    __shared__ float s_w[kMaxSlots];
    __shared__ float s_f[kThreads / 32];
    __shared__ float s_o[kThreads];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int u = blockIdx.x, lr = blockIdx.y, b = u / p.h_kv, g = u % p.h_kv;
    int q0, n_q, kv_len;
    bool bad;
    if (!kv4_sequence(p, b, q0, n_q, kv_len, bad) || lr >= n_q * p.group) return;
    int64_t first, step;  // slots first, first + step, ... (tensor cores: after the first one)
    int n;
    if (p.ctas) {
        const int2 c = ld_dep(kv4_unit_ctas(p) + u);
        n = c.y - c.x + 1;
        if (n == 1) return;  // the output is there already
        first = 2 * (int64_t)c.x;
        step = 2;
    } else {
        n = p.n_splits;
        first = (int64_t)u * n;
        step = 1;
    }
    auto slot = [&](int i) { return first + i * step + (p.ctas && i == 0 ? 1 : 0); };
    constexpr int kGroups = kThreads / D;
    const int col = tid % D, grp = tid / D;
    float pre[kPre];
#pragma unroll
    for (int k = 0; k < kPre; ++k) {
        const int i = grp + k * kGroups;
        pre[k] = i < n ? kv4_slot_o(p, slot(i), lr)[col] : 0.f;
    }
    float M = -INFINITY;
    for (int i = tid; i < n; i += kThreads) M = fmaxf(M, s_w[i] = kv4_slot_ml(p, slot(i), lr)[0]);
    M = warp_max(M);
    if (lane == 0) s_f[warp] = M;
    __syncthreads();
    M = s_f[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) M = fmaxf(M, s_f[w]);
    __syncthreads();
    float L = 0.f;
    for (int i = tid; i < n; i += kThreads) {
        const float w = s_w[i] == -INFINITY ? 0.f : exp2f(s_w[i] - M);
        s_w[i] = w;
        L += w * kv4_slot_ml(p, slot(i), lr)[1];
    }
    L = warp_sum(L);
    if (lane == 0) s_f[warp] = L;
    __syncthreads();
    L = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) L += s_f[w];
    float acc = 0.f;
#pragma unroll
    for (int k = 0; k < kPre; ++k) {
        const int i = grp + k * kGroups;
        if (i < n) acc = fmaf(s_w[i], pre[k], acc);
    }
#pragma unroll 8
    for (int i = grp + kPre * kGroups; i < n; i += kGroups)
        acc = fmaf(s_w[i], kv4_slot_o(p, slot(i), lr)[col], acc);
    s_o[tid] = acc;
    __syncthreads();
    if (grp) return;
#pragma unroll
    for (int q = 1; q < kGroups; ++q) acc += s_o[q * D + col];
    const float o = L == 0.f ? 0.f : acc / L;  // (a NaN sum gives NaN)
    const int64_t at = ((int64_t)(q0 + lr / p.group) * p.h_q + g * p.group + lr % p.group) * D + col;
    if constexpr (sizeof(T) == 4)
        static_cast<float *>(p.out)[at] = o;
    else
        static_cast<unsigned short *>(p.out)[at] = (unsigned short)f32_to_bf16_bits(o);
}

template <typename T, int D>
cudaError_t launch_d(const Kv4Params &p, cudaStream_t s) {
    const dim3 grid(p.batch * p.h_kv, p.group * p.max_q_rows);
    // slots that a unit has on average (two more where its ends are shared)
    const int slots = p.ctas ? p.ctas / (p.batch * p.h_kv) : p.n_splits;
    return slots > 8 ? launch_pdl(kv4_merge_kernel<T, D, 4 * D>, grid, dim3(4 * D), 0, s, p)
                     : launch_pdl(kv4_merge_kernel<T, D, D>, grid, dim3(D), 0, s, p);
}

}  // namespace

cudaError_t launch_kv4_merge(const Kv4Params &p, cudaStream_t s) {
    if (p.dtype == SD_BF16)
        return p.head_dim == 128 ? launch_d<unsigned short, 128>(p, s)
                                 : launch_d<unsigned short, 64>(p, s);
    return p.head_dim == 128 ? launch_d<float, 128>(p, s) : launch_d<float, 64>(p, s);
}

}  // namespace sd
