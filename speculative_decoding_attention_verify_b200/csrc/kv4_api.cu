// C-ABI entry points of the cache appends and of attention over a 4-bit cache: host-side
// validation and dispatch.  Every check runs before any launch.
#include <math.h>

#include "sd_internal.h"

using namespace sd;

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

bool dtype_ok(int dtype) { return dtype == SD_F32 || dtype == SD_BF16; }
bool head_dim_ok(int d) { return d == 64 || d == 128; }

// Geometry that both kinds of cache share (row strides >= 0).
bool paging_ok(int page_size, int64_t stride_b, int64_t stride_h, const int32_t *block_table,
               int max_pages, int num_pages) {
    if (page_size == 0) return stride_b >= 0 && stride_h >= 0;
    return page_size == kPageSize && block_table && max_pages >= 1 && num_pages >= 1;
}

sd_status check_kv4(const sd_kv4_desc *kv, int batch) {
    if (!kv || batch < 1 || batch > 65535 || !dtype_ok(kv->dtype) || kv->h_kv < 1 ||
        kv->h_kv > 65535 || !kv->k || !kv->v || !kv->k_param || !kv->v_param || !kv->kv_len)
        return SD_ERR_INVALID_ARG;
    if (!aligned(kv->k, 16) || !aligned(kv->v, 16) || !aligned(kv->k_param, 4) ||
        !aligned(kv->v_param, 4))
        return SD_ERR_INVALID_ARG;
    if (!paging_ok(kv->page_size, kv->stride_b, kv->stride_h, kv->block_table,
                   kv->max_pages_per_seq, kv->num_pages))
        return SD_ERR_INVALID_ARG;
    return head_dim_ok(kv->head_dim) ? SD_OK : SD_ERR_UNSUPPORTED;
}

// Frequencies in turns per position, in fp64 (see sd_rope_desc).
sd_status make_rope(const sd_rope_desc *r, int head_dim, RopeParams *out) {
    *out = RopeParams{};
    if (!r) return SD_OK;
    if (r->layout != SD_ROPE_HALF && r->layout != SD_ROPE_INTERLEAVED) return SD_ERR_INVALID_ARG;
    const int n = r->rotary_dim;
    if (n < 2 || n > head_dim || n % 2) return SD_ERR_INVALID_ARG;
    if (r->scaling < SD_ROPE_UNSCALED || r->scaling > SD_ROPE_YARN) return SD_ERR_INVALID_ARG;
    if (!(r->gain >= 0.f) || isinf(r->gain)) return SD_ERR_INVALID_ARG;
    out->layout = r->layout;
    out->rotary_dim = n;
    out->gain = r->gain > 0.f ? (double)r->gain : 1.0;
    const double two_pi = 6.283185307179586476925286766559;
    if (r->inv_freq) {
        for (int m = 0; m < n / 2; ++m) {
            if (!isfinite(r->inv_freq[m])) return SD_ERR_INVALID_ARG;
            out->turns[m] = (double)r->inv_freq[m] / two_pi;
        }
        return SD_OK;
    }
    const bool scaled = r->scaling != SD_ROPE_UNSCALED;
    if (!(r->theta > 0.f) || isinf(r->theta)) return SD_ERR_INVALID_ARG;
    if (scaled && (!(r->factor >= 1.f) || isinf(r->factor))) return SD_ERR_INVALID_ARG;
    double theta = r->theta;
    const double factor = scaled ? (double)r->factor : 1.0;
    if (r->scaling == SD_ROPE_NTK) {
        if (n < 4) return SD_ERR_INVALID_ARG;
        theta *= pow(factor, n / (n - 2.0));
    }
    double lo = 0.0, hi = 1.0;
    if (r->scaling == SD_ROPE_YARN) {
        if (!(r->theta > 1.f) || r->original_len < 1) return SD_ERR_INVALID_ARG;
        const double c = n / (2.0 * log(theta));
        lo = fmax(floor(c * log(r->original_len / (32.0 * two_pi))), 0.0);
        hi = fmin(ceil(c * log(r->original_len / two_pi)), n - 1.0);
        if (!(hi > lo)) hi = lo + 0.001;
        if (!(r->gain > 0.f)) out->gain = 0.1 * log(factor) + 1.0;
    }
    // theta^(-2m/n) as powers of one root, in long double: 64 products are off by less than an
    // eighth of a double's last place, and cost less than one pow
    const long double root = powl((long double)theta, -2.0L / n);
    long double power = 1.0L;
    for (int m = 0; m < n / 2; ++m, power *= root) {
        double f = (double)power;
        if (r->scaling == SD_ROPE_LINEAR) f /= factor;
        if (r->scaling == SD_ROPE_YARN) {
            const double t = fmin(1.0, fmax(0.0, (m - lo) / (hi - lo)));
            f = f * (1.0 - t) + f * t / factor;
        }
        out->turns[m] = f / two_pi;
    }
    return SD_OK;
}

// Checks of the rows of an append and their share of its parameters; *wide: 16-byte accesses fit.
sd_status fill_rows(const sd_rope_desc *rope, const sd_rows_desc *rows, int dtype, int h_kv,
                    int head_dim, int batch, void *q_out, AppendParams *p, bool *wide) {
    if (!rows || !rows->q_start || rows->h_q < 0 || rows->n_rows < 0 ||
        rows->n_rows > (1 << 30) || rows->max_kv_len < 1)
        return SD_ERR_INVALID_ARG;
    // (an empty tensor may have no address)
    if (rows->n_rows > 0 && (!rows->k || !rows->v || (rows->h_q > 0) != (rows->q != nullptr) ||
                             (rows->h_q > 0) != (q_out != nullptr)))
        return SD_ERR_INVALID_ARG;
    if (rows->h_q > 65535) return SD_ERR_INVALID_ARG;
    const int64_t kw = (int64_t)h_kv * head_dim, qw = (int64_t)rows->h_q * head_dim;
    if (rows->k_stride < kw || rows->v_stride < kw || (rows->h_q > 0 && rows->q_stride < qw))
        return SD_ERR_INVALID_ARG;
    if (rows->q && q_out == rows->q && rows->q_stride != qw) return SD_ERR_INVALID_ARG;
    const int esz = dtype == SD_BF16 ? 2 : 4;
    if (!aligned(rows->k, esz) || !aligned(rows->v, esz) || !aligned(rows->q, esz) ||
        !aligned(q_out, esz))
        return SD_ERR_INVALID_ARG;
    sd_status st = make_rope(rope, head_dim, &p->rope);
    if (st != SD_OK) return st;
    p->dtype = dtype;
    p->head_dim = head_dim;
    p->h_q = rows->h_q;
    p->h_kv = h_kv;
    p->batch = batch;
    p->n_rows = rows->n_rows;
    p->max_kv_len = rows->max_kv_len;
    p->q_start = rows->q_start;
    p->pos = rows->pos;
    p->q = rows->q;
    p->k = rows->k;
    p->v = rows->v;
    p->q_stride = rows->q_stride;
    p->k_stride = rows->k_stride;
    p->v_stride = rows->v_stride;
    p->q_out = q_out;
    const int64_t strides = (rows->q ? rows->q_stride : 0) | rows->k_stride | rows->v_stride;
    *wide = aligned(rows->q, 16) && aligned(rows->k, 16) && aligned(rows->v, 16) &&
            aligned(q_out, 16) && (strides * esz) % 16 == 0;
    return SD_OK;
}

sd_status status_of(cudaError_t e) { return e == cudaSuccess ? SD_OK : SD_ERR_CUDA; }

struct Kv4Plan {
    int n_splits, simt_slots;  // CUDA-core engine
    int ctas, tile;            // tensor-core engines (0 CTAs: neither serves this call)
    bool whole;                // their CTAs share whole units
    bool tcgen05;              // which of the two
    size_t ws_bytes;
};

sd_status plan_kv4(const sd_q_desc *q, const sd_kv4_desc *kv, int batch, Kv4Plan *plan) {
    sd_status st = check_kv4(kv, batch);
    if (st != SD_OK && st != SD_ERR_UNSUPPORTED) return st;
    if (!q || q->h_q < 1 || q->h_q % kv->h_kv != 0 || q->max_q_rows < 1 || q->max_kv_len < 1 ||
        !q->q_start || !(q->softmax_scale >= 0.f) || isinf(q->softmax_scale))
        return SD_ERR_INVALID_ARG;
    if (st != SD_OK) return st;
    const long long rows = (long long)(q->h_q / kv->h_kv) * q->max_q_rows;
    // (rows of all units, the grids of the merge, and positions rounded up to a tile's end)
    if (q->max_kv_len > (1 << 30) || (long long)batch * q->max_q_rows > (1LL << 30) || rows > 65535 ||
        (long long)batch * kv->h_kv > (1LL << 30))
        return SD_ERR_INVALID_ARG;
    *plan = Kv4Plan{};
    plan->n_splits = kv4_simt_splits(batch, kv->h_kv, (int)rows, q->max_kv_len);
    plan->simt_slots = plan->n_splits > 1 ? batch * kv->h_kv * plan->n_splits : 0;
    plan->tcgen05 = rows > kv4_mma_max_rows();
    if (kv->dtype == SD_BF16 && rows <= kv4_tc_max_rows()) {
        int per_sm = 1;
        if (plan->tcgen05)
            kv4_tc_plan(&plan->tile, &per_sm);
        else
            kv4_mma_plan(&plan->tile, &per_sm);
        const long long per_unit = ((long long)q->max_kv_len + plan->tile - 1) / plan->tile;
        const long long units = (long long)batch * kv->h_kv;
        const long long slots = (long long)device_sm_count() * per_sm;
        // Whole units per CTA, where the longest CTA then has few tiles more than with an even
        // share of all tiles: a share's end, its partial results and the launch that merges them
        // cost about as much as 4 tiles of the mma.sync kernel or 8 of the tcgen05 one.  (28
        // sequences, 4 KV heads: 7 rows at 1,024 positions 12.5 us whole, 18.2 shared, at 2,048
        // 17.3 and 20.7; 63 rows at 1,024 23.1 and 45.7.  8 sequences of 4,096, 7 rows: 26.7 and
        // 17.6.)  Not beyond 16 tiles, since sequences shorter than the hint leave CTAs idle.
        const long long longest = (units + slots - 1) / slots * per_unit;
        const long long even = (units * per_unit + slots - 1) / slots;
        plan->whole = per_unit <= 16 && longest <= even + (plan->tcgen05 ? 8 : 4);
        const long long n = plan->whole ? units : units * per_unit;
        plan->ctas = (int)(n < slots ? n : slots);
    }
    // (whichever engine the pointers' alignment leaves)
    const size_t slot = (size_t)rows * (kv->head_dim + 2) * sizeof(float);
    const size_t simt = plan->simt_slots * slot;
    // (and the CTAs of every unit)
    const size_t tc = !plan->ctas || plan->whole
                          ? 0
                          : 2 * plan->ctas * slot + (size_t)batch * kv->h_kv * 2 * sizeof(int32_t);
    plan->ws_bytes = simt > tc ? simt : tc;
    return SD_OK;
}

}  // namespace

extern "C" {

sd_status sd_kv_append(const sd_rope_desc *rope, const sd_rows_desc *rows, const sd_kv_desc *cache,
                       int32_t batch, void *q_out, int32_t *dev_err, void *stream) {
    SD_RANGE("sd_kv_append");
    if (!cache || batch < 1 || batch > 65535 || !dtype_ok(cache->dtype) || cache->h_kv < 1 ||
        cache->h_kv > 65535 || !cache->k || !cache->v || !cache->kv_len)
        return SD_ERR_INVALID_ARG;
    const int esz = cache->dtype == SD_BF16 ? 2 : 4;
    if (!aligned(cache->k, 16) || !aligned(cache->v, 16) ||
        !paging_ok(cache->page_size, cache->stride_b, cache->stride_h, cache->block_table,
                   cache->max_pages_per_seq, cache->num_pages))
        return SD_ERR_INVALID_ARG;
    if (cache->page_size == 0 &&
        (cache->stride_pos != cache->head_dim || (cache->stride_h * esz) % 16 != 0 ||
         (cache->stride_b * esz) % 16 != 0))
        return SD_ERR_INVALID_ARG;
    if (!head_dim_ok(cache->head_dim)) return SD_ERR_UNSUPPORTED;
    AppendParams p{};
    bool wide = false;
    sd_status st = fill_rows(rope, rows, cache->dtype, cache->h_kv, cache->head_dim, batch, q_out,
                             &p, &wide);
    if (st != SD_OK) return st;
    if (p.n_rows == 0) return SD_OK;
    p.kv_len = cache->kv_len;
    p.page_size = cache->page_size;
    p.k_cache = const_cast<void *>(cache->k);
    p.v_cache = const_cast<void *>(cache->v);
    p.stride_b = cache->stride_b;
    p.stride_h = cache->stride_h;
    p.block_table = cache->block_table;
    p.max_pages = cache->max_pages_per_seq;
    p.num_pages = cache->num_pages;
    p.dev_err = dev_err;
    return status_of(launch_append(p, wide, reinterpret_cast<cudaStream_t>(stream)));
}

sd_status sd_kv4_append(const sd_rope_desc *rope, const sd_rows_desc *rows,
                        const sd_kv4_desc *cache, int32_t batch, void *q_out, void *k_out,
                        void *v_out, int32_t *dev_err, void *stream) {
    SD_RANGE("sd_kv4_append");
    sd_status st = check_kv4(cache, batch);
    if (st != SD_OK) return st;
    AppendParams p{};
    bool wide = false;
    st = fill_rows(rope, rows, cache->dtype, cache->h_kv, cache->head_dim, batch, q_out, &p, &wide);
    if (st != SD_OK) return st;
    const int esz = cache->dtype == SD_BF16 ? 2 : 4;
    if (!aligned(k_out, esz) || !aligned(v_out, esz)) return SD_ERR_INVALID_ARG;
    if (p.n_rows == 0) return SD_OK;
    wide = wide && aligned(k_out, 16) && aligned(v_out, 16);
    p.kv4 = 1;
    p.k_out = k_out;
    p.v_out = v_out;
    p.kv_len = cache->kv_len;
    p.page_size = cache->page_size;
    p.k_cache = cache->k;
    p.v_cache = cache->v;
    p.k_param = static_cast<uint32_t *>(cache->k_param);
    p.v_param = static_cast<uint32_t *>(cache->v_param);
    p.stride_b = cache->stride_b;
    p.stride_h = cache->stride_h;
    p.block_table = cache->block_table;
    p.max_pages = cache->max_pages_per_seq;
    p.num_pages = cache->num_pages;
    p.dev_err = dev_err;
    return status_of(launch_append(p, wide, reinterpret_cast<cudaStream_t>(stream)));
}

sd_status sd_kv4_attention_workspace_size(const sd_q_desc *q, const sd_kv4_desc *kv, int32_t batch,
                                          size_t *bytes) {
    if (!bytes) return SD_ERR_INVALID_ARG;
    Kv4Plan plan;
    const sd_status st = plan_kv4(q, kv, batch, &plan);
    if (st == SD_OK) *bytes = plan.ws_bytes;
    return st;
}

sd_status sd_kv4_verify_attention(const sd_q_desc *q, const void *q_data, const sd_kv4_desc *kv,
                                  int32_t batch, void *out, void *workspace,
                                  size_t workspace_bytes, int32_t *dev_err, void *stream) {
    SD_RANGE("sd_kv4_verify_attention");
    Kv4Plan plan;
    sd_status st = plan_kv4(q, kv, batch, &plan);
    if (st != SD_OK) return st;
    const int esz = kv->dtype == SD_BF16 ? 2 : 4;
    if (!q_data || !out || !aligned(q_data, esz) || !aligned(out, esz)) return SD_ERR_INVALID_ARG;
    if (plan.ws_bytes &&
        (!workspace || plan.ws_bytes > workspace_bytes || !aligned(workspace, 16)))
        return SD_ERR_WORKSPACE;
    Kv4Params p{};
    p.k = static_cast<const unsigned char *>(kv->k);
    p.v = static_cast<const unsigned char *>(kv->v);
    p.kp = static_cast<const uint32_t *>(kv->k_param);
    p.vp = static_cast<const uint32_t *>(kv->v_param);
    p.page_size = kv->page_size;
    p.stride_b = kv->stride_b;
    p.stride_h = kv->stride_h;
    p.block_table = kv->block_table;
    p.max_pages = kv->max_pages_per_seq;
    p.num_pages = kv->num_pages;
    p.kv_len = kv->kv_len;
    p.dtype = kv->dtype;
    p.head_dim = kv->head_dim;
    p.h_kv = kv->h_kv;
    p.batch = batch;
    p.h_q = q->h_q;
    p.group = q->h_q / kv->h_kv;
    p.max_q_rows = q->max_q_rows;
    p.max_kv_len = q->max_kv_len;
    p.rows_cap = batch * q->max_q_rows;
    p.scale_log2 = (q->softmax_scale > 0.f ? q->softmax_scale
                                           : (float)(1.0 / sqrt((double)kv->head_dim))) * kLog2e;
    p.q = q_data;
    p.q_start = q->q_start;
    p.out = out;
    p.ws = static_cast<float *>(workspace);
    p.dev_err = dev_err;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (plan.ctas && aligned(q_data, 16) && aligned(out, 16)) {
        p.ctas = plan.ctas;
        p.tile = plan.tile;
        p.whole = plan.whole;
        p.n_slots = 2 * plan.ctas;
        p.wait_ns = wait_limit_ns();
        return status_of(plan.tcgen05 ? launch_kv4_tc(p, s) : launch_kv4_mma(p, s));
    }
    p.n_splits = plan.n_splits;
    p.n_slots = plan.simt_slots;
    return status_of(launch_kv4_simt(p, s));
}

}  // extern "C"
