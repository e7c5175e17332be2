// C ABI of the operators between the products (declared in include/qgemv.h):
// the norms, the rotation, the paged 8-bit cache with its tables, its append
// and its attention, and the sampling behind the last product.  As in capi.hip,
// arguments are checked on the host before any HIP call.
#include <cmath>
#include <cstdint>

#include "../../include/qgemv.h"
#include "kv_cache.h"
#include "qk_rope.h"
#include "rmsnorm.h"
#include "sample.h"

namespace {

using namespace qg;

constexpr int64_t INT32_END = int64_t(1) << 31;
constexpr int64_t ROWS_MAX = int64_t(1) << 30;
// A launch has fewer than 2^32 threads: the norm takes up to 1024 a row, the
// append 8 a token, the attention's join 64 a row and head, in workgroups of 8.
constexpr int64_t NORM_ROWS_MAX = (int64_t(1) << 22) - 1;
constexpr int64_t APPEND_TOKENS_MAX = int64_t(1) << 28;
constexpr int64_t JOINS_MAX = (int64_t(1) << 26) - 8;
// (the rotation takes 64 a token, more only of up to 2048 tokens)
constexpr int64_t ROPE_TOKENS_MAX = (int64_t(1) << 26) - 8;
// (the sampling takes a workgroup of 256 for each chunk of a row)
constexpr int64_t SAMPLE_GROUPS_MAX = (int64_t(1) << 24) - 1;
constexpr int64_t LEN_MAX = int64_t(1) << 30;
constexpr int64_t STRIDE_MAX = int64_t(1) << 31;

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

int hip_status(hipError_t e) { return e == hipSuccess ? QG_OK : QG_EHIP; }

bool page_size(int64_t page) { return page == 32 || page == 64 || page == 128 || page == 256; }

bool head_size(int64_t D) { return D == 64 || D == 128 || D == 256; }

int check_cache(const qg_kv_cache *c) {
    if (!c) return QG_EINVAL;
    if (c->fmt != QG_KV_INT8 && c->fmt != QG_KV_E4M3) return QG_EINVAL;
    if (!page_size(c->page) || !head_size(c->D) || c->Hkv < 1 || c->Hkv > 1024 || c->pages < 1 ||
        c->pages >= INT32_END / c->page)
        return QG_ESHAPE;
    if (!c->k || !c->v || !c->k_scales || !c->v_scales) return QG_EINVAL;
    if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scales, 4) || !aligned(c->v_scales, 4))
        return QG_EALIGN;
    return QG_OK;
}

bool row_stride(int64_t stride, int64_t width) { return stride >= width && stride % 8 == 0 && stride < STRIDE_MAX; }

// Where a sampling call's workspace holds what, from its start on; the last
// is its size.  False: refused.
struct SampleLayout {
    int64_t chunks;
    size_t rows, masses, counts, kept, tops, top_at, lists, bytes;
};
bool sample_layout(int64_t M, int64_t V, SampleLayout *l) {
    if (M < 0 || V < 1 || V > SAMPLE_V_MAX) return false;
    l->chunks = (V + SAMPLE_CHUNK - 1) / SAMPLE_CHUNK;
    if (M > SAMPLE_GROUPS_MAX / l->chunks) return false;
    size_t at = 0;
    const auto take = [&](size_t each) {
        const size_t here = at;
        at += (each * (size_t)M + 255) / 256 * 256;
        return here;
    };
    const size_t C = (size_t)l->chunks;
    l->rows = take(sizeof(SampleRow));
    l->masses = take(8 * SAMPLE_BINS);
    l->counts = take(4 * SAMPLE_BINS);
    l->kept = take(8 * C * SAMPLE_SUBS);
    l->tops = take(4 * C * SAMPLE_SUBS);
    l->top_at = take(4 * C * SAMPLE_SUBS);
    l->lists = take(8 * SAMPLE_LIST);
    l->bytes = at;
    return true;
}

// shape rules and plan of an attention call (false: refused)
bool attention_plan(int64_t R, int64_t M, int64_t Hq, int64_t Hkv, int64_t D, int64_t page,
                    int64_t max_q, int64_t max_len, int64_t window, KvAttnPlan *p, size_t *bytes) {
    if (R < 0 || R > KV_R_MAX || M < 0 || M > ROWS_MAX || Hkv < 1 || Hkv > 1024 || Hq < 1 || Hq > 8192 ||
        Hq % Hkv || !head_size(D) || !page_size(page) || max_q < 1 || max_q > KV_ROWS_MAX ||
        max_len < 1 || max_len > LEN_MAX || window < 0 || window > LEN_MAX || R * max_q * Hq > JOINS_MAX)
        return false;
    const int64_t seen = window > 0 && window + max_q - 1 < max_len ? window + max_q - 1 : max_len;
    if (!kv_attention_plan(R, Hkv, Hq / Hkv, D, max_q, seen, p)) return false;
    *bytes = R == 0 || M == 0 ? 0 : (size_t)p->head_bytes + (size_t)p->part_slots * (size_t)p->part_rows * (size_t)(D + 2) * 4;
    return true;
}

// the same behind a shared prefix
bool prefix_plan(int64_t R, int64_t M, int64_t Hq, int64_t Hkv, int64_t D, int64_t page, int64_t max_q,
                 int64_t max_len, int64_t max_prefix, KvPrefixPlan *p) {
    if (R < 0 || R > KV_R_MAX || M < 0 || Hkv < 1 || Hkv > 1024 || Hq < 1 || Hq > 8192 || Hq % Hkv ||
        M > JOINS_MAX / Hq || !head_size(D) || !page_size(page) || max_q < 1 || max_q > KV_ROWS_MAX ||
        max_len < 1 || max_len > LEN_MAX || max_prefix < 0 || max_prefix > LEN_MAX || R * max_q * Hq > JOINS_MAX)
        return false;
    return kv_prefix_plan(R, M, Hkv, Hq / Hkv, D, max_q, max_len, max_prefix, p);
}

}  // namespace

extern "C" {

int rmsnorm_quant_run(const void *x, int x_dtype, const void *residual, void *residual_out,
                      int res_dtype, const void *weight, float eps, const int8_t *signs,
                      int64_t M, int64_t K, void *y, int8_t *Xq, float *x_scales, void *stream) {
    try {
        for (const int t : {x_dtype, res_dtype}) {
            if (t == QG_OUT_I32_GROUPS) return QG_EUNSUPPORTED;
            if (t != QG_OUT_BF16 && t != QG_OUT_F32) return QG_EINVAL;
        }
        if (M < 0 || M > NORM_ROWS_MAX || K < 32 || K > RMS_K_MAX || K % 32) return QG_ESHAPE;
        if (!x || !weight || (!y && !Xq) || (Xq != nullptr) != (x_scales != nullptr) ||
            (signs && !Xq) || (residual_out && !residual))
            return QG_EINVAL;
        if (!(eps > 0.f) || !std::isfinite(eps)) return QG_EINVAL;
        if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(residual_out, 16) ||
            !aligned(weight, 16) || !aligned(signs, 16) || !aligned(y, 16) || !aligned(Xq, 16) ||
            !aligned(x_scales, 4))
            return QG_EALIGN;
        if (M == 0) return QG_OK;
        RmsArgs a;
        a.x = x;
        a.residual = residual;
        a.residual_out = residual_out;
        a.weight = reinterpret_cast<const uint16_t *>(weight);
        a.signs = signs;
        a.y = reinterpret_cast<uint16_t *>(y);
        a.Xq = Xq;
        a.x_scales = x_scales;
        a.denom = signs ? 127.0 * std::sqrt(32.0) : 127.0;
        a.M = M;
        a.K = (int)K;
        a.eps = eps;
        return hip_status(launch_rmsnorm(a, x_dtype == QG_OUT_F32,
                                         !residual ? 0 : res_dtype == QG_OUT_F32 ? 2 : 1,
                                         reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return QG_EINTERNAL;
    }
}

int qk_norm_rope_run(const void *q, int64_t q_stride, const void *k, int64_t k_stride, int x_dtype,
                     int64_t M, int64_t Hq, int64_t Hkv, int64_t D, const void *q_weight,
                     const void *k_weight, float eps, const int32_t *positions, int axes,
                     const uint8_t *axis, const float *inv_freq, int64_t rotated, int interleaved,
                     void *q_out, int64_t q_out_stride, void *k_out, int64_t k_out_stride,
                     void *stream) {
    try {
        if (x_dtype == QG_OUT_I32_GROUPS) return QG_EUNSUPPORTED;
        if ((x_dtype != QG_OUT_BF16 && x_dtype != QG_OUT_F32) || (interleaved != 0 && interleaved != 1))
            return QG_EINVAL;
        if (M < 0 || M > ROPE_TOKENS_MAX || Hq < 0 || Hq > 8192 || Hkv < 0 || Hkv > 1024 || D < 8 ||
            D > ROPE_D_MAX || D % 8 || rotated < 0 || rotated > D || rotated % 16 || axes < 1 || axes > 4 ||
            (Hq > 0 && (!row_stride(q_stride, Hq * D) || !row_stride(q_out_stride, Hq * D))) ||
            (Hkv > 0 && (!row_stride(k_stride, Hkv * D) || !row_stride(k_out_stride, Hkv * D))))
            return QG_ESHAPE;
        if ((Hq > 0 && (!q || !q_out)) || (Hkv > 0 && (!k || !k_out)) || (rotated > 0 && (!positions || !inv_freq)))
            return QG_EINVAL;
        if ((q_weight || k_weight) && (!(eps > 0.f) || !std::isfinite(eps))) return QG_EINVAL;
        if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16) ||
            !aligned(positions, 4) || !aligned(inv_freq, 4) || !aligned(q_out, 16) || !aligned(k_out, 16))
            return QG_EALIGN;
        if (M == 0 || Hq + Hkv == 0) return QG_OK;
        QkRopeArgs a;
        a.q = q;
        a.k = k;
        a.q_weight = reinterpret_cast<const uint16_t *>(q_weight);
        a.k_weight = reinterpret_cast<const uint16_t *>(k_weight);
        a.positions = positions;
        a.axis = axis;
        a.inv_freq = inv_freq;
        a.q_out = reinterpret_cast<uint16_t *>(q_out);
        a.k_out = reinterpret_cast<uint16_t *>(k_out);
        a.q_stride = q_stride;
        a.k_stride = k_stride;
        a.qo_stride = q_out_stride;
        a.ko_stride = k_out_stride;
        a.M = (int)M;
        a.Hq = (int)Hq;
        a.H = (int)(Hq + Hkv);
        a.D = (int)D;
        a.half = (int)(rotated / 2);
        a.axes = axes;
        a.parts = a.per_wave = 0;
        a.eps = eps;
        return hip_status(launch_qk_rope(a, x_dtype == QG_OUT_F32, interleaved != 0, reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return QG_EINTERNAL;
    }
}

int kv_tables_run(int64_t R, int64_t page, int64_t pages, int64_t max_blocks, int64_t max_tokens,
                  int32_t *lens, const int32_t *keep, const int32_t *add, int32_t *table,
                  int32_t *free_pages, int32_t *free_count, int32_t *q_start, int32_t *slots,
                  int32_t *positions, int32_t *status, void *stream) {
    try {
        if (R < 0 || R > KV_R_MAX || !page_size(page) || pages < 1 || pages >= INT32_END / page ||
            max_blocks < 1 || max_blocks > LEN_MAX / page || max_tokens < 0 || max_tokens > ROWS_MAX)
            return QG_ESHAPE;
        if ((R > 0 && (!lens || !add || !table)) || !free_pages || !free_count || !q_start || !status ||
            (max_tokens > 0 && (!slots || !positions)))
            return QG_EINVAL;
        for (const void *p : {(const void *)lens, (const void *)keep, (const void *)add,
                              (const void *)table, (const void *)free_pages,
                              (const void *)free_count, (const void *)q_start,
                              (const void *)slots, (const void *)positions, (const void *)status})
            if (!aligned(p, 4)) return QG_EALIGN;
        KvTablesArgs a;
        a.lens = lens;
        a.table = table;
        a.free_pages = free_pages;
        a.free_count = free_count;
        a.keep = keep;
        a.add = add;
        a.q_start = q_start;
        a.slots = slots;
        a.positions = positions;
        a.status = status;
        a.pages = pages;
        a.R = (int)R;
        a.page = (int)page;
        a.max_blocks = (int)max_blocks;
        a.max_tokens = (int)max_tokens;
        return hip_status(launch_kv_tables(a, reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return QG_EINTERNAL;
    }
}

int kv_append_run(const qg_kv_cache *cache, int64_t M, const void *K, int64_t k_stride,
                  const void *V, int64_t v_stride, const int32_t *slots, void *stream) {
    try {
        const int st = check_cache(cache);
        if (st != QG_OK) return st;
        const int64_t width = (int64_t)cache->Hkv * cache->D;
        if (M < 0 || M > APPEND_TOKENS_MAX || !row_stride(k_stride, width) || !row_stride(v_stride, width))
            return QG_ESHAPE;
        if (!K || !V || !slots) return QG_EINVAL;
        if (!aligned(K, 16) || !aligned(V, 16) || !aligned(slots, 4)) return QG_EALIGN;
        if (M == 0) return QG_OK;
        KvAppendArgs a;
        a.k = reinterpret_cast<uint8_t *>(cache->k);
        a.v = reinterpret_cast<uint8_t *>(cache->v);
        a.k_scales = cache->k_scales;
        a.v_scales = cache->v_scales;
        a.K = reinterpret_cast<const uint16_t *>(K);
        a.V = reinterpret_cast<const uint16_t *>(V);
        a.slots = slots;
        a.k_stride = k_stride;
        a.v_stride = v_stride;
        a.slots_end = cache->pages * cache->page;
        a.M = (int)M;
        a.Hkv = cache->Hkv;
        a.D = cache->D;
        a.page = cache->page;
        return hip_status(launch_kv_append(a, cache->fmt == QG_KV_E4M3, reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return QG_EINTERNAL;
    }
}

size_t qg_kv_attention_workspace_bytes(int64_t R, int64_t M, int64_t Hq, int64_t Hkv, int64_t D,
                                       int64_t page, int64_t max_q, int64_t max_len,
                                       int64_t window) {
    KvAttnPlan p;
    size_t bytes = 0;
    return attention_plan(R, M, Hq, Hkv, D, page, max_q, max_len, window, &p, &bytes) ? bytes : 0;
}

int kv_attention_run(const qg_kv_cache *cache, int64_t R, int64_t M, int64_t Hq, const void *q,
                     int64_t q_stride, const int32_t *q_start, const int32_t *lens,
                     const int32_t *table, int64_t max_blocks, const uint32_t *tree_mask,
                     int64_t window, float scale, int64_t max_q, int64_t max_len,
                     void *workspace, size_t workspace_bytes, void *out, int64_t out_stride,
                     int out_dtype, void *stream) {
    try {
        if (out_dtype != QG_OUT_BF16 && out_dtype != QG_OUT_F32 && out_dtype != QG_OUT_I32_GROUPS)
            return QG_EINVAL;
        if (out_dtype == QG_OUT_I32_GROUPS || (tree_mask && window != 0)) return QG_EUNSUPPORTED;
        const int st = check_cache(cache);
        if (st != QG_OK) return st;
        KvAttnPlan p;
        size_t need = 0;
        if (max_blocks < 1 || max_blocks > LEN_MAX / cache->page ||
            max_len > max_blocks * cache->page ||
            !attention_plan(R, M, Hq, cache->Hkv, cache->D, cache->page, max_q, max_len, window, &p, &need) ||
            !row_stride(q_stride, Hq * cache->D) || !row_stride(out_stride, Hq * cache->D))
            return QG_ESHAPE;
        const float scale2 = scale * 1.44269504088896340736f;  // scores in powers of two
        if (!std::isfinite(scale2)) return QG_EINVAL;
        if (!q || !q_start || !lens || !table || !out || (need && !workspace)) return QG_EINVAL;
        if (need && workspace_bytes < need) return QG_ESIZE;
        if (!aligned(q, 16) || !aligned(q_start, 4) || !aligned(lens, 4) || !aligned(table, 4) ||
            !aligned(tree_mask, 4) || !aligned(workspace, 16) || !aligned(out, 16))
            return QG_EALIGN;
        if (R == 0 || M == 0) return QG_OK;
        KvAttnArgs a{};
        a.k = reinterpret_cast<const uint8_t *>(cache->k);
        a.v = reinterpret_cast<const uint8_t *>(cache->v);
        a.k_scales = cache->k_scales;
        a.v_scales = cache->v_scales;
        a.q = reinterpret_cast<const uint16_t *>(q);
        a.q_start = q_start;
        a.lens = lens;
        a.table = table;
        a.tree = tree_mask;
        a.out = out;
        a.head = reinterpret_cast<int32_t *>(workspace);
        a.part = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(workspace) + p.head_bytes);
        a.part_ml = a.part + (size_t)p.part_slots * (size_t)p.part_rows * (size_t)cache->D;
        a.q_stride = q_stride;
        a.out_stride = out_stride;
        a.pages = cache->pages;
        a.R = (int)R;
        a.M = (int)M;
        a.Hq = (int)Hq;
        a.Hkv = cache->Hkv;
        a.G = (int)(Hq / cache->Hkv);
        a.page = cache->page;
        a.max_blocks = (int)max_blocks;
        a.max_q = (int)max_q;
        a.window = (int)window;
        a.max_len = (int)max_len;
        a.groups = p.groups;
        a.slots = p.slots;
        a.min_run = p.min_run;
        a.part_rows = p.part_rows;
        a.part_slots = (int)p.part_slots;
        a.whole = p.whole;
        a.aligned = p.aligned;
        a.scale = scale2;
        a.out_f32 = out_dtype == QG_OUT_F32;
        return hip_status(launch_kv_attention(a, cache->D, cache->fmt == QG_KV_E4M3,
                                              reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return QG_EINTERNAL;
    }
}

size_t qg_kv_prefix_attention_workspace_bytes(int64_t R, int64_t M, int64_t Hq, int64_t Hkv, int64_t D,
                                              int64_t page, int64_t max_q, int64_t max_len,
                                              int64_t max_prefix) {
    KvPrefixPlan p;
    return prefix_plan(R, M, Hq, Hkv, D, page, max_q, max_len, max_prefix, &p) && R > 0 && M > 0 ? p.bytes : 0;
}

int kv_prefix_attention_run(const qg_kv_cache *cache, int64_t R, int64_t M, int64_t Hq, const void *q,
                            int64_t q_stride, const int32_t *q_start, const int32_t *lens,
                            const int32_t *table, int64_t max_blocks, const int32_t *prefix_table,
                            int64_t prefix_blocks, const int32_t *prefix_len,
                            const uint32_t *tree_mask, float scale, int64_t max_q, int64_t max_len,
                            int64_t max_prefix, void *workspace, size_t workspace_bytes, void *out,
                            int64_t out_stride, int out_dtype, void *stream) {
    try {
        if (out_dtype != QG_OUT_BF16 && out_dtype != QG_OUT_F32 && out_dtype != QG_OUT_I32_GROUPS)
            return QG_EINVAL;
        if (out_dtype == QG_OUT_I32_GROUPS) return QG_EUNSUPPORTED;
        const int st = check_cache(cache);
        if (st != QG_OK) return st;
        KvPrefixPlan p;
        if (max_blocks < 1 || max_blocks > LEN_MAX / cache->page || max_len > max_blocks * cache->page ||
            prefix_blocks < 1 || prefix_blocks > LEN_MAX / cache->page || max_prefix > prefix_blocks * cache->page ||
            !prefix_plan(R, M, Hq, cache->Hkv, cache->D, cache->page, max_q, max_len, max_prefix, &p) ||
            !row_stride(q_stride, Hq * cache->D) || !row_stride(out_stride, Hq * cache->D))
            return QG_ESHAPE;
        const float scale2 = scale * 1.44269504088896340736f;  // scores in powers of two
        if (!std::isfinite(scale2)) return QG_EINVAL;
        const bool none = R == 0 || M == 0;
        if (!q || !q_start || !lens || !table || !prefix_table || !prefix_len || !out || (!none && !workspace))
            return QG_EINVAL;
        if (!none && workspace_bytes < p.bytes) return QG_ESIZE;
        if (!aligned(q, 16) || !aligned(q_start, 4) || !aligned(lens, 4) || !aligned(table, 4) || !aligned(prefix_table, 4) ||
            !aligned(prefix_len, 4) || !aligned(tree_mask, 4) || !aligned(workspace, 16) || !aligned(out, 16))
            return QG_EALIGN;
        if (none) return QG_OK;
        KvAttnArgs a{};
        a.k = reinterpret_cast<const uint8_t *>(cache->k);
        a.v = reinterpret_cast<const uint8_t *>(cache->v);
        a.k_scales = cache->k_scales;
        a.v_scales = cache->v_scales;
        a.q = reinterpret_cast<const uint16_t *>(q);
        a.q_start = q_start;
        a.lens = lens;
        a.table = table;
        a.tree = tree_mask;
        a.out = out;
        a.q_stride = q_stride;
        a.out_stride = out_stride;
        a.pages = cache->pages;
        a.R = (int)R;
        a.M = (int)M;
        a.Hq = (int)Hq;
        a.Hkv = cache->Hkv;
        a.G = (int)(Hq / cache->Hkv);
        a.page = cache->page;
        a.max_blocks = (int)max_blocks;
        a.max_q = (int)max_q;
        a.max_len = (int)max_len;
        a.scale = scale2;
        a.out_f32 = out_dtype == QG_OUT_F32;
        a.prefix_table = prefix_table;
        a.prefix_len = prefix_len;
        a.prefix_blocks = (int)prefix_blocks;
        a.max_prefix = (int)max_prefix;
        a.starts = p.own_starts;
        a.cuts = p.cuts;
        uint8_t *w = reinterpret_cast<uint8_t *>(workspace);
        const auto line = [&](const KvAttnPlan &l, size_t head, size_t part) {
            KvAttnArgs b = a;
            b.head = reinterpret_cast<int32_t *>(w + head);
            b.part = reinterpret_cast<float *>(w + part);
            b.part_ml = b.part + (size_t)l.part_slots * (size_t)l.part_rows * (size_t)cache->D;
            b.groups = l.groups;
            b.slots = l.slots;
            b.min_run = l.min_run;
            b.part_rows = l.part_rows;
            b.part_slots = (int)l.part_slots;
            b.aligned = l.aligned;
            return b;
        };
        KvAttnArgs own = line(p.own, 0, p.own_part);
        const KvAttnArgs pre = line(p.pre, (size_t)p.own.head_bytes, p.pre_part);
        own.pre_part = pre.part;
        own.pre_ml = pre.part_ml;
        own.pre_head = pre.head;
        own.pre_rw = p.pre_rw;
        own.pre_rows = pre.part_rows;
        own.pre_slots = pre.part_slots;
        return hip_status(launch_kv_prefix_attention(own, pre, p, cache->D, cache->fmt == QG_KV_E4M3,
                                                     reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return QG_EINTERNAL;
    }
}

size_t qg_sample_workspace_bytes(int64_t M, int64_t V) {
    SampleLayout l;
    return sample_layout(M, V, &l) ? l.bytes : 0;
}

int sample_run(const void *logits, int x_dtype, int64_t M, int64_t V, int64_t stride, const float *u,
               const float *temperature, const int32_t *top_k, const float *top_p, const float *min_p,
               void *workspace, size_t workspace_bytes, int32_t *tokens, float *logprobs, void *stream) {
    try {
        if (x_dtype == QG_OUT_I32_GROUPS) return QG_EUNSUPPORTED;
        if (x_dtype != QG_OUT_BF16 && x_dtype != QG_OUT_F32) return QG_EINVAL;
        SampleLayout l;
        if (!sample_layout(M, V, &l) || stride < V || stride >= STRIDE_MAX) return QG_ESHAPE;
        if (!logits || !u || !tokens || (M > 0 && !workspace)) return QG_EINVAL;
        if (workspace_bytes < l.bytes) return QG_ESIZE;
        if (!aligned(logits, x_dtype == QG_OUT_F32 ? 4 : 2) || !aligned(workspace, 16)) return QG_EALIGN;
        for (const void *p : {(const void *)u, (const void *)temperature, (const void *)top_k,
                              (const void *)top_p, (const void *)min_p, (const void *)tokens,
                              (const void *)logprobs})
            if (!aligned(p, 4)) return QG_EALIGN;
        if (M == 0) return QG_OK;
        uint8_t *w = reinterpret_cast<uint8_t *>(workspace);
        SampleArgs a;
        a.logits = logits;
        a.stride = stride;
        a.u = u;
        a.temperature = temperature;
        a.top_p = top_p;
        a.min_p = min_p;
        a.top_k = top_k;
        a.tokens = tokens;
        a.logprobs = logprobs;
        a.rows = reinterpret_cast<SampleRow *>(w + l.rows);
        a.masses = reinterpret_cast<unsigned long long *>(w + l.masses);
        a.counts = reinterpret_cast<unsigned *>(w + l.counts);
        a.kept = reinterpret_cast<unsigned long long *>(w + l.kept);
        a.tops = reinterpret_cast<float *>(w + l.tops);
        a.top_at = reinterpret_cast<int32_t *>(w + l.top_at);
        a.lists = reinterpret_cast<u32x2_t *>(w + l.lists);
        a.M = (int)M;
        a.V = (int)V;
        a.chunks = (int)l.chunks;
        // (151936 tokens, top-k and top-p: 1 row 21.7 us against 23.4, 16 rows 29.6
        // against 30.8, 24 rows, 912 workgroups, 32.5 against 33.0; 32000 tokens: 64
        // rows 29.4 against 29.6, 96 rows, 768 workgroups, 32.7 against 31.6, 128 rows
        // 36.6 against 33.5)
        a.few = M * l.chunks <= 640;
        return hip_status(launch_sample(a, x_dtype == QG_OUT_F32, reinterpret_cast<hipStream_t>(stream)));
    } catch (...) {
        return QG_EINTERNAL;
    }
}

}  // extern "C"
