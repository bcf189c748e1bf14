// Entry points of the decoder block's other operators: the paged cache, the
// rotary append, attention of one new token and the residual norm.  Arguments
// are checked here; include/scute.h has the contract.
#include <cmath>

#include "host.h"

using namespace scute;

namespace {

bool aligned(const void *p, size_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// log2 of a power of two, -1 of any other number.
int shift_of(int x) { return (x & (x - 1)) == 0 ? __builtin_ctz(x) : -1; }

int kv_esz(int dtype) { return dtype == SCUTE_KV_FP32 ? 4 : dtype == SCUTE_KV_BF16 ? 2 : 1; }

scute_status check_cache(scute_ctx *c, const scute_kv_cache *kv, KvView *out) {
    if (!kv || !kv->k || !kv->v) return fail(c, SCUTE_ERR_ARG, "null cache");
    if (c->dtype == SCUTE_FP32 ? kv->dtype != SCUTE_KV_FP32
                               : kv->dtype != SCUTE_KV_BF16 && kv->dtype != SCUTE_KV_E4M3)
        return fail(c, SCUTE_ERR_DTYPE, "cache dtype %d does not go with the context's", kv->dtype);
    if (kv->n_pages < 1 || kv->page_size < 1 || kv->kv_heads < 1 ||
        (int64_t)kv->n_pages * kv->page_size > 0x7fffffff)
        return fail(c, SCUTE_ERR_SHAPE, "cache of %d pages of %d tokens, %d heads", kv->n_pages, kv->page_size,
                    kv->kv_heads);
    if (kv->head_dim < 16 || kv->head_dim > SCUTE_MAX_HEAD_DIM || kv->head_dim % 16)
        return fail(c, SCUTE_ERR_SHAPE, "head_dim %d is not a multiple of 16 up to %d", kv->head_dim,
                    SCUTE_MAX_HEAD_DIM);
    const int64_t per16 = 16 / kv_esz(kv->dtype);
    for (int64_t s : {kv->page_stride, kv->token_stride, kv->head_stride})
        if (s < kv->head_dim || s % per16)
            return fail(c, SCUTE_ERR_SHAPE, "cache stride %lld is below head_dim or not a multiple of 16 bytes",
                        (long long)s);
    if (!aligned(kv->k, 16) || !aligned(kv->v, 16)) return fail(c, SCUTE_ERR_ARG, "cache pools must be 16-byte aligned");
    out->k = kv->k;
    out->v = kv->v;
    out->dtype = kv->dtype;
    out->n_pages = kv->n_pages;
    out->page_size = kv->page_size;
    out->heads = kv->kv_heads;
    out->dim = kv->head_dim;
    out->page_stride = kv->page_stride;
    out->token_stride = kv->token_stride;
    out->head_stride = kv->head_stride;
    out->table = kv->block_table;
    out->table_stride = kv->table_stride;
    out->table_cols = kv->table_cols;
    out->k_scale = kv->k_scale;
    out->v_scale = kv->v_scale;
    return SCUTE_OK;
}

}  // namespace

extern "C" {

scute_status scute_kv_resize(scute_ctx *c, const int32_t *len_in, const int32_t *len_new, int n_req,
                             int32_t *block_table, int64_t table_stride, int table_cols, int page_size,
                             int32_t *free_pages, int64_t n_free_max, const int32_t *free_in, int32_t *free_out,
                             int32_t *len_out, int32_t *cu_new, int32_t *slot_map, int32_t *positions,
                             int32_t *token_req, int64_t max_new, void *stream) {
    if (!c) return SCUTE_ERR_ARG;
    if (n_req < 0 || n_req > SCUTE_MAX_REQUESTS)
        return fail(c, SCUTE_ERR_ARG, "n_req = %d outside 0..%d", n_req, SCUTE_MAX_REQUESTS);
    if (max_new < 0 || max_new > (1 << 30) || n_free_max < 0 || n_free_max > 0x7fffffff)
        return fail(c, SCUTE_ERR_ARG, "max_new or n_free_max out of range");
    if (page_size < 1 || table_cols < 1 || table_stride < table_cols)
        return fail(c, SCUTE_ERR_SHAPE, "pages of %d tokens, %d table columns, row pitch %lld", page_size, table_cols,
                    (long long)table_stride);
    if ((int64_t)n_req * table_cols > 0x7fffffff || (int64_t)table_cols * page_size > 0x7fffffff)
        return fail(c, SCUTE_ERR_SHAPE, "block table beyond 2^31 - 1 entries, or a row beyond 2^31 - 1 tokens");
    if (!free_in || !free_out || !cu_new || (n_free_max > 0 && !free_pages) ||
        (n_req > 0 && (!len_in || !len_new || !block_table || !len_out)) ||
        (max_new > 0 && (!slot_map || !positions || !token_req)))
        return fail(c, SCUTE_ERR_ARG, "null argument");
    DeviceGuard dg(c->device);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    ResizeArgs a{};
    a.len_in = len_in;
    a.len_new = len_new;
    a.n_req = n_req;
    a.cols = table_cols;
    a.page_size = page_size;
    a.page_shift = shift_of(page_size);
    a.table = block_table;
    a.table_stride = table_stride;
    a.free_pages = free_pages;
    a.n_free_max = n_free_max;
    a.free_in = free_in;
    a.free_out = free_out;
    a.len_out = len_out;
    a.cu_new = cu_new;
    a.slot_map = slot_map;
    a.positions = positions;
    a.token_req = token_req;
    a.max_new = (int)max_new;
    const auto overlap = [](const int32_t *p, const int32_t *q, int64_t k) { return p < q + k && q < p + k; };
    a.in_place = free_in == free_out || overlap(len_in, len_out, n_req) || overlap(len_new, len_out, n_req) ||
                 overlap(len_in, free_out, n_req) || overlap(len_new, free_out, n_req) || overlap(len_out, free_in, n_req);
    a.ctr = c->srv_ctr;
    a.status = c->d_status;
    TimedLaunch tl{c, st};
    CU_TRY(c, tl.begin());
    CU_TRY(c, launch_kv_resize(a, c->num_sms, st));
    count_launch(c, 1);
    CU_TRY(c, tl.end(SCUTE_KIND_KV_RESIZE));
    return SCUTE_OK;
}

scute_status scute_rope_table(scute_ctx *c, float *cos_sin, int n_pos, int rotary_dim, double theta,
                              const double *inv_freq, void *stream) {
    if (!c) return SCUTE_ERR_ARG;
    if (!cos_sin) return fail(c, SCUTE_ERR_ARG, "null argument");
    if (n_pos < 1 || rotary_dim < 2 || rotary_dim % 2 || rotary_dim > SCUTE_MAX_HEAD_DIM)
        return fail(c, SCUTE_ERR_SHAPE, "rotary table of %d positions, %d elements", n_pos, rotary_dim);
    if (!inv_freq && !(theta > 0.0 && std::isfinite(theta))) return fail(c, SCUTE_ERR_ARG, "theta must be positive");
    DeviceGuard dg(c->device);
    CU_TRY(c, launch_rope_table(cos_sin, n_pos, rotary_dim, theta, inv_freq, reinterpret_cast<cudaStream_t>(stream)));
    count_launch(c, 1);
    return SCUTE_OK;
}

scute_status scute_kv_append(scute_ctx *c, const scute_kv_cache *kv, const int32_t *slot_map, int64_t n, const void *k,
                             int64_t k_stride, const void *v, int64_t v_stride, const void *q, int64_t q_stride,
                             int q_heads, void *q_out, int64_t q_out_stride, const scute_rope *rope, void *stream) {
    if (!c) return SCUTE_ERR_ARG;
    AppendArgs a{};
    scute_status s = check_cache(c, kv, &a.kv);
    if (s) return s;
    if (n < 0 || n > (1 << 24)) return fail(c, SCUTE_ERR_ARG, "n out of range");
    if (q && (q_heads < 1 || q_heads > (1 << 16))) return fail(c, SCUTE_ERR_SHAPE, "q_heads = %d", q_heads);
    const int64_t kv_row = (int64_t)kv->kv_heads * kv->head_dim, q_row = (int64_t)q_heads * kv->head_dim;
    if (k_stride < kv_row || v_stride < kv_row || (q && (q_stride < q_row || q_out_stride < q_row)))
        return fail(c, SCUTE_ERR_SHAPE, "a row stride is below heads * head_dim");
    if (q && !rope) return fail(c, SCUTE_ERR_ARG, "q without rotary positions");
    if (rope) {
        if (rope->rotary_dim < 2 || rope->rotary_dim % 2 || rope->rotary_dim > kv->head_dim || rope->n_pos < 1 ||
            rope->n_axes < 1 || rope->n_axes > 4)
            return fail(c, SCUTE_ERR_SHAPE, "rotary_dim %d, %d positions, %d axes", rope->rotary_dim, rope->n_pos,
                        rope->n_axes);
        int sum = 0;
        for (int i = 0; i < rope->n_axes; ++i) {
            const int part = rope->n_axes == 1 ? rope->rotary_dim / 2 : rope->section[i];
            if (part < 0 || part > rope->rotary_dim / 2) return fail(c, SCUTE_ERR_SHAPE, "rotary section %d", part);
            sum += part;
            a.bound[i] = sum;
        }
        for (int i = rope->n_axes; i < 4; ++i) a.bound[i] = sum;
        if (sum != rope->rotary_dim / 2)
            return fail(c, SCUTE_ERR_SHAPE, "rotary sections sum to %d, not %d", sum, rope->rotary_dim / 2);
        if (rope->axis_stride < 0) return fail(c, SCUTE_ERR_SHAPE, "negative axis stride");
    }
    if (n == 0) return SCUTE_OK;
    if (!slot_map || !k || !v || (q && !q_out) || (rope && (!rope->cos_sin || !rope->positions)))
        return fail(c, SCUTE_ERR_ARG, "null argument");
    if (!aligned(k, c->esz) || !aligned(v, c->esz) || !aligned(q, c->esz) || !aligned(q_out, c->esz))
        return fail(c, SCUTE_ERR_ARG, "an input is not aligned to its elements");
    DeviceGuard dg(c->device);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    a.slot_map = slot_map;
    a.n = (int)n;
    a.k = k;
    a.v = v;
    a.q = q;
    a.q_out = q_out;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_stride = q_stride;
    a.q_out_stride = q_out_stride;
    a.q_heads = q ? q_heads : 0;
    if (rope) {
        a.rot = rope->rotary_dim;
        a.interleaved = rope->interleaved != 0;
        a.n_axes = rope->n_axes;
        a.n_pos = rope->n_pos;
        a.cos_sin = rope->cos_sin;
        a.table16 = aligned(rope->cos_sin, 16) && rope->rotary_dim % 8 == 0;
        a.positions = rope->positions;
        a.axis_stride = rope->axis_stride;
    }
    a.status = c->d_status;
    TimedLaunch tl{c, st};
    CU_TRY(c, tl.begin());
    CU_TRY(c, launch_kv_append(c->dtype == SCUTE_FP32, a, c->num_sms, st));
    count_launch(c, 1);
    CU_TRY(c, tl.end(SCUTE_KIND_KV_APPEND));
    return SCUTE_OK;
}

scute_status scute_paged_attention(scute_ctx *c, const scute_kv_cache *kv, const scute_attention *t, void *stream) {
    if (!c) return SCUTE_ERR_ARG;
    if (!t) return fail(c, SCUTE_ERR_ARG, "null argument");
    AttendArgs a{};
    scute_status s = check_cache(c, kv, &a.kv);
    if (s) return s;
    if (t->n_req < 0 || t->n_req > SCUTE_MAX_REQUESTS)
        return fail(c, SCUTE_ERR_ARG, "n_req = %d outside 0..%d", t->n_req, SCUTE_MAX_REQUESTS);
    if (t->q_heads < 1 || t->q_heads % kv->kv_heads || t->q_heads > (1 << 16))
        return fail(c, SCUTE_ERR_SHAPE, "%d query heads on %d key/value heads", t->q_heads, kv->kv_heads);
    const int64_t row = (int64_t)t->q_heads * kv->head_dim, per16 = 16 / c->esz;
    if (t->q_stride < row || t->out_stride < row || t->q_stride % per16 || t->out_stride % per16)
        return fail(c, SCUTE_ERR_SHAPE, "q or out stride is below a row or not a multiple of 16 bytes");
    if (kv->table_cols < 1 || kv->table_stride < kv->table_cols ||
        (int64_t)kv->table_cols * kv->page_size > (1 << 30) ||
        (int64_t)kv->table_cols * kv->page_size * t->n_req > (1ll << 33))
        return fail(c, SCUTE_ERR_SHAPE, "block table of %d columns, row pitch %lld", kv->table_cols,
                    (long long)kv->table_stride);
    if (!std::isfinite(t->scale) || !std::isfinite(t->softcap) || t->softcap < 0.f || t->window < 0)
        return fail(c, SCUTE_ERR_ARG, "bad scale, softcap or window");
    if (t->n_req == 0) return SCUTE_OK;
    if (!t->q || !t->out || !t->kv_len || !kv->block_table) return fail(c, SCUTE_ERR_ARG, "null argument");
    if (!aligned(t->q, 16) || !aligned(t->out, 16)) return fail(c, SCUTE_ERR_ARG, "q and out must be 16-byte aligned");
    DeviceGuard dg(c->device);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    a.q = t->q;
    a.out = t->out;
    a.q_stride = t->q_stride;
    a.out_stride = t->out_stride;
    a.lse = t->lse;
    a.kv_len = t->kv_len;
    a.n_req = t->n_req;
    a.q_heads = t->q_heads;
    a.group = t->q_heads / kv->kv_heads;
    a.scale = t->scale != 0.f ? t->scale : 1.f / sqrtf((float)kv->head_dim);
    a.softcap = t->softcap;
    a.window = t->window;
    a.page_shift = shift_of(kv->page_size);
    a.part = c->att_part;
    a.ctr = c->srv_ctr + 1;
    a.status = c->d_status;
    a.hold = c->inject_attend ? 1 : 0;
    c->inject_attend = false;
    TimedLaunch tl{c, st};
    CU_TRY(c, tl.begin());
    CU_TRY(c, launch_attend(a, c->num_sms, st));
    count_launch(c, 1);
    CU_TRY(c, tl.end(SCUTE_KIND_ATTENTION));
    return SCUTE_OK;
}

scute_status scute_residual_norm(scute_ctx *c, const scute_norm *t, int64_t n, int d, void *stream) {
    if (!c) return SCUTE_ERR_ARG;
    if (!t) return fail(c, SCUTE_ERR_ARG, "null argument");
    if (n < 0 || n > (1 << 24)) return fail(c, SCUTE_ERR_ARG, "n out of range");
    if (d < 1 || d > SCUTE_MAX_NORM_DIM) return fail(c, SCUTE_ERR_SHAPE, "d = %d outside 1..%d", d, SCUTE_MAX_NORM_DIM);
    if (t->y_stride < d || (t->residual && t->residual_stride < d) ||
        (t->residual_out && t->residual_out_stride < d) || (t->out && t->out_stride < d) ||
        (t->gate_rows && t->gate_stride < d))
        return fail(c, SCUTE_ERR_SHAPE, "a row stride is below d");
    if (!(t->eps >= 0.f) || !std::isfinite(t->eps) || !std::isfinite(t->scale))
        return fail(c, SCUTE_ERR_ARG, "bad eps or scale");
    if (t->gate_vec && t->gate_rows) return fail(c, SCUTE_ERR_ARG, "two gates");
    if (!t->post_w && t->post_b) return fail(c, SCUTE_ERR_ARG, "post_b without post_w");
    if (n == 0) return SCUTE_OK;
    if (!t->out && !t->residual_out) return fail(c, SCUTE_ERR_ARG, "no output");
    if (!t->out && (t->pre_w || t->pre_b)) return fail(c, SCUTE_ERR_ARG, "pre_w or pre_b without out");
    if (!t->y) return fail(c, SCUTE_ERR_ARG, "null argument");
    for (const void *p : {t->y, t->residual, (const void *)t->residual_out, (const void *)t->out, t->gate_rows})
        if (!aligned(p, c->esz)) return fail(c, SCUTE_ERR_ARG, "an input is not aligned to its elements");
    DeviceGuard dg(c->device);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    NormArgs a{};
    a.y = t->y;
    a.residual = t->residual;
    a.residual_out = t->residual_out;
    a.out = t->out;
    a.y_stride = t->y_stride;
    a.residual_stride = t->residual_stride;
    a.residual_out_stride = t->residual_out_stride;
    a.out_stride = t->out_stride;
    a.post_w = t->post_w;
    a.post_b = t->post_b;
    a.pre_w = t->pre_w;
    a.pre_b = t->pre_b;
    a.gate_vec = t->gate_vec;
    a.gate_rows = t->gate_rows;
    a.gate_stride = t->gate_stride;
    a.scale = t->scale;
    a.eps = t->eps;
    a.layer = t->layer != 0;
    a.n = (int)n;
    a.d = d;
    TimedLaunch tl{c, st};
    CU_TRY(c, tl.begin());
    CU_TRY(c, launch_residual_norm(c->dtype == SCUTE_FP32, a, c->num_sms, st));
    count_launch(c, 1);
    CU_TRY(c, tl.end(SCUTE_KIND_NORM));
    return SCUTE_OK;
}

}  // extern "C"
