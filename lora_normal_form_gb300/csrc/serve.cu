// Entry points of the decoder block's other operators: the paged cache and rows
// that share its pages, the rotary append, attention of one new token and the
// residual norm.  Arguments are checked here; include/scute.h has the contract.
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

// scute_kv_append, and with `norm` scute_kv_append_norm.
scute_status append(scute_ctx *c, const scute_kv_cache *kv, const int32_t *slot_map, int64_t n, const void *k, int64_t k_stride,
                    const void *v, int64_t v_stride, const void *q, int64_t q_stride, int q_heads, void *q_out,
                    int64_t q_out_stride, const scute_rope *rope, const scute_head_norm *norm, void *stream) {
    AppendArgs a{};
    scute_status s = check_cache(c, kv, &a.kv);
    if (s) return s;
    if (n < 0 || n > (1 << 24)) return fail(c, SCUTE_ERR_ARG, "n out of range");
    if (q && (q_heads < 1 || q_heads > (1 << 16))) return fail(c, SCUTE_ERR_SHAPE, "q_heads = %d", q_heads);
    const int64_t kv_row = (int64_t)kv->kv_heads * kv->head_dim, q_row = (int64_t)q_heads * kv->head_dim;
    if (k_stride < kv_row || v_stride < kv_row || (q && (q_stride < q_row || q_out_stride < q_row)))
        return fail(c, SCUTE_ERR_SHAPE, "a row stride is below heads * head_dim");
    if (q && !rope && !norm) return fail(c, SCUTE_ERR_ARG, "q without rotary positions");
    HeadNormArgs w{};
    if (norm) {
        if (!(norm->eps >= 0.f) || !std::isfinite(norm->eps)) return fail(c, SCUTE_ERR_ARG, "bad eps");
        if (!norm->q_w && !norm->k_w) return fail(c, SCUTE_ERR_ARG, "no weights to norm with");
        for (int64_t stride : {norm->q_w ? norm->q_w_stride : 0, norm->k_w ? norm->k_w_stride : 0})
            if (stride != 0 && stride < kv->head_dim)
                return fail(c, SCUTE_ERR_SHAPE, "norm weights %lld apart", (long long)stride);
        if ((q ? q_row : 0) + 2 * kv_row > 0x7fffffff)        // elements of a row are counted in 32 bits there
            return fail(c, SCUTE_ERR_UNSUPPORTED, "rows of %lld elements with norms", (long long)((q ? q_row : 0) + 2 * kv_row));
        if (!aligned(norm->q_w, 4) || !aligned(norm->k_w, 4)) return fail(c, SCUTE_ERR_ARG, "weights are not aligned to their elements");
        w.q_w = q ? norm->q_w : nullptr;
        w.k_w = norm->k_w;
        w.q_stride = norm->q_w ? norm->q_w_stride : 0;
        w.k_stride = norm->k_w ? norm->k_w_stride : 0;
        w.eps = norm->eps;
        w.layer = norm->layer != 0;
    }
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
    CU_TRY(c, norm ? launch_kv_append_norm(c->dtype == SCUTE_FP32, a, w, c->num_sms, st)
                   : launch_kv_append(c->dtype == SCUTE_FP32, a, c->num_sms, st));
    count_launch(c, 1);
    CU_TRY(c, tl.end(SCUTE_KIND_KV_APPEND));
    return SCUTE_OK;
}

// Windows and first tokens go to warps on their own (k_attend_own.cu) where there are two
// rows (of a request and key/value head) to an SM or, with more than eight query heads to
// a key, one; up to as many tokens as this.  Device times in us, by CTAs and by warps,
// heads of 128:
//     4 to a key, e4m3    64 requests, window 200 17.2 and 14.5, 1000 26.7 and 19.4, 8000 60.0
//                         and 50.4, 30000 152 and 132; 200, window 1000 64.1 and 36.8, 8000 162
//                         and 129; 40 (320 rows), window 200 12.4 and 14.0, 1000 18.8 and
//                         15.8; 16 (128 rows) 11.5 and 12.8, 12.3 and 14.3
//     the same, bf16      64 requests, 200 16.6 and 13.6, 2000 35.2 and 35.2, 4000 53.3 and
//                         55.6; 200, 200 33.6 and 24.4, 2000 90.6 and 89.6, 8000 243 and 253
//     16 to a key, e4m3   64 requests (256 rows), window 1000 32.8 and 21.4, 30000 161 and
//                         104; bf16 31.6 and 20.8, 169 and 143
//     1 to a key of 64, e4m3: 64 requests, window 4000 44.5 and 42.5, 30000 171 and 185
// One limit for each type, so that some shapes next to it are on the slower side: of these, 64
// requests with 4 to a key and 30000 e4m3 tokens (15 %), and 40 with a window of 200 (13 %).
int own_row_limit(int dtype, int group) { return group > 8 ? 0x7fffffff : dtype == SCUTE_KV_E4M3 ? 16384 : 2048; }

// The parts of scute_shared's workspace, and its bytes (-1: too large).
struct SharedWork {
    int64_t own_at, stat, o, own_rows, bytes;
};
SharedWork shared_work(int64_t n_req, int64_t q_heads, int64_t kv_heads, int64_t dim, int num_sms) {
    SharedWork w;
    w.own_rows = own_rows(n_req, (int)q_heads, (int)kv_heads, num_sms);
    const int64_t rows = w.own_rows + shared_rows(n_req, q_heads, num_sms);
    w.own_at = 16 * n_req * kv_heads;
    w.stat = (w.own_at + 8 * n_req + 31) / 32 * 32;
    w.o = (w.stat + 8 * rows + 31) / 32 * 32;
    w.bytes = rows > 0x7fffffff ? -1 : w.o + 4 * rows * dim;
    return w;
}

// scute_paged_attention, with sinks scute_paged_attention_sinks, with `sh`
// scute_paged_attention_shared.
scute_status attend(scute_ctx *c, const scute_kv_cache *kv, const scute_attention *t, int32_t sinks, const scute_shared *sh,
                    void *stream) {
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
    if (sinks < 0 || sinks > (1 << 30)) return fail(c, SCUTE_ERR_ARG, "sinks = %d outside 0..2^30", sinks);
    SharedWork w{};
    if (sh) {
        if (t->window != 0) return fail(c, SCUTE_ERR_ARG, "shared beginnings with a window");
        if (sh->n_groups < 0 || sh->n_groups > SCUTE_MAX_GROUPS)
            return fail(c, SCUTE_ERR_ARG, "n_groups = %d outside 0..%d", sh->n_groups, SCUTE_MAX_GROUPS);
        w = shared_work(t->n_req, t->q_heads, kv->kv_heads, kv->head_dim, c->num_sms);
        if (w.bytes < 0 || sh->work_bytes < w.bytes)
            return fail(c, SCUTE_ERR_ARG, "a workspace of %lld bytes, %lld needed", (long long)sh->work_bytes, (long long)w.bytes);
        if (t->n_req > 0 && sh->n_groups > 0 && (!sh->start || !sh->len || !sh->work)) return fail(c, SCUTE_ERR_ARG, "null argument");
        if (!aligned(sh->work, 32)) return fail(c, SCUTE_ERR_ARG, "the workspace must be 32-byte aligned");
    }
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
    a.sinks = sinks;
    a.page_shift = shift_of(kv->page_size);
    a.part = c->att_part;
    a.ctr = c->srv_ctr + 1;
    a.status = c->d_status;
    a.hold = c->inject_attend ? 1 : 0;
    c->inject_attend = false;
    // by type and size: heads that the shared kernel's tiles hold (its sums are those of
    // 16-bit products, and 128 elements and rows are what its tensor memory takes)
    const bool together = sh && sh->n_groups > 0 && kv->dtype != SCUTE_KV_FP32 && kv->head_dim <= SHARED_MAX_DIM &&
                          a.group <= SHARED_MAX_GROUP_HEADS && t->n_req * t->q_stride / 8 < 0x7fffffff;
    SharedArgs b{};
    if (sh) {
        a.start = sh->start;
        a.shared_len = sh->len;
        a.n_groups = sh->n_groups;
        a.always = sh->always != 0;
    }
    if (together) {
        char *work = static_cast<char *>(sh->work);
        b.kv = a.kv;
        b.q = a.q;
        b.q_stride = a.q_stride;
        b.kv_len = a.kv_len;
        b.n_req = a.n_req;
        b.group = a.group;
        b.tile_req = 128 / a.group;
        b.scale = a.scale;
        b.softcap = a.softcap;
        b.page_shift = a.page_shift;
        b.start = a.start;
        b.shared_len = a.shared_len;
        b.n_groups = a.n_groups;
        b.always = a.always;
        b.first_row = (int)w.own_rows;
        b.piece = reinterpret_cast<int4 *>(work);
        a.own_at = reinterpret_cast<int2 *>(work + w.own_at);
        b.stat = a.stat = reinterpret_cast<float2 *>(work + w.stat);
        b.o = a.part_o = reinterpret_cast<float *>(work + w.o);
        b.status = a.status;
        b.hold = a.hold;
    }
    // and with sinks by rows and visible tokens, where the parts find room in the context's workspace
    bool by_warps = false;
    if (sinks && t->window && kv->dtype != SCUTE_KV_FP32 && kv->head_dim <= SHARED_MAX_DIM &&
        (int64_t)t->window + sinks <= own_row_limit(kv->dtype, a.group) &&
        (int64_t)t->n_req * kv->kv_heads >= (a.group > 8 ? 1 : 2) * c->num_sms) {
        const int64_t rows = own_rows(t->n_req, t->q_heads, kv->kv_heads, c->num_sms), at = (2 * t->n_req + 7) / 8 * 8;
        by_warps = at + rows * (2 + kv->head_dim) <= (int64_t)attend_part_floats(c->num_sms);
        if (by_warps) {
            a.own_at = reinterpret_cast<int2 *>(c->att_part);
            a.part_o = c->att_part + at;
            a.stat = reinterpret_cast<float2 *>(a.part_o + rows * kv->head_dim);
        }
    }
    TimedLaunch tl{c, st};
    CU_TRY(c, tl.begin());
    if (together) {
        CU_TRY(c, launch_shared(b, c->num_sms, st));
        count_launch(c, 1);
    }
    CU_TRY(c, together   ? launch_attend_own(a, c->num_sms, st)
              : by_warps ? launch_attend_own_sinks(a, c->num_sms, st)
              : sinks && t->window ? launch_attend_sinks(a, c->num_sms, st)
                                   : launch_attend(a, c->num_sms, st));
    count_launch(c, 1);
    if (sh && !together && sh->n_groups > 0) {
        CU_TRY(c, launch_check_groups(a, st));
        count_launch(c, 1);
    }
    if (together || by_warps) {
        JoinArgs j{};
        j.piece = b.piece;
        j.own_at = a.own_at;
        j.stat = a.stat;
        j.o = a.part_o;
        j.v_scale = kv->v_scale;
        j.out = a.out;
        j.out_stride = a.out_stride;
        j.lse = a.lse;
        j.rows = a.n_req * a.q_heads;
        j.q_heads = a.q_heads;
        j.group = a.group;
        j.dim = kv->head_dim;
        CU_TRY(c, launch_join(j, together ? shared_parts(sh->n_groups, kv->kv_heads, c->num_sms) : 0, st));
        count_launch(c, 1);
    }
    CU_TRY(c, tl.end(SCUTE_KIND_ATTENTION));
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
    return append(c, kv, slot_map, n, k, k_stride, v, v_stride, q, q_stride, q_heads, q_out, q_out_stride, rope, nullptr, stream);
}

scute_status scute_kv_append_norm(scute_ctx *c, const scute_kv_cache *kv, const int32_t *slot_map, int64_t n, const void *k,
                                  int64_t k_stride, const void *v, int64_t v_stride, const void *q, int64_t q_stride,
                                  int q_heads, void *q_out, int64_t q_out_stride, const scute_rope *rope,
                                  const scute_head_norm *norm, void *stream) {
    if (!c) return SCUTE_ERR_ARG;
    if (!norm) return fail(c, SCUTE_ERR_ARG, "null argument");
    return append(c, kv, slot_map, n, k, k_stride, v, v_stride, q, q_stride, q_heads, q_out, q_out_stride, rope, norm, stream);
}

scute_status scute_kv_fork(scute_ctx *c, const scute_fork *f, void *stream) {
    if (!c) return SCUTE_ERR_ARG;
    if (!f) return fail(c, SCUTE_ERR_ARG, "null argument");
    if (f->n_in < 0 || f->n_in > SCUTE_MAX_REQUESTS || f->n_out < 0 || f->n_out > SCUTE_MAX_REQUESTS)
        return fail(c, SCUTE_ERR_ARG, "%d old rows, %d new ones: outside 0..%d", f->n_in, f->n_out, SCUTE_MAX_REQUESTS);
    if (f->n_pages < 0 || f->n_pages > (1 << 30) || f->n_free_max < 0 || f->n_free_max > 0x7fffffff)
        return fail(c, SCUTE_ERR_ARG, "n_pages or n_free_max out of range");
    if (f->page_size < 1 || f->table_cols < 1 || f->table_in_stride < f->table_cols || f->table_out_stride < f->table_cols)
        return fail(c, SCUTE_ERR_SHAPE, "pages of %d tokens, %d table columns, row pitches %lld and %lld", f->page_size,
                    f->table_cols, (long long)f->table_in_stride, (long long)f->table_out_stride);
    const int64_t rows = f->n_in > f->n_out ? f->n_in : f->n_out;
    if (rows * f->table_cols > 0x7fffffff || (int64_t)f->table_cols * f->page_size > 0x7fffffff)
        return fail(c, SCUTE_ERR_SHAPE, "block table beyond 2^31 - 1 entries, or a row beyond 2^31 - 1 tokens");
    if (!f->free_in || !f->free_out || (f->n_free_max > 0 && !f->free_pages) || (f->n_pages > 0 && !f->extra) ||
        (f->n_in > 0 && (!f->table_in || !f->len_in)) ||
        (f->n_out > 0 && (!f->source || !f->table_out || !f->len_out || !f->copy_from || !f->copy_to || !f->copy_tokens)))
        return fail(c, SCUTE_ERR_ARG, "null argument");
    // what is written may lie neither over what is read nor over anything else that is
    // written: the steps read their inputs until the last one
    const auto table = [&](int n, int64_t pitch) { return n > 0 ? (n - 1) * pitch + f->table_cols : 0; };
    const struct {
        const int32_t *p;
        int64_t n;
    } in[] = {{f->table_in, table(f->n_in, f->table_in_stride)}, {f->len_in, f->n_in}, {f->source, f->n_out},
              {f->len_new, f->len_new ? f->n_out : 0}, {f->free_in, 1}},
      out[] = {{f->table_out, table(f->n_out, f->table_out_stride)}, {f->len_out, f->n_out}, {f->copy_from, f->n_out},
               {f->copy_to, f->n_out}, {f->copy_tokens, f->n_out}, {f->extra, f->n_pages}, {f->free_pages, f->n_free_max},
               {f->free_out, 1}};
    const auto overlap = [](const auto &x, const auto &y) { return x.n > 0 && y.n > 0 && x.p < y.p + y.n && y.p < x.p + x.n; };
    for (const auto &y : out) {
        for (const auto &x : in)
            if (overlap(x, y) && !(x.p == f->free_in && y.p == f->free_out))
                return fail(c, SCUTE_ERR_ARG, "an output overlaps an input");
        for (const auto &x : out)
            if (&x != &y && overlap(x, y)) return fail(c, SCUTE_ERR_ARG, "two outputs overlap");
    }
    DeviceGuard dg(c->device);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    ForkArgs a{};
    a.table_in = f->table_in;
    a.len_in = f->len_in;
    a.in_stride = f->table_in_stride;
    a.source = f->source;
    a.len_new = f->len_new;
    a.table_out = f->table_out;
    a.len_out = f->len_out;
    a.out_stride = f->table_out_stride;
    a.n_in = f->n_in;
    a.n_out = f->n_out;
    a.cols = f->table_cols;
    a.page_size = f->page_size;
    a.page_shift = shift_of(f->page_size);
    a.n_pages = f->n_pages;
    a.extra = f->extra;
    a.free_pages = f->free_pages;
    a.n_free_max = f->n_free_max;
    a.free_in = f->free_in;
    a.free_out = f->free_out;
    a.copy_from = f->copy_from;
    a.copy_to = f->copy_to;
    a.copy_tokens = f->copy_tokens;
    a.ws = c->fork_ws;
    a.status = c->d_status;
    int launches = 0;
    TimedLaunch tl{c, st};
    CU_TRY(c, tl.begin());
    CU_TRY(c, launch_kv_fork(a, c->num_sms, &launches, st));
    count_launch(c, launches);
    CU_TRY(c, tl.end(SCUTE_KIND_KV_FORK));
    return SCUTE_OK;
}

scute_status scute_kv_copy(scute_ctx *c, const scute_kv_cache *caches, int n_caches, const int32_t *copy_from,
                           const int32_t *copy_to, const int32_t *tokens, int64_t n, void *stream) {
    if (!c) return SCUTE_ERR_ARG;
    if (!caches || n_caches < 1 || n_caches > SCUTE_MAX_CACHES)
        return fail(c, SCUTE_ERR_ARG, "n_caches = %d outside 1..%d", n_caches, SCUTE_MAX_CACHES);
    if (n < 0 || n > (1 << 20)) return fail(c, SCUTE_ERR_ARG, "n out of range");
    KvView one{}, next{};
    scute_status s = check_cache(c, &caches[0], &one);
    for (int i = 0; i < n_caches; ++i) {
        if (s) return s;
        s = check_cache(c, &caches[i], &next);
        if (!s && (next.dtype != one.dtype || next.n_pages != one.n_pages || next.page_size != one.page_size ||
                   next.heads != one.heads || next.dim != one.dim || next.page_stride != one.page_stride ||
                   next.token_stride != one.token_stride || next.head_stride != one.head_stride))
            return fail(c, SCUTE_ERR_SHAPE, "cache %d is not of the first one's type, size and strides", i);
    }
    if (s) return s;
    if ((int64_t)one.page_size * one.heads * (one.dim * kv_esz(one.dtype) / 16) > 0x7fffffff)
        return fail(c, SCUTE_ERR_UNSUPPORTED, "a page of %d tokens of %d heads is beyond 2^31 - 1 pieces of 16 bytes", one.page_size, one.heads);
    if (n == 0) return SCUTE_OK;
    if (!copy_from || !copy_to) return fail(c, SCUTE_ERR_ARG, "null argument");
    DeviceGuard dg(c->device);
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int esz = kv_esz(one.dtype);
    PageCopyArgs a{};
    a.heads = one.heads;
    a.page_size = one.page_size;
    a.n_pages = one.n_pages;
    a.n = (int)n;
    a.row_bytes = one.dim * esz;
    a.page_bytes = one.page_stride * esz;
    a.token_bytes = one.token_stride * esz;
    a.head_bytes = one.head_stride * esz;
    a.from = copy_from;
    a.to = copy_to;
    a.tokens = tokens;
    a.status = c->d_status;
    TimedLaunch tl{c, st};
    CU_TRY(c, tl.begin());
    for (int first = 0; first < n_caches; first += COPY_POOLS / 2) {
        a.pools = 0;
        for (int i = first; i < n_caches && i < first + COPY_POOLS / 2; ++i) {
            a.pool[a.pools++] = caches[i].k;
            a.pool[a.pools++] = caches[i].v;
        }
        CU_TRY(c, launch_kv_copy(a, c->num_sms, st));
        count_launch(c, 1);
    }
    CU_TRY(c, tl.end(SCUTE_KIND_KV_COPY));
    return SCUTE_OK;
}

scute_status scute_paged_attention(scute_ctx *c, const scute_kv_cache *kv, const scute_attention *t, void *stream) {
    if (!c) return SCUTE_ERR_ARG;
    return attend(c, kv, t, 0, nullptr, stream);
}

scute_status scute_paged_attention_sinks(scute_ctx *c, const scute_kv_cache *kv, const scute_attention *t, int32_t sinks,
                                         void *stream) {
    if (!c) return SCUTE_ERR_ARG;
    return attend(c, kv, t, sinks, nullptr, stream);
}

scute_status scute_paged_attention_shared(scute_ctx *c, const scute_kv_cache *kv, const scute_attention *t, const scute_shared *s,
                                          void *stream) {
    if (!c) return SCUTE_ERR_ARG;
    if (!s) return fail(c, SCUTE_ERR_ARG, "null argument");
    return attend(c, kv, t, 0, s, stream);
}

int64_t scute_shared_bytes(const scute_ctx *c, int n_req, int q_heads, int kv_heads, int head_dim) {
    if (!c || n_req < 0 || n_req > SCUTE_MAX_REQUESTS || kv_heads < 1 || q_heads < 1 || q_heads > (1 << 16) || q_heads % kv_heads ||
        head_dim < 16 || head_dim > SCUTE_MAX_HEAD_DIM || head_dim % 16)
        return -1;
    return shared_work(n_req, q_heads, kv_heads, head_dim, c->num_sms).bytes;
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
