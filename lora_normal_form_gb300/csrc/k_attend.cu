// Attention of one new token of each request over its paged cache.
#include <cuda_fp8.h>

#include "internal.h"

namespace scute {

namespace {

__device__ __forceinline__ float ld(const float *p) { return *p; }
__device__ __forceinline__ void st(float *p, float x) { *p = x; }

constexpr int AT_HEADS = 8, AT_TILE = 32;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// One CTA per request, key/value head and up to 8 of its query heads: tiles of
// 32 tokens with a running maximum and sum.  IO: type of q and out, KV: of the cache.
template <typename IO, typename KV>
__global__ void __launch_bounds__(128) attend_kernel(const AttendArgs a) {
    __shared__ float sq[AT_HEADS][ATT_MAX_DIM];
    __shared__ float sp[AT_HEADS][AT_TILE];
    __shared__ float s_alpha[AT_HEADS];
    __shared__ long long s_off[AT_TILE];
    const int r = blockIdx.x, hk = blockIdx.y, D = a.kv.dim, t = threadIdx.x;
    const int h0 = blockIdx.z * AT_HEADS, nh = min(AT_HEADS, a.group - h0);
    const long long cap = (long long)a.kv.table_cols * a.kv.page_size;
    int len = a.kv_len[r];
    if (len < 0 || len > cap) {
        if (t == 0) atomicOr(a.status, STATUS_PAGES);
        len = len < 0 ? 0 : (int)cap;
    }
    const int first = a.window > 0 ? max(0, len - a.window) : 0;
    const IO *q = reinterpret_cast<const IO *>(a.q) + r * a.q_stride + (long long)(hk * a.group + h0) * D;
    const float ks = a.kv.k_scale ? a.kv.k_scale[hk] : 1.f;
    for (int i = t; i < nh * D; i += 128) sq[i / D][i % D] = ld(q + i) * (ks * a.scale);
    const KV *k = reinterpret_cast<const KV *>(a.kv.k) + hk * a.kv.head_stride;
    const KV *v = reinterpret_cast<const KV *>(a.kv.v) + hk * a.kv.head_stride;
    const int lane = t & 31, warp = t >> 5;
    float acc[AT_HEADS][2] = {};
    float top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};    // heads warp and warp + 4
    for (int t0 = first; t0 < len; t0 += AT_TILE) {
        __syncthreads();
        if (t < AT_TILE) {
            long long off = -1;
            if (t0 + t < len) {
                const int page = a.kv.table[r * a.kv.table_stride + (t0 + t) / a.kv.page_size];
                if (page >= 0 && page < a.kv.n_pages)
                    off = page * a.kv.page_stride + ((t0 + t) % a.kv.page_size) * a.kv.token_stride;
                else
                    atomicOr(a.status, STATUS_PAGES);
            }
            s_off[t] = off;
        }
        __syncthreads();
        {
            const int tok = t >> 2, part = t & 3;
            const long long off = s_off[tok];
            float s[AT_HEADS] = {};
            if (off >= 0)
                for (int i = part; i < D; i += 4) {
                    const float x = ld(k + off + i);
                    for (int h = 0; h < nh; ++h) s[h] += x * sq[h][i];
                }
            for (int h = 0; h < nh; ++h) {
                float x = s[h];
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                if (a.softcap > 0.f) x = a.softcap * tanhf(x / a.softcap);
                if (part == 0) sp[h][tok] = off >= 0 ? x : -INFINITY;
            }
        }
        __syncthreads();
        for (int j = 0; j < 2; ++j) {
            const int h = warp + 4 * j;
            if (h >= nh) break;
            const float x = sp[h][lane];
            float m = x;
            for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            m = fmaxf(m, top[j]);
            const float ref = m == -INFINITY ? 0.f : m;
            const float p = expf(x - ref), alpha = expf(top[j] - ref);
            float all = p;
            for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
            sum[j] = sum[j] * alpha + all;
            top[j] = m;
            sp[h][lane] = p;
            if (lane == 0) s_alpha[h] = alpha;
        }
        __syncthreads();
        for (int h = 0; h < nh; ++h) {
            acc[h][0] *= s_alpha[h];
            acc[h][1] *= s_alpha[h];
        }
        for (int tok = 0; tok < AT_TILE; ++tok) {
            const long long off = s_off[tok];
            if (off < 0) continue;
            for (int e = 0; e < 2; ++e) {
                const int i = t + 128 * e;
                if (i >= D) break;
                const float x = ld(v + off + i);
                for (int h = 0; h < nh; ++h) acc[h][e] += sp[h][tok] * x;
            }
        }
    }
    __syncthreads();
    for (int j = 0; j < 2; ++j) {
        const int h = warp + 4 * j;
        if (h < nh && lane == 0) {
            s_alpha[h] = sum[j] > 0.f ? 1.f / sum[j] : 0.f;
            if (a.lse) a.lse[(long long)r * a.q_heads + hk * a.group + h0 + h] = top[j] + logf(sum[j]);
        }
    }
    __syncthreads();
    const float vs = a.kv.v_scale ? a.kv.v_scale[hk] : 1.f;
    IO *out = reinterpret_cast<IO *>(a.out) + r * a.out_stride + (long long)(hk * a.group + h0) * D;
    for (int h = 0; h < nh; ++h)
        for (int e = 0; e < 2; ++e)
            if (t + 128 * e < D) st(out + h * D + t + 128 * e, acc[h][e] * s_alpha[h] * vs);
}


// ---------------------------------------------------------------- 16- and 8-bit caches
// The products run on the warp-wide matrix instructions with the cache as the
// operand of 16 rows and the query heads as the one of 8 columns:
//     S^T [16 tokens x 8 heads] = K [16 x D] Q^T,
//     O^T [D x 8 heads] += V^T [D x 16 tokens] P^T,
// so a group of 4 or 8 query heads wastes little, and both operands come from
// the cache straight into registers: a product's inner index may be numbered in
// any way that both operands share, so lane (g, c) = (lane / 4, lane % 4) takes 16
// consecutive bytes of token g's (and g + 8's) key, the query's fragment the
// same elements; and 16 consecutive bytes of the values of tokens 2c, 2c + 1,
// 2c + 8, 2c + 9, of which pairs of tokens are interleaved by byte permutes.
// Nothing is staged in shared memory, and no warp waits for another inside a row.
//
// The work is one sequence of units (UT tokens of one request and head row),
// cut into equal contiguous ranges, one per CTA; the warps of a CTA take every
// fourth tile of a unit run and merge their maxima, sums and outputs in shared
// memory when the row ends.  A row that several CTAs share is joined by the
// last of them to arrive, in the order of the CTAs.
constexpr int AW = 4;              // warps of a CTA

__device__ __forceinline__ uint4 ldg16(const void *p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                 : "l"(p));
    return r;
}
__device__ __forceinline__ uint2 ldg8(const void *p) {
    uint2 r;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
}
template <bool F16>
__device__ __forceinline__ void mma16816(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                     "{%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// Two e4m3 values (the low 16 bits) as two halves.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t x) {
    uint32_t y;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t y;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t y;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}

// The batch's work list: units of UT tokens, rows (request, key/value head, head
// chunk) in this order; every row has a unit, an empty request's too.
struct Plan {
    int hz;                  // rows of a request
    int upt;                 // tokens of a unit
    long long total;         // units
    int ctas;                // CTAs that have any
};
__device__ __forceinline__ void seen_of(const AttendArgs &a, int r, int *first, int *len, bool *bad) {
    const int cap = a.kv.table_cols * a.kv.page_size;
    int n = a.kv_len[r];
    *bad = n < 0 || n > cap;
    n = n < 0 ? 0 : n > cap ? cap : n;
    *len = n;
    *first = a.window > 0 ? max(0, n - a.window) : 0;
}
__device__ __forceinline__ long long range_start(const Plan &p, int cta) { return p.total * cta / p.ctas; }
// The CTA whose range holds unit x.
__device__ __forceinline__ int owner_of(const Plan &p, long long x) {
    return (int)(((x + 1) * p.ctas - 1) / p.total);
}

// units_at[r] = units of the requests before r (one head row), for r <= n_req.
__device__ __forceinline__ void plan_units(const AttendArgs &a, int upt, int *units_at, int *warp_sum) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, n = a.n_req, threads = AW * 32;
    const int per = (n + threads - 1) / threads, r0 = min(n, t * per), r1 = min(n, r0 + per);
    int mine = 0;
    bool any = false;
    for (int r = r0; r < r1; ++r) {
        int first, len;
        bool bad;
        seen_of(a, r, &first, &len, &bad);
        any |= bad;
        mine += max(1, (len - first + upt - 1) / upt);
    }
    if (any && blockIdx.x == 0) atomicOr(a.status, STATUS_PAGES);
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    int at = inc - mine;
#pragma unroll
    for (int w = 0; w < AW; ++w) at += w < warp ? warp_sum[w] : 0;
    for (int r = r0; r < r1; ++r) {
        int first, len;
        bool bad;
        seen_of(a, r, &first, &len, &bad);
        units_at[r] = at;
        at += max(1, (len - first + upt - 1) / upt);
    }
    if (t == threads - 1) units_at[n] = at;
    __syncthreads();
}

// A CTA's share of a row: unnormalised output of every head and dimension, its
// maximum (in powers of two) and its sum.
struct PartView {
    float *m, *l, *o;
};
constexpr int PART_FLOATS = ATT_HEADS * (ATT_MAX_DIM + 2);
__device__ __forceinline__ PartView part_of(const AttendArgs &a, int slot) {
    float *p = a.part + (size_t)slot * PART_FLOATS;
    return {p, p + ATT_HEADS, p + 2 * ATT_HEADS};
}

template <bool FP8, int DC, int NT, int MINB>
__global__ void __launch_bounds__(AW * 32, MINB) attend_mma_kernel(const AttendArgs a) {
    // 16-token tiles of one pass: 4 KB of keys where two tiles (a lane finds one
    // token's place) can make that
    constexpr int MT = DC * (FP8 ? 1 : 2) <= 128 ? 2 : 1;
    constexpr int TT = 16 * MT, UT = AW * TT;
    constexpr int KE = FP8 ? 16 : 8;                 // elements of 16 bytes
    constexpr int KP = DC / (4 * KE);                // key pieces of a lane, each four lanes wide
    constexpr int VE = FP8 && DC > 64 ? 16 : 8;      // elements of a value piece, eight lanes wide
    constexpr int VP = DC / (8 * VE);
    constexpr int VW = FP8 ? VE / 4 : VE / 2;        // its words
    constexpr int OT = VE / 2;                       // 16-row output tiles of a value piece
    constexpr int HC = 8 * NT, ESZ = FP8 ? 1 : 2;
    constexpr int SO_LD = DC + 4;                    // floats between heads in shared memory

    extern __shared__ int units_at[];
    __shared__ int s_warp[AW];
    __shared__ int s_last;
    __shared__ float s_m[AW][HC], s_l[AW][HC], s_top[HC], s_sum[HC];
    __shared__ __align__(16) float s_o[HC][SO_LD];

    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, g = lane >> 2, c = lane & 3;
    const int D = a.kv.dim, Z = (a.group + HC - 1) / HC;
    plan_units(a, UT, units_at, s_warp);
    Plan plan;
    plan.hz = a.kv.heads * Z;
    plan.upt = UT;
    plan.total = (long long)units_at[a.n_req] * plan.hz;
    plan.ctas = (int)min((long long)gridDim.x, plan.total);
    const int cta = blockIdx.x;
    if (cta >= plan.ctas) return;
    long long at = range_start(plan, cta);
    const long long end = range_start(plan, cta + 1);

    // the request of the first unit
    int r = 0;
    {
        int hi = a.n_req - 1;
        while (r < hi) {
            const int mid = (r + hi + 1) >> 1;
            if ((long long)units_at[mid] * plan.hz <= at) r = mid;
            else hi = mid - 1;
        }
    }
    while (at < end) {
        while ((long long)units_at[r + 1] * plan.hz <= at) ++r;
        const int ur = units_at[r + 1] - units_at[r];
        const long long in_req = at - (long long)units_at[r] * plan.hz;
        const int row = (int)(in_req / ur), u0 = (int)(in_req - (long long)row * ur);
        const int u1 = (int)min((long long)ur, u0 + (end - at));
        const int hk = row / Z, z = row - hk * Z;
        const int h0 = hk * a.group + z * HC, nh = min(HC, a.group - z * HC);
        int first, len;
        bool bad;
        seen_of(a, r, &first, &len, &bad);

        // queries: the fragments' elements are those of the keys' pieces
        uint32_t qf[NT][KP][KE / 2];
        float mul[NT][2];         // score to power-of-two exponent (without a cap), per head of this lane's columns
        const float ks = a.kv.k_scale ? a.kv.k_scale[hk] : 1.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int h = nt * 8 + g;
            const __nv_bfloat16 *q =
                reinterpret_cast<const __nv_bfloat16 *>(a.q) + r * a.q_stride + (long long)(h0 + h) * D;
#pragma unroll
            for (int p = 0; p < KP; ++p)
#pragma unroll
                for (int e = 0; e < KE / 8; ++e) {
                    const int d = (p * 4 + c) * KE + e * 8;
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (h < nh && d < D) x = *reinterpret_cast<const uint4 *>(q + d);
                    qf[nt][p][e * 4 + 0] = x.x;
                    qf[nt][p][e * 4 + 1] = x.y;
                    qf[nt][p][e * 4 + 2] = x.z;
                    qf[nt][p][e * 4 + 3] = x.w;
                }
            float back = 1.f;
            if constexpr (FP8) {
                // 16-bit halves have 11 bits where bf16 has 8: scaled by a power of
                // two that takes the head's largest element to 2^8 or below, every
                // element down to 2^-22 of it stays exact
                float big = 0.f;
#pragma unroll
                for (int p = 0; p < KP; ++p)
#pragma unroll
                    for (int e = 0; e < KE / 2; ++e) {
                        const uint32_t w = qf[nt][p][e];
                        big = fmaxf(big, fmaxf(fabsf(__uint_as_float(w << 16)), fabsf(__uint_as_float(w & 0xffff0000u))));
                    }
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                int ex = 0;
                if (big > 0.f && big < INFINITY) frexpf(big, &ex);
                ex = max(-100, min(100, ex - 8));
                const float down = ldexpf(1.f, -ex);
                back = ldexpf(1.f, ex);
#pragma unroll
                for (int p = 0; p < KP; ++p)
#pragma unroll
                    for (int e = 0; e < KE / 2; ++e) {
                        const uint32_t w = qf[nt][p][e];
                        qf[nt][p][e] = pack_f16(__uint_as_float(w << 16) * down, __uint_as_float(w & 0xffff0000u) * down);
                    }
            }
            mul[nt][0] = __shfl_sync(0xffffffffu, back, (2 * c) * 4) * ks * a.scale;
            mul[nt][1] = __shfl_sync(0xffffffffu, back, (2 * c + 1) * 4) * ks * a.scale;
        }

        float o[NT][VP][OT][4] = {};
        float top[NT][2], sum[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) top[nt][0] = top[nt][1] = -INFINITY, sum[nt][0] = sum[nt][1] = 0.f;

        const char *kb = reinterpret_cast<const char *>(a.kv.k) + hk * a.kv.head_stride * ESZ;
        const char *vb = reinterpret_cast<const char *>(a.kv.v) + hk * a.kv.head_stride * ESZ;
        const int stop = min(len, first + u1 * UT);
        const int32_t *table = a.kv.table + r * a.kv.table_stride;

        // lane i finds token i of a pass: its page, one pass ahead of its place
        auto page_at = [&](int tok) -> int {
            const int i = tok + (lane & (TT - 1));
            return i < stop ? table[i / a.kv.page_size] : -1;
        };
        auto place_of = [&](int tok, int page) -> long long {
            const int i = tok + (lane & (TT - 1));
            if (i >= stop) return -1;
            if (page < 0 || page >= a.kv.n_pages) {
                atomicOr(a.status, STATUS_PAGES);
                return -1;
            }
            return ((long long)page * a.kv.page_stride + (long long)(i % a.kv.page_size) * a.kv.token_stride) * ESZ;
        };
        uint4 kr[MT][2][KP];
        uint32_t vr[MT][4][VP][VW];
        auto load_k = [&](long long place) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const long long p = __shfl_sync(0xffffffffu, place, m * 16 + i * 8 + g);
#pragma unroll
                    for (int j = 0; j < KP; ++j) {
                        const int d = (j * 4 + c) * KE;
                        kr[m][i][j] = make_uint4(0, 0, 0, 0);
                        if (p >= 0 && (DC == 16 * KP || d < D)) kr[m][i][j] = ldg16(kb + p + d * ESZ);
                    }
                }
        };
        auto load_v = [&](long long place) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const long long p = __shfl_sync(0xffffffffu, place, m * 16 + 2 * c + (i & 1) + (i >> 1) * 8);
#pragma unroll
                    for (int j = 0; j < VP; ++j) {
                        const int d = (j * 8 + g) * VE;
                        const bool in = p >= 0 && d < D;
                        if constexpr (VW == 4) {
                            uint4 x = make_uint4(0, 0, 0, 0);
                            if (in) x = ldg16(vb + p + d * ESZ);
                            vr[m][i][j][0] = x.x, vr[m][i][j][1] = x.y, vr[m][i][j][2] = x.z, vr[m][i][j][3] = x.w;
                        } else {
                            uint2 x = make_uint2(0, 0);
                            if (in) x = ldg8(vb + p + d * ESZ);
                            vr[m][i][j][0] = x.x, vr[m][i][j][1] = x.y;
                        }
                    }
                }
        };

        int tok = first + u0 * UT + warp * TT;
        if (tok < stop) {
            long long place = place_of(tok, page_at(tok));
            int page_next = page_at(tok + UT);
            load_k(place);
            load_v(place);
            for (;;) {
                const unsigned ok = __ballot_sync(0xffffffffu, place >= 0);
                const int next = tok + UT;
                const bool more = next < stop;
                const long long place_next = more ? place_of(next, page_next) : -1;
                if (more) page_next = page_at(next + UT);

                float s[MT][NT][4] = {};
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int j = 0; j < KP; ++j) {
                        const uint32_t w0[4] = {kr[m][0][j].x, kr[m][0][j].y, kr[m][0][j].z, kr[m][0][j].w};
                        const uint32_t w1[4] = {kr[m][1][j].x, kr[m][1][j].y, kr[m][1][j].z, kr[m][1][j].w};
                        if constexpr (FP8) {
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const uint32_t a0 = e4m3x2_f16x2(w0[e]), a2 = e4m3x2_f16x2(w0[e] >> 16);
                                const uint32_t a1 = e4m3x2_f16x2(w1[e]), a3 = e4m3x2_f16x2(w1[e] >> 16);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma16816<true>(s[m][nt], a0, a1, a2, a3, qf[nt][j][2 * e], qf[nt][j][2 * e + 1]);
                            }
                        } else {
#pragma unroll
                            for (int e = 0; e < 2; ++e)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
                                    mma16816<false>(s[m][nt], w0[2 * e], w1[2 * e], w0[2 * e + 1], w1[2 * e + 1],
                                                    qf[nt][j][2 * e], qf[nt][j][2 * e + 1]);
                        }
                    }
                if (more) load_k(place_next);

                // running maximum and sum, in powers of two
                uint32_t pf[MT][NT][2][2];            // [tokens 0-7, 8-15][weights, what their rounding left]
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            float x = s[m][nt][i] * mul[nt][i & 1];
                            if (a.softcap > 0.f) x = a.softcap * tanhf(x / a.softcap);
                            x *= LOG2E;
                            if (!(ok >> (m * 16 + (i >> 1) * 8 + g) & 1)) x = -INFINITY;
                            s[m][nt][i] = x;
                            mx[i & 1] = fmaxf(mx[i & 1], x);
                        }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float x = mx[i];
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                        mx[i] = fmaxf(x, top[nt][i]);
                    }
                    if (__any_sync(0xffffffffu, mx[0] != top[nt][0] || mx[1] != top[nt][1])) {
                        float al[2];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            al[i] = mx[i] == top[nt][i] ? 1.f : exp2f(top[nt][i] - mx[i]);
                            top[nt][i] = mx[i];
                            sum[nt][i] *= al[i];
                        }
#pragma unroll
                        for (int j = 0; j < VP; ++j)
#pragma unroll
                            for (int i = 0; i < OT; ++i) {
                                o[nt][j][i][0] *= al[0];
                                o[nt][j][i][1] *= al[1];
                                o[nt][j][i][2] *= al[0];
                                o[nt][j][i][3] *= al[1];
                            }
                    }
                    const float ref[2] = {top[nt][0] == -INFINITY ? 0.f : top[nt][0],
                                          top[nt][1] == -INFINITY ? 0.f : top[nt][1]};
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        float p[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            p[i] = exp2f(s[m][nt][i] - ref[i & 1]);
                            sum[nt][i & 1] += p[i];
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            if constexpr (FP8) {
                                pf[m][nt][i][0] = transpose8(pack_f16(p[2 * i], p[2 * i + 1]));
                            } else {
                                // bf16 keeps 8 bits of a weight: a second product takes the rest
                                const uint32_t hi = pack_bf16(p[2 * i], p[2 * i + 1]);
                                const float r0 = p[2 * i] - __uint_as_float(hi << 16);
                                const float r1 = p[2 * i + 1] - __uint_as_float(hi & 0xffff0000u);
                                pf[m][nt][i][0] = transpose8(hi);
                                pf[m][nt][i][1] = transpose8(pack_bf16(r0, r1));
                            }
                        }
                    }
                }

#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int j = 0; j < VP; ++j)
#pragma unroll
                        for (int w = 0; w < VW; ++w) {
                            const uint32_t x0 = vr[m][0][j][w], x1 = vr[m][1][j][w];
                            const uint32_t x2 = vr[m][2][j][w], x3 = vr[m][3][j][w];
                            if constexpr (FP8) {
                                const uint32_t y0 = __byte_perm(x0, x1, 0x5140), y1 = __byte_perm(x0, x1, 0x7362);
                                const uint32_t y2 = __byte_perm(x2, x3, 0x5140), y3 = __byte_perm(x2, x3, 0x7362);
#pragma unroll
                                for (int i = 0; i < 2; ++i) {
                                    const uint32_t ya = i ? y1 : y0, yb = i ? y3 : y2;
                                    const uint32_t a0 = e4m3x2_f16x2(ya), a1 = e4m3x2_f16x2(ya >> 16);
                                    const uint32_t a2 = e4m3x2_f16x2(yb), a3 = e4m3x2_f16x2(yb >> 16);
#pragma unroll
                                    for (int nt = 0; nt < NT; ++nt)
                                        mma16816<true>(o[nt][j][2 * w + i], a0, a1, a2, a3, pf[m][nt][0][0],
                                                       pf[m][nt][1][0]);
                                }
                            } else {
                                const uint32_t a0 = __byte_perm(x0, x1, 0x5410), a1 = __byte_perm(x0, x1, 0x7632);
                                const uint32_t a2 = __byte_perm(x2, x3, 0x5410), a3 = __byte_perm(x2, x3, 0x7632);
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    mma16816<false>(o[nt][j][w], a0, a1, a2, a3, pf[m][nt][0][0], pf[m][nt][1][0]);
                                    mma16816<false>(o[nt][j][w], a0, a1, a2, a3, pf[m][nt][0][1], pf[m][nt][1][1]);
                                }
                            }
                        }
                if (!more) break;
                load_v(place_next);
                place = place_next;
                tok = next;
            }
        }

        // the warps' shares of the row
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float x = sum[nt][i];
                x += __shfl_xor_sync(0xffffffffu, x, 4);
                x += __shfl_xor_sync(0xffffffffu, x, 8);
                x += __shfl_xor_sync(0xffffffffu, x, 16);
                sum[nt][i] = x;
                if (g == 0) {
                    s_m[warp][nt * 8 + 2 * c + i] = top[nt][i];
                    s_l[warp][nt * 8 + 2 * c + i] = x;
                }
            }
        __syncthreads();
        if (t < HC) {
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int w = 0; w < AW; ++w) m = fmaxf(m, s_m[w][t]);
            if (m > -INFINITY)
#pragma unroll
                for (int w = 0; w < AW; ++w) l += s_l[w][t] * exp2f(s_m[w][t] - m);
            s_top[t] = m;
            s_sum[t] = l;
        }
        __syncthreads();
#pragma unroll 1
        for (int w = 0; w < AW; ++w) {
            if (warp == w) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int ha = nt * 8 + 2 * c;
                    const float m0 = s_top[ha], m1 = s_top[ha + 1];
                    const float f0 = m0 > -INFINITY ? exp2f(top[nt][0] - m0) : 0.f;
                    const float f1 = m1 > -INFINITY ? exp2f(top[nt][1] - m1) : 0.f;
#pragma unroll
                    for (int j = 0; j < VP; ++j)
#pragma unroll
                        for (int i = 0; i < OT; ++i) {
                            const int d = (j * 8 + g) * VE + 2 * i;
                            float2 *p0 = reinterpret_cast<float2 *>(&s_o[ha][d]);
                            float2 *p1 = reinterpret_cast<float2 *>(&s_o[ha + 1][d]);
                            float2 x = make_float2(o[nt][j][i][0] * f0, o[nt][j][i][2] * f0);
                            float2 y = make_float2(o[nt][j][i][1] * f1, o[nt][j][i][3] * f1);
                            if (w) {
                                x.x += p0->x, x.y += p0->y;
                                y.x += p1->x, y.y += p1->y;
                            }
                            *p0 = x;
                            *p1 = y;
                        }
                }
            }
            __syncthreads();
        }

        const float vs = a.kv.v_scale ? a.kv.v_scale[hk] : 1.f;
        __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(a.out) + r * a.out_stride + (long long)h0 * D;
        float *lse = a.lse ? a.lse + (long long)r * a.q_heads + h0 : nullptr;
        if (u0 == 0 && u1 == ur) {
            for (int i = t; i < nh * (D / 2); i += AW * 32) {
                const int h = i / (D / 2), d = 2 * (i - h * (D / 2));
                const float f = s_sum[h] > 0.f ? vs / s_sum[h] : 0.f;
                *reinterpret_cast<uint32_t *>(out + h * D + d) = pack_bf16(s_o[h][d] * f, s_o[h][d + 1] * f);
            }
            if (lse && t < nh) lse[t] = (s_top[t] + log2f(s_sum[t])) * LN2;
        } else {
            const long long row0 = at - u0;
            const int c0 = owner_of(plan, row0), c1 = owner_of(plan, row0 + ur - 1);
            const PartView p = part_of(a, 2 * cta + (u0 == 0 ? 1 : 0));
            for (int i = t; i < nh * (D / 4); i += AW * 32) {
                const int h = i / (D / 4), d = 4 * (i - h * (D / 4));
                *reinterpret_cast<float4 *>(p.o + h * D + d) = *reinterpret_cast<float4 *>(&s_o[h][d]);
            }
            if (t < nh) p.m[t] = s_top[t], p.l[t] = s_sum[t];
            __threadfence();
            __syncthreads();
            if (t == 0) {
                s_last = atomicAdd(a.ctr + c0, 1) == c1 - c0;
                if (s_last) a.ctr[c0] = 0;
            }
            __syncthreads();
            if (s_last) {
                __threadfence();
                const int parts = c1 - c0 + 1;
                auto slot = [&](int i) { return i == 0 ? 2 * c0 + 1 : 2 * (c0 + i); };
                for (int h = warp; h < nh; h += AW) {
                    float m = -INFINITY;
                    for (int i = lane; i < parts; i += 32) m = fmaxf(m, __ldcg(part_of(a, slot(i)).m + h));
#pragma unroll
                    for (int x = 16; x; x >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
                    float l = 0.f;
                    if (m > -INFINITY)
                        for (int i = lane; i < parts; i += 32) {
                            const PartView q = part_of(a, slot(i));
                            l += __ldcg(q.l + h) * exp2f(__ldcg(q.m + h) - m);
                        }
#pragma unroll
                    for (int x = 16; x; x >>= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
                    if (lane == 0) s_top[h] = m, s_sum[h] = l;
                }
                __syncthreads();
                for (int i = t; i < nh * (D / 4); i += AW * 32) {
                    const int h = i / (D / 4), d = 4 * (i - h * (D / 4));
                    const float m = s_top[h];
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (m > -INFINITY)
#pragma unroll 4
                        for (int k = 0; k < parts; ++k) {
                            const PartView q = part_of(a, slot(k));
                            const float w = exp2f(__ldcg(q.m + h) - m);
                            const float4 y = __ldcg(reinterpret_cast<const float4 *>(q.o + h * D + d));
                            x.x += w * y.x, x.y += w * y.y, x.z += w * y.z, x.w += w * y.w;
                        }
                    const float f = s_sum[h] > 0.f ? vs / s_sum[h] : 0.f;
                    uint2 y;
                    y.x = pack_bf16(x.x * f, x.y * f);
                    y.y = pack_bf16(x.z * f, x.w * f);
                    *reinterpret_cast<uint2 *>(out + h * D + d) = y;
                }
                if (lse && t < nh) lse[t] = (s_top[t] + log2f(s_sum[t])) * LN2;
            }
        }
        __syncthreads();
        at += u1 - u0;
    }
}

// CTAs of a launch: every SM's, as many as reside (a CTA never waits for
// another, so more would only be slower).
template <bool FP8, int DC, int NT, int MINB>
cudaError_t launch_mma(const AttendArgs &a, int num_sms, cudaStream_t st) {
    static std::atomic<unsigned long long> done{0};
    const size_t smem = sizeof(int) * ((size_t)a.n_req + 1);
    if (smem > 16 * 1024) {
        const cudaError_t e = allow_max_dynamic_smem(attend_mma_kernel<FP8, DC, NT, MINB>, done);
        if (e != cudaSuccess) return e;
    }
    attend_mma_kernel<FP8, DC, NT, MINB><<<num_sms * MINB, AW * 32, smem, st>>>(a);
    return cudaGetLastError();
}

template <bool FP8>
cudaError_t launch_by_dim(const AttendArgs &a, int num_sms, cudaStream_t st) {
    const int D = a.kv.dim;
    if (D > 128) return launch_mma<FP8, 256, 1, 2>(a, num_sms, st);
    if (D > 64) return a.group > 8 ? launch_mma<FP8, 128, 2, 2>(a, num_sms, st) : launch_mma<FP8, 128, 1, 3>(a, num_sms, st);
    return a.group > 8 ? launch_mma<FP8, 64, 2, 3>(a, num_sms, st) : launch_mma<FP8, 64, 1, 3>(a, num_sms, st);
}

}  // namespace

constexpr int ATT_CTAS = 4;      // CTAs of an SM, at most
size_t attend_part_floats(int num_sms) { return (size_t)num_sms * ATT_CTAS * 2 * PART_FLOATS; }
int attend_ctrs(int num_sms) { return num_sms * ATT_CTAS; }

cudaError_t launch_attend(const AttendArgs &a, int num_sms, cudaStream_t st) {
    if (a.kv.dtype == KV_BF16) return launch_by_dim<false>(a, num_sms, st);
    if (a.kv.dtype == KV_E4M3) return launch_by_dim<true>(a, num_sms, st);
    const dim3 grid(a.n_req, a.kv.heads, (a.group + AT_HEADS - 1) / AT_HEADS);
    attend_kernel<float, float><<<grid, 128, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace scute
