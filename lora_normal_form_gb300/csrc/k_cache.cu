// The paged cache's bookkeeping and writes: pages and slots from request
// lengths (kv_resize), rotary positions and the cache write (kv_append), and
// the rotary table.
#include <climits>

#include <cuda_fp8.h>

#include "internal.h"
#include "ptx.cuh"

namespace scute {

namespace {

// ---------------------------------------------------------------- kv_resize
// Request r has o = len_in tokens in have = ceil(o / page) pages and wants w =
// len_new in want = ceil(w / page).  With drop = max(have - want, 0), need =
// max(want - have, 0) and their exclusive prefix sums over the requests,
//   freed page j (0 <= j < P = sum drop) belongs to the last r whose drop_at <= j;
//   the list then holds L = F + P pages, and the k-th page taken is its entry
//   L - 1 - k: a freed page again, or one of the F there were.
// A request is refused when need > 0 and need_at + need > L, or when its new
// tokens' inclusive prefix (over requests not refused so far) passes max_new.
// Both prefixes only grow, so the requests that do take pages are the first
// ones that need any, and their k run from 0 without a gap.  Nothing that is
// read is written: rows of shrinking requests are only read, the rows of
// growing ones written behind their old pages, and list entries are written
// only from F on.  So no thread waits for another, except that lengths and a
// count that are written in place follow a launch-wide arrival count.
//
// Bound by latency: lengths, two scans, a binary search for every row in shared
// memory, the page, the stores.  64 requests of one new token take 3.6 us (a launch
// of nothing 1.5), 4096 with their prompts 10.6 to 11.8 by the draw (all in one CTA
// 126).  Every CTA scans all requests for itself, which costs less than a second
// launch would; 256 threads are enough up to 256 requests (3.5 us against 4.4 with
// 1024).  Pages that come back are handed on one to a thread, each with a search and
// a dependent load, by as many CTAs as the new rows want: 256 requests of 4096 tokens
// that end in a step of few rows take 143 us in pages of 16, 2.2 ms in pages of one
// (1.2 us of bytes).
constexpr int RS_THREADS = 1024;       // at most

// Pages of so many tokens (at most 2^31 - 1 with a page's rounding); page of a position.
__device__ __forceinline__ int page_index(const ResizeArgs &a, int pos) {
    return a.page_shift >= 0 ? pos >> a.page_shift : pos / a.page_size;
}
__device__ __forceinline__ int pages_of(const ResizeArgs &a, int tokens) {
    return tokens == 0 ? 0 : page_index(a, tokens - 1) + 1;
}

// Last i in [0, n] with at[i] <= x, for at[0] = 0 <= x and at rising.
__device__ __forceinline__ int last_at_most(const int *at, int n, int x) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (at[mid] <= x) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// Exclusive prefix sum over the CTA's threads; *total receives the sum.
__device__ __forceinline__ unsigned long long cta_exclusive(unsigned long long x, unsigned long long *warp_sum,
                                                            unsigned long long *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    unsigned long long inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        const unsigned long long own = lane < (int)blockDim.x / 32 ? warp_sum[lane] : 0;
        unsigned long long sum = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long y = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += y;
        }
        warp_sum[lane] = sum - own;
        if (lane == 31) warp_sum[32] = sum;
    }
    __syncthreads();
    *total = warp_sum[32];
    const unsigned long long before = warp_sum[warp] + inc - x;
    __syncthreads();
    return before;
}

struct Span {
    int o, w;      // old and wanted length, inside the row
    bool bad;
};
__device__ __forceinline__ Span span_of(const ResizeArgs &a, int o, int w) {
    const int cap = a.cols * a.page_size;
    Span s;
    s.bad = o < 0 || o > cap || w < 0 || w > cap;
    s.o = o < 0 ? 0 : o > cap ? cap : o;
    s.w = w < 0 || w > cap ? s.o : w;
    return s;
}
__device__ __forceinline__ Span span_of(const ResizeArgs &a, int r) { return span_of(a, a.len_in[r], a.len_new[r]); }
// Entries between the kernel's lists, in shared memory (16-byte aligned).
__host__ __device__ inline int list_pitch(int n) { return (n + 4) & ~3; }

// A thread's entries of a list.
template <int ITEMS>
__device__ __forceinline__ void put_list(int *list, int r0, int n, const int (&x)[ITEMS]) {
    if (ITEMS % 4 == 0 && r0 + ITEMS <= n) {
#pragma unroll
        for (int i = 0; i + 3 < ITEMS; i += 4) *reinterpret_cast<int4 *>(list + r0 + i) = make_int4(x[i], x[i + 1], x[i + 2], x[i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i)
            if (r0 + i < n) list[r0 + i] = x[i];
    }
}

// ITEMS consecutive requests of a thread, held in registers.
template <int ITEMS>
__global__ void __launch_bounds__(RS_THREADS) kv_resize_kernel(const ResizeArgs a) {
    extern __shared__ __align__(16) int sm[];
    __shared__ unsigned long long warp_sum[33];
    __shared__ int s_taken, s_rows, s_flag, s_last;
    const int n = a.n_req, t = threadIdx.x;
    const int pitch = list_pitch(n);
    int *drop_at = sm, *need_at = sm + pitch, *cu = sm + 2 * pitch;
    // lengths, where the batch leaves room for them
    constexpr bool KEEP = ITEMS <= 4;
    int *old_of = sm + 3 * pitch, *new_of = sm + 4 * pitch;
    if (t == 0) s_taken = s_rows = s_flag = 0;
    const int r0 = t * ITEMS;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    int F = *a.free_in;
    Span sp[ITEMS];
    if (ITEMS == 4 && r0 + 3 < n && ((reinterpret_cast<uintptr_t>(a.len_in) | reinterpret_cast<uintptr_t>(a.len_new)) & 15) == 0) {
        const int4 o = *reinterpret_cast<const int4 *>(a.len_in + r0), w = *reinterpret_cast<const int4 *>(a.len_new + r0);
        const int ov[4] = {o.x, o.y, o.z, o.w}, wv[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) sp[i] = span_of(a, ov[i & 3], wv[i & 3]);
    } else {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            sp[i] = {0, 0, false};
            if (r0 + i < n) sp[i] = span_of(a, r0 + i);
        }
    }
    bool bad = false;
    if (F < 0 || F > a.n_free_max) {
        bad = true;
        F = F < 0 ? 0 : (int)a.n_free_max;
    }

    // pages given up and needed: one scan of both sums (each below 2^31)
    int need[ITEMS], drop[ITEMS];
    unsigned long long mine = 0;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        bad |= sp[i].bad;
        const int have = pages_of(a, sp[i].o), want = pages_of(a, sp[i].w);
        need[i] = max(want - have, 0);
        drop[i] = max(have - want, 0);
        mine += (unsigned long long)(unsigned)drop[i] << 32 | (unsigned)need[i];
    }
    unsigned long long total;
    unsigned long long run = cta_exclusive(mine, warp_sum, &total);
    const int P = (int)(total >> 32);
    const long long L = (long long)F + P;

    // new tokens of the requests that get their pages
    unsigned long long rows = 0;
    int drops[ITEMS], needs[ITEMS], olds[ITEMS], news[ITEMS];
    int first_need = (int)(run & 0xffffffffu), at_need = first_need, at_drop = (int)(run >> 32);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        drops[i] = at_drop, needs[i] = at_need, olds[i] = sp[i].o, news[i] = sp[i].w;
        if (sp[i].w > sp[i].o && (need[i] == 0 || at_need + (long long)need[i] <= L)) rows += sp[i].w - sp[i].o;
        at_drop += drop[i];
        at_need += need[i];
    }
    put_list(drop_at, r0, n, drops);
    put_list(need_at, r0, n, needs);
    if (KEEP) put_list(old_of, r0, n, olds), put_list(new_of, r0, n, news);
    if (t == 0) {
        drop_at[n] = P;
        need_at[n] = (int)(total & 0xffffffffu);
    }
    unsigned long long all_rows;
    unsigned long long at = cta_exclusive(rows, warp_sum, &all_rows);
    int taken = 0, served = 0, mine_at[ITEMS];
    at_need = first_need;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        mine_at[i] = (int)min(at, (unsigned long long)a.max_new + 1);
        if (sp[i].w > sp[i].o) {
            const bool paged = need[i] == 0 || at_need + (long long)need[i] <= L;
            if (paged) at += sp[i].w - sp[i].o;
            if (paged && at <= (unsigned long long)a.max_new) {
                served = (int)at;
                if (need[i]) taken = at_need + need[i];
            } else {
                bad = true;
            }
        }
        at_need += need[i];
    }
    taken = __reduce_max_sync(0xffffffffu, taken);
    served = __reduce_max_sync(0xffffffffu, served);
    if ((t & 31) == 0) {
        atomicMax(&s_taken, taken);
        atomicMax(&s_rows, served);
    }
    if (bad) s_flag = 1;
    __syncthreads();
    const int A = s_taken, T = s_rows;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) mine_at[i] = min(mine_at[i], T);
    put_list(cu, r0, n, mine_at);
    if (t == 0) cu[n] = T;
    __syncthreads();
    const long long left = L - A;

    auto old_len = [&](int r) { return KEEP ? old_of[r] : span_of(a, r).o; };
    auto new_len = [&](int r) { return KEEP ? new_of[r] : span_of(a, r).w; };
    // the k-th page taken from the top of the list
    auto taken_page = [&](int k) -> int {
        const long long at_list = L - 1 - k;
        if (at_list < F) return a.free_pages[at_list];
        const int j = (int)(at_list - F), r = last_at_most(drop_at, n, j);
        const int want = pages_of(a, new_len(r));
        return a.table[(long long)r * a.table_stride + want + (j - drop_at[r])];
    };
    const int step = gridDim.x * blockDim.x, g0 = blockIdx.x * blockDim.x + t;
    for (int k = g0; k < A; k += step) {
        const int r = last_at_most(need_at, n, k);
        const int have = pages_of(a, old_len(r));
        a.table[(long long)r * a.table_stride + have + (k - need_at[r])] = taken_page(k);
    }
    for (long long j = g0; F + j < left; j += step) {
        if (F + j >= a.n_free_max) {
            s_flag = 1;
            break;
        }
        const int r = last_at_most(drop_at, n, (int)j);
        const int want = pages_of(a, new_len(r));
        a.free_pages[F + j] = a.table[(long long)r * a.table_stride + want + ((int)j - drop_at[r])];
    }
    bool unslotted = false;
    for (long long i = g0; i < a.max_new; i += step) {
        int slot = -1, pos = 0, r = -1;
        if (i < T) {
            r = last_at_most(cu, n, (int)i);
            const int o = old_len(r);
            pos = o + ((int)i - cu[r]);
            const int pg = page_index(a, pos), have = pages_of(a, o);
            const int page = pg < have ? a.table[(long long)r * a.table_stride + pg] : taken_page(need_at[r] + (pg - have));
            // page numbers are not checked before: one that forms no slot must become
            // neither the mark of a padding row nor, cut to 32 bits, another's slot
            const long long at_slot = (long long)page * a.page_size + (pos - pg * a.page_size);
            const bool none = (unsigned long long)at_slot > INT_MAX;      // a negative page's too
            unslotted |= none;
            slot = none ? INT_MIN : (int)at_slot;
        }
        a.slot_map[i] = slot;
        a.positions[i] = pos;
        a.token_req[i] = r;
    }
    if (unslotted) s_flag = 1;
    for (int r = g0; r <= n; r += step) a.cu_new[r] = cu[r];

    // lengths and the count: where they are written in place, by the last CTA to
    // have read them
    const bool arrive = a.in_place && gridDim.x > 1;
    if (arrive) __threadfence();
    __syncthreads();
    if (t == 0) {
        s_last = arrive ? atomicAdd(a.ctr, 1) == (int)gridDim.x - 1 : blockIdx.x == 0;
        if (s_flag) atomicOr(a.status, STATUS_PAGES);
    }
    __syncthreads();
    if (!s_last) return;
    if (arrive) __threadfence();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int r = r0 + i;
        if (r < n) a.len_out[r] = sp[i].w > sp[i].o ? sp[i].o + (cu[r + 1] - cu[r]) : sp[i].w;
    }
    if (t == 0) {
        *a.free_out = (int)min(left, a.n_free_max);
        if (arrive) *a.ctr = 0;
    }
}

template <int ITEMS>
cudaError_t launch_resize(const ResizeArgs &a, int grid, int threads, cudaStream_t st) {
    static std::atomic<unsigned long long> done{0};
    const size_t smem = sizeof(int) * (ITEMS <= 4 ? 5 : 3) * (size_t)list_pitch(a.n_req);
    if (smem > 40 * 1024) {
        const cudaError_t e = allow_max_dynamic_smem(kv_resize_kernel<ITEMS>, done);
        if (e != cudaSuccess) return e;
    }
    return launch_chained(kv_resize_kernel<ITEMS>, grid, threads, smem, st, a);
}

// ---------------------------------------------------------------- kv_append
template <typename T> __device__ __forceinline__ float to_f(T x) { return (float)x; }
template <typename T> __device__ __forceinline__ T from_f(float x) { return (T)x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Any strides and rotary halves: one thread turns one pair, or passes one element,
// of one head of one row.  What it costs: 8772 rows of 48 heads of 128 take 137 us,
// 16 bytes at a time 38.
template <typename T>
__global__ void __launch_bounds__(256) kv_append_kernel(const AppendArgs a) {
    const int row = blockIdx.x, dim = a.kv.dim, half = a.rot / 2;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int slot = a.slot_map[row];
    const bool in = slot >= 0 && slot < (long long)a.kv.n_pages * a.kv.page_size;
    if (slot < -1 || (slot >= 0 && !in)) atomicOr(a.status, STATUS_PAGES);
    const int per_head = dim - half;                // pairs, then the elements that pass
    const int heads = a.q_heads + 2 * a.kv.heads;
    const long long at = in ? (slot / a.kv.page_size) * a.kv.page_stride + (slot % a.kv.page_size) * a.kv.token_stride : 0;
    for (int i = threadIdx.x; i < heads * per_head; i += blockDim.x) {
        const int h = i / per_head, e = i - h * per_head;
        const int kind = h < a.q_heads ? 0 : h < a.q_heads + a.kv.heads ? 1 : 2;     // q, k, v
        const int hk = kind == 0 ? h : kind == 1 ? h - a.q_heads : h - a.q_heads - a.kv.heads;
        if (kind && !in) continue;
        const T *src = reinterpret_cast<const T *>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) +
                       (long long)row * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) + hk * dim;
        int e0, e1 = -1;
        if (e < half) {
            e0 = a.interleaved ? 2 * e : e;
            e1 = a.interleaved ? 2 * e + 1 : e + half;
        } else {
            e0 = e + half;
        }
        float x0 = to_f(src[e0]), x1 = e1 >= 0 ? to_f(src[e1]) : 0.f;
        if (kind < 2 && e1 >= 0) {
            int ax = 0;
            while (ax < 3 && e >= a.bound[ax]) ++ax;
            int p = a.positions[ax * a.axis_stride + row];
            if (p < 0 || p >= a.n_pos) {
                atomicOr(a.status, STATUS_PAGES);
                p = p < 0 ? 0 : a.n_pos - 1;
            }
            const float c = a.cos_sin[(long long)p * a.rot + e], s = a.cos_sin[(long long)p * a.rot + half + e];
            const float y0 = x0 * c - x1 * s;
            x1 = x1 * c + x0 * s;
            x0 = y0;
        }
        if (kind == 0) {
            T *dst = reinterpret_cast<T *>(a.q_out) + (long long)row * a.q_out_stride + hk * dim;
            dst[e0] = from_f<T>(x0);
            if (e1 >= 0) dst[e1] = from_f<T>(x1);
        } else {
            const float *scale = kind == 1 ? a.kv.k_scale : a.kv.v_scale;
            if (scale) {
                x0 /= scale[hk];
                x1 /= scale[hk];
            }
            void *pool = kind == 1 ? a.kv.k : a.kv.v;
            const long long o = at + hk * a.kv.head_stride;
            if (a.kv.dtype == KV_E4M3) {
                __nv_fp8_e4m3 *dst = reinterpret_cast<__nv_fp8_e4m3 *>(pool) + o;
                dst[e0] = __nv_fp8_e4m3(x0);
                if (e1 >= 0) dst[e1] = __nv_fp8_e4m3(x1);
            } else {
                T *dst = reinterpret_cast<T *>(pool) + o;
                dst[e0] = from_f<T>(x0);
                if (e1 >= 0) dst[e1] = from_f<T>(x1);
            }
        }
    }
}

// 16 bytes of a row as 32-bit values; the stores of a cache's types.
template <typename T> struct Piece;
template <> struct Piece<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void open(const uint4 v, float *x) {
        x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ void store(float *p, const float *x) {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    }
};
template <> struct Piece<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void open(const uint4 v, float *x) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *x) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ void store(__nv_fp8_e4m3 *p, const float *x) {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const __nv_fp8x4_e4m3 b(make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
            w[i] = b.__x;
        }
        *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    }
};

// 16 bytes at a time.  A head is cut into `items`: pieces j and j + half / VE,
// which the pairs (i, i + half) join, and behind them single pieces; with
// interleaved pairs, single pieces only.  A row's threads (per_row of them, a
// multiple of the items or cut to one) keep their item from head to head, so that
// its cosines and sines are fetched once; heads are taken U at a time, loads first.
// Bound by memory: 8772 rows of 32 + 2 x 8 heads of 128 with positions of three
// axes, bf16, take 38.0 us, 5800 GB/s (86 % of the copy rate), fp32 67.6 us (95 %),
// bf16 rows to an e4m3 cache 40.3 us (74 %: fewer bytes, and its divisions).  U = 3 or
// 6, 5 or 6 CTAs on an SM and 128 threads for a row are slower.  The 64 registers of
// four CTAs on an SM leave the two bf16 forms 36 bytes of spills.
template <typename T, typename KV>
__global__ void __launch_bounds__(256, 4) kv_append_vec_kernel(const AppendArgs a, int per_row) {
    constexpr int VE = Piece<T>::N, U = 2;
    const int rows = blockDim.x / per_row, sub = threadIdx.x / per_row, t = threadIdx.x - sub * per_row;
    const int row = blockIdx.x * rows + sub;
    if (row >= a.n) return;
    const int dim = a.kv.dim, half = a.rot / 2;
    const int joined = a.interleaved ? 0 : half / VE;
    const int items = dim / VE - joined, heads = a.q_heads + 2 * a.kv.heads;
    const int stride = per_row / items;                 // heads between a thread's turns
    const int item = t % items;
    int h = t / items;
    if (h >= stride) return;
    const bool two = item < joined;
    const int d0 = (two ? item : item + joined) * VE, d1 = d0 + half;
    const bool turned = two || (a.interleaved && d0 < a.rot);

    // the row in q, k and v, and a head's in one of them
    const T *const q_row = reinterpret_cast<const T *>(a.q) + row * a.q_stride;
    const T *const k_row = reinterpret_cast<const T *>(a.k) + row * a.k_stride - a.q_heads * dim;
    const T *const v_row = reinterpret_cast<const T *>(a.v) + row * a.v_stride - (a.q_heads + a.kv.heads) * dim;
    auto source = [&](int hh) -> const T * {
        return (hh < a.q_heads ? q_row : hh < a.q_heads + a.kv.heads ? k_row : v_row) + hh * dim;
    };
    uint4 x0[U], x1[U];
    auto load = [&](int from) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int hh = from + u * stride;
            if (hh >= heads) continue;
            const T *src = source(hh);
            x0[u] = *reinterpret_cast<const uint4 *>(src + d0);
            if (two) x1[u] = *reinterpret_cast<const uint4 *>(src + d1);
        }
    };
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int slot = a.slot_map[row];
    load(h);

    // the item's cosines and sines: VE pairs (half as many where they are interleaved)
    float c[VE], s[VE];
    if (turned) {
        const int pairs = two ? VE : VE / 2, p0 = two ? d0 : d0 / 2;
        auto axis_of = [&](int i) { return (i >= a.bound[0]) + (i >= a.bound[1]) + (i >= a.bound[2]); };
        bool bad = false;
        auto row_of = [&](int ax) {
            int p = a.positions[ax * a.axis_stride + row];
            if (p < 0 || p >= a.n_pos) {
                bad = true;
                p = p < 0 ? 0 : a.n_pos - 1;
            }
            return a.cos_sin + (long long)p * a.rot + p0;
        };
        const int ax = axis_of(p0);
        if (pairs % 4 == 0 && a.table16 && ax == axis_of(p0 + pairs - 1)) {
            const float *at = row_of(ax);
#pragma unroll
            for (int e = 0; e < VE; e += 4) {
                if (e >= pairs) break;
                const float4 x = *reinterpret_cast<const float4 *>(at + e), y = *reinterpret_cast<const float4 *>(at + half + e);
                c[e] = x.x, c[e + 1] = x.y, c[e + 2] = x.z, c[e + 3] = x.w;
                s[e] = y.x, s[e + 1] = y.y, s[e + 2] = y.z, s[e + 3] = y.w;
            }
        } else {                     // an axis ends among the item's pairs
            int last_ax = ax;
            const float *at = row_of(ax);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                if (e >= pairs) break;
                const int next = axis_of(p0 + e);
                if (next != last_ax) at = row_of(next);
                last_ax = next;
                c[e] = at[e];
                s[e] = at[half + e];
            }
        }
        if (bad) atomicOr(a.status, STATUS_PAGES);
    }
    const bool in = slot >= 0 && slot < (long long)a.kv.n_pages * a.kv.page_size;
    if (slot < -1 || (slot >= 0 && !in)) atomicOr(a.status, STATUS_PAGES);
    const long long at = in ? (slot / a.kv.page_size) * a.kv.page_stride + (slot % a.kv.page_size) * a.kv.token_stride : 0;

    T *const q_to = reinterpret_cast<T *>(a.q_out) + row * a.q_out_stride;
    KV *const k_to = reinterpret_cast<KV *>(a.kv.k) + at - a.q_heads * a.kv.head_stride;
    KV *const v_to = reinterpret_cast<KV *>(a.kv.v) + at - (a.q_heads + a.kv.heads) * a.kv.head_stride;
    for (;;) {
        const int next = h + U * stride;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int hh = h + u * stride;
            const bool is_q = hh < a.q_heads, is_v = hh >= a.q_heads + a.kv.heads;
            if (hh >= heads || (!is_q && !in)) continue;
            float y0[VE], y1[VE];
            Piece<T>::open(x0[u], y0);
            if (two) Piece<T>::open(x1[u], y1);
            if (turned && !is_v) {
                if (two) {
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        const float w = y0[e] * c[e] - y1[e] * s[e];
                        y1[e] = y1[e] * c[e] + y0[e] * s[e];
                        y0[e] = w;
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < VE / 2; ++e) {
                        const float w = y0[2 * e] * c[e] - y0[2 * e + 1] * s[e];
                        y0[2 * e + 1] = y0[2 * e + 1] * c[e] + y0[2 * e] * s[e];
                        y0[2 * e] = w;
                    }
                }
            }
            if (is_q) {
                T *dst = q_to + hh * dim;
                Piece<T>::store(dst + d0, y0);
                if (two) Piece<T>::store(dst + d1, y1);
            } else {
                const float *scale = is_v ? a.kv.v_scale : a.kv.k_scale;
                if (scale) {
                    const float f = scale[hh - a.q_heads - (is_v ? a.kv.heads : 0)];
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        y0[e] /= f;
                        if (two) y1[e] /= f;
                    }
                }
                KV *dst = (is_v ? v_to : k_to) + hh * a.kv.head_stride;
                Piece<T>::store(dst + d0, y0);
                if (two) Piece<T>::store(dst + d1, y1);
            }
        }
        if (next >= heads) break;
        h = next;
        load(h);
    }
}

// Whether a call's rows and rotary halves can be taken 16 bytes at a time.
template <typename T>
bool by_pieces(const AppendArgs &a) {
    constexpr int VE = Piece<T>::N;
    if (a.interleaved ? a.rot % VE : (a.rot / 2) % VE) return false;
    uintptr_t p = reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v);
    long long s = a.k_stride % VE | a.v_stride % VE;
    if (a.q_heads) {
        p |= reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.q_out);
        s |= a.q_stride % VE | a.q_out_stride % VE;
    }
    return (p & 15) == 0 && s == 0;
}

__global__ void __launch_bounds__(256) rope_table_kernel(float *out, int n_pos, int half, double theta,
                                                         const double *inv_freq) {
    const long long step = (long long)gridDim.x * blockDim.x, all = (long long)n_pos * half;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < all; i += step) {
        const long long p = i / half;
        const int j = (int)(i - p * half);
        const double f = inv_freq ? inv_freq[j] : pow(theta, -(double)j / half);
        double s, c;
        sincos((double)p * f, &s, &c);
        out[p * 2 * half + j] = (float)c;
        out[p * 2 * half + half + j] = (float)s;
    }
}

}  // namespace

cudaError_t launch_kv_resize(const ResizeArgs &a, int num_sms, cudaStream_t st) {
    // every CTA scans the requests for itself and takes its share of the rows; a
    // small step is one CTA's, which needs no launch-wide arrival
    const int n = a.n_req, threads = n <= 256 ? 256 : RS_THREADS;
    const long long rows = a.max_new > n ? a.max_new : n;
    const int grid = (int)min((long long)num_sms, (rows + threads - 1) / threads + (rows == 0));
    if (n <= RS_THREADS) return launch_resize<1>(a, grid, threads, st);
    if (n <= 4 * RS_THREADS) return launch_resize<4>(a, grid, threads, st);
    return launch_resize<16>(a, grid, threads, st);
}

cudaError_t launch_kv_append(bool f32, const AppendArgs &a, int num_sms, cudaStream_t st) {
    if (f32 ? by_pieces<float>(a) : by_pieces<__nv_bfloat16>(a)) {
        // few rows: a CTA for each, every head at once (64 rows 2.3 us, 64 threads each
        // 3.7; 608 rows 3.6 and 3.9); many: 64 threads for a row, whose cosines are
        // fetched fewer times (1216 rows 5.4 us, 256 threads 6.4; 8772 rows 38.0 and 61.6)
        const int per_row = a.n <= 4 * num_sms ? 256 : 64, rows = 256 / per_row;
        const int grid = (a.n + rows - 1) / rows;
        if (f32) return launch_chained(kv_append_vec_kernel<float, float>, grid, 256, 0, st, a, per_row);
        if (a.kv.dtype == KV_E4M3)
            return launch_chained(kv_append_vec_kernel<__nv_bfloat16, __nv_fp8_e4m3>, grid, 256, 0, st, a, per_row);
        return launch_chained(kv_append_vec_kernel<__nv_bfloat16, __nv_bfloat16>, grid, 256, 0, st, a, per_row);
    }
    if (f32) return launch_chained(kv_append_kernel<float>, a.n, 256, 0, st, a);
    return launch_chained(kv_append_kernel<__nv_bfloat16>, a.n, 256, 0, st, a);
}

cudaError_t launch_rope_table(float *cos_sin, int n_pos, int rot, double theta, const double *inv_freq,
                              cudaStream_t st) {
    const long long all = (long long)n_pos * (rot / 2);
    const int grid = (int)min((all + 255) / 256, (long long)4096);
    rope_table_kernel<<<grid, 256, 0, st>>>(cos_sin, n_pos, rot / 2, theta, inv_freq);
    return cudaGetLastError();
}

}  // namespace scute
