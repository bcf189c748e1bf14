// Rows of a block table that continue rows of another one (kv_fork), and the copy
// of the pages that they cannot share (kv_copy).
#include "internal.h"
#include "ptx.cuh"

namespace scute {

namespace {

// ---------------------------------------------------------------- kv_fork
// Four steps, each over the whole grid and each needing all of the one before:
//   count   every page of an old row loses a holder, every full page of a new row
//           gains one (a page at the same place of the old row and the new row of
//           one number does neither: most pages of a beam's new row are its old
//           one's).  Afterwards extra[p] < 0 says that nobody holds page p whole;
//   claim   a new row whose last page, filled in part, is such a page claims it:
//           the smallest row's mark stays, r - INT_MAX, below every count.  Every page
//           that a new row took whole is looked at again: counts that held fewer rows
//           than the tables named would give it up or to another row, and are recorded;
//   settle  rows whose claim stayed keep the page, others that end in part get their
//           bit set (they copy); pages left without holder are counted by ranges;
//   assign  with L = F + P entries in the list (F old ones, P pages given up, in the
//           order of their numbers), the n-th copying row takes entry L - 1 - n: an
//           old entry, or the page of rank L - 1 - n - F, whose own thread finds the
//           row through the bits; the others of the P are written to the list.
// No step waits for another's threads, so that the order in which the device works
// decides nothing.  Bound by latency, a chain of three or four dependent loads in every
// step and the launches (or the cluster's barriers) between: 64 beams of 200 to 8192 tokens
// 12.5 us, one prompt to 64 samples 15.4, 4096 beams 13.5 (counts and tables are 0.5 MB);
// without the second look at pages held whole 11.1, 12.8 and 12.8.
constexpr int FK_THREADS = 512;
constexpr int FK_LIST = 0, FK_FREED = 16, FK_BITS = FK_FREED + FORK_MAX_CTAS;    // the workspace's parts
constexpr int FK_CLAIM = -(1 << 30);                  // claims are below, counts above
constexpr int FK_SPAN = 256;                          // table entries that a warp takes at a time
constexpr int FK_WORDS = 16384 / 32;

__device__ __forceinline__ int page_index(const ForkArgs &a, int pos) {
    return a.page_shift >= 0 ? pos >> a.page_shift : pos / a.page_size;
}
__device__ __forceinline__ int pages_of(const ForkArgs &a, int tokens) { return tokens == 0 ? 0 : page_index(a, tokens - 1) + 1; }
__device__ __forceinline__ int old_len(const ForkArgs &a, int r, bool *bad) {
    const int cap = a.cols * a.page_size, n = a.len_in[r];
    if (n < 0 || n > cap) *bad = true;
    return n < 0 ? 0 : n > cap ? cap : n;
}
// A new row's source (-1: none) and tokens.
struct NewRow {
    int source, len;
};
__device__ __forceinline__ NewRow new_row(const ForkArgs &a, int r, bool *bad) {
    int s = a.source[r];
    if (s < -1 || s >= a.n_in) *bad = true, s = -1;
    if (s < 0) return {-1, 0};
    const int have = old_len(a, s, bad);
    int n = have;
    if (a.len_new) {
        n = a.len_new[r];
        if (n < 0 || n > have) *bad = true;
        n = n < 0 ? 0 : n > have ? have : n;
    }
    return {s, n};
}
__device__ __forceinline__ bool in_pool(const ForkArgs &a, int p) { return (unsigned)p < (unsigned)a.n_pages; }
__device__ __forceinline__ int now(const int *p) { return *(const volatile int *)p; }

__device__ __forceinline__ void fork_count(const ForkArgs &a, int cta, int ctas) {
    const int lane = threadIdx.x & 31;
    const int rows = max(a.n_in, a.n_out), spans = (a.cols - 1) / FK_SPAN + 1;
    const long long items = (long long)rows * spans, step = (long long)ctas * (FK_THREADS / 32);
    bool bad = false;
    for (long long i = (long long)cta * (FK_THREADS / 32) + (threadIdx.x >> 5); i < items; i += step) {
        const int r = (int)(i / spans), j0 = (int)(i - (long long)r * spans) * FK_SPAN;
        int have = 0, full = 0;
        const int32_t *old = a.table_in, *from = a.table_in;
        if (r < a.n_in) {
            have = pages_of(a, old_len(a, r, &bad));
            old += r * a.in_stride;
        }
        if (r < a.n_out) {
            const NewRow x = new_row(a, r, &bad);
            full = page_index(a, x.len);
            from += max(x.source, 0) * a.in_stride;
        }
        int32_t *to = a.table_out + r * a.out_stride;
        int p[FK_SPAN / 32], q[FK_SPAN / 32];
#pragma unroll
        for (int k = 0; k < FK_SPAN / 32; ++k) {
            const int j = j0 + k * 32 + lane;
            p[k] = j < have ? old[j] : -1;
            q[k] = j < full ? from[j] : -1;
        }
#pragma unroll
        for (int k = 0; k < FK_SPAN / 32; ++k) {
            const int j = j0 + k * 32 + lane;
            if (j < full) to[j] = q[k];
            bad |= (j < have && !in_pool(a, p[k])) || (j < full && !in_pool(a, q[k]));
            if (j < have && j < full && p[k] == q[k]) continue;
            if (j < have && in_pool(a, p[k])) atomicSub(a.extra + p[k], 1);
            if (j < full && in_pool(a, q[k])) atomicAdd(a.extra + q[k], 1);
        }
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.status, STATUS_PAGES);
}

// The page of a new row's last tokens where they do not fill it (-1: none).
__device__ __forceinline__ int last_page(const ForkArgs &a, int r, NewRow *x) {
    bool bad = false;                                  // recorded by the first step
    *x = new_row(a, r, &bad);
    const int full = page_index(a, x->len);
    return x->len > full * a.page_size ? a.table_in[x->source * a.in_stride + full] : -1;
}

__device__ __forceinline__ void fork_claim(const ForkArgs &a, int cta, int ctas) {
    const int lane = threadIdx.x & 31;
    bool bad = false;
    if (cta < a.claiming) {
        for (int r = cta * FK_THREADS + threadIdx.x; r < a.n_out; r += a.claiming * FK_THREADS) {
            NewRow x;
            const int p = last_page(a, r, &x), e = in_pool(a, p) ? now(a.extra + p) : 0;
            if (e >= 0) continue;
            bad |= e < -1 && e > FK_CLAIM;             // more rows than holders: the claim takes the count's place
            atomicMin(a.extra + p, r - INT32_MAX);
        }
    } else {                                           // beside them, so that neither waits for the other's loads
        const int spans = (a.cols - 1) / FK_SPAN + 1, items = a.n_out * a.parts, step = (ctas - a.claiming) * (FK_THREADS / 32);
#pragma unroll 1
        for (int i = (cta - a.claiming) * (FK_THREADS / 32) + (threadIdx.x >> 5); i < items; i += step) {
            const int r = i / a.parts;
            const int32_t *to = a.table_out + r * a.out_stride;
            const int first = i - r * a.parts;
            int full = a.cols;                         // of the first span's entries, asked for before the row's tokens are known
#pragma unroll 1
            for (int s = first; s < spans; s += a.parts) {
                const int j0 = s * FK_SPAN;
                if (j0 >= full) break;
                int q[FK_SPAN / 32], e[FK_SPAN / 32], any = 0;
#pragma unroll
                for (int k = 0; k < FK_SPAN / 32; ++k) {
                    const int j = j0 + k * 32 + lane;
                    q[k] = j < full ? now(to + j) : -1;
                }
                bool seen = false;                     // recorded by the first step
                if (s == first) full = page_index(a, new_row(a, r, &seen).len);
#pragma unroll
                for (int k = 0; k < FK_SPAN / 32; ++k) e[k] = j0 + k * 32 + lane < full && in_pool(a, q[k]) ? now(a.extra + q[k]) : 0;
#pragma unroll
                for (int k = 0; k < FK_SPAN / 32; ++k) any |= e[k];
                bad |= any < 0;
            }
        }
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.status, STATUS_PAGES);
}

// Exclusive prefix sum over the CTA's threads; *total receives the sum.
__device__ __forceinline__ int cta_exclusive(int x, int *warp_sum, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    if (lane == 31) warp_sum[warp] = inc;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < FK_THREADS / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        all += warp_sum[w];
    }
    __syncthreads();
    *total = all;
    return before + inc - x;
}

// A CTA's range of pages.
__device__ __forceinline__ void range_of(const ForkArgs &a, int cta, int ctas, int *p0, int *p1) {
    const int each = (a.n_pages + ctas - 1) / ctas;
    *p0 = (int)min((long long)cta * each, (long long)a.n_pages);
    *p1 = (int)min((long long)*p0 + each, (long long)a.n_pages);
}

__device__ __forceinline__ void fork_settle(const ForkArgs &a, int cta, int ctas, int *warp_sum) {
    bool bad = false;
    const int n32 = (a.n_out + 31) & ~31;
    for (int r = cta * FK_THREADS + threadIdx.x; r < n32; r += ctas * FK_THREADS) {
        bool copies = false;
        if (r < a.n_out) {
            NewRow x;
            const int p = last_page(a, r, &x), full = page_index(a, x.len);
            const bool in_part = x.len > full * a.page_size;
            const bool keeps = in_part && (!in_pool(a, p) || now(a.extra + p) == r - INT32_MAX);
            copies = in_part && !keeps;
            if (keeps) {
                a.table_out[r * a.out_stride + full] = p;
                if (in_pool(a, p)) a.extra[p] = 0;      // another row that asks sees the claim or the holder: not its own
                else bad = true;
            }
            a.len_out[r] = x.len;
            a.copy_from[r] = copies ? p : -1;
            a.copy_to[r] = -1;
            a.copy_tokens[r] = copies ? x.len - full * a.page_size : 0;
        }
        const unsigned bits = __ballot_sync(0xffffffffu, copies);
        if ((threadIdx.x & 31) == 0) a.ws[FK_BITS + r / 32] = (int)bits;
    }
    int p0, p1, mine = 0, total;
    range_of(a, cta, ctas, &p0, &p1);
#pragma unroll 4
    for (int p = p0 + threadIdx.x; p < p1; p += FK_THREADS) {
        const int e = now(a.extra + p);
        if (e < 0 && e > FK_CLAIM) {
            ++mine;
            if (e < -1) bad = true;                     // more rows than holders
        }
    }
    cta_exclusive(mine, warp_sum, &total);
    if (threadIdx.x == 0) a.ws[FK_FREED + cta] = total;
    if (cta == 0 && threadIdx.x == 0) {
        int F = *a.free_in;
        if (F < 0 || F > a.n_free_max) {
            bad = true;
            F = F < 0 ? 0 : (int)a.n_free_max;
        }
        a.ws[FK_LIST] = F;
    }
    if (__any_sync(0xffffffffu, bad) && (threadIdx.x & 31) == 0) atomicOr(a.status, STATUS_PAGES);
}

struct AssignShared {
    int warp_sum[FK_THREADS / 32];
    unsigned bits[FK_WORDS];
    int before[FK_WORDS];          // copying rows before each word's
};
__device__ __forceinline__ void fork_assign(const ForkArgs &a, int cta, int ctas, AssignShared &s) {
    static_assert(FK_WORDS <= FK_THREADS && FORK_MAX_CTAS <= 2 * FK_THREADS, "one word and two ranges of a thread");
    const int t = threadIdx.x, lane = t & 31, words = (a.n_out + 31) / 32;
    const unsigned word = t < words ? (unsigned)now(a.ws + FK_BITS + t) : 0u;
    const int F = now(a.ws + FK_LIST);
    int copies, P, mine_before, total;
    s.bits[t] = word;
    s.before[t] = cta_exclusive(__popc(word), s.warp_sum, &copies);
    int ahead = 0, all = 0;
    for (int i = t; i < ctas; i += FK_THREADS) {
        const int x = now(a.ws + FK_FREED + i);
        all += x;
        if (i < cta) ahead += x;
    }
    cta_exclusive(all, s.warp_sum, &P);
    cta_exclusive(ahead, s.warp_sum, &mine_before);
    const long long L = (long long)F + P, left = max(L - copies, 0ll);
    bool bad = false;

    auto give = [&](int r, int page) {                  // the copying row r its page
        const int full = page_index(a, a.len_out[r]);
        a.table_out[r * a.out_stride + full] = page;
        a.copy_to[r] = page;
    };
    // rows that take an old entry, and rows for which nothing is left
    for (int r = cta * FK_THREADS + t; r < a.n_out; r += ctas * FK_THREADS) {
        const unsigned w = s.bits[r >> 5];
        if (!(w >> (r & 31) & 1)) continue;
        const int nth = s.before[r >> 5] + __popc(w & ((1u << (r & 31)) - 1));
        const long long at = L - 1 - nth;
        if (at < 0) {
            bad = true;
            a.len_out[r] = page_index(a, a.len_out[r]) * a.page_size;
            a.copy_from[r] = -1;
            a.copy_tokens[r] = 0;
        } else if (at < F) {
            const int page = a.free_pages[at];
            bad |= !in_pool(a, page);
            give(r, page);
        }
    }
    // pages that nobody holds any more
    int p0, p1, rank = mine_before;
    range_of(a, cta, ctas, &p0, &p1);
    for (int base = p0; base < p1; base += FK_THREADS) {
        const int p = base + t, e = p < p1 ? now(a.extra + p) : 0;
        const bool gone = e < 0 && e > FK_CLAIM;        // the pages that `settle` counted
        bad |= e <= FK_CLAIM;                           // (claims are settled: no count at all)
        const int k = rank + cta_exclusive(gone, s.warp_sum, &total);
        rank += total;
        if (!gone) continue;
        a.extra[p] = 0;
        const long long at = (long long)F + k;
        if (at < left) {
            if (at < a.n_free_max) a.free_pages[at] = p;
            else bad = true;
            continue;
        }
        const int nth = (int)(L - 1 - at);
        int lo = 0, hi = words - 1;                     // the last word with at most nth rows before it
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s.before[mid] <= nth) lo = mid;
            else hi = mid - 1;
        }
        give(lo * 32 + __fns(s.bits[lo], 0, nth - s.before[lo] + 1), p);
    }
    if (cta == 0 && t == 0) *a.free_out = (int)min(left, a.n_free_max);
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.status, STATUS_PAGES);
}

template <int STEP>
__global__ void __launch_bounds__(FK_THREADS) fork_step_kernel(const ForkArgs a) {
    __shared__ AssignShared s;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    if (STEP == 0) fork_count(a, blockIdx.x, gridDim.x);
    if (STEP == 1) fork_claim(a, blockIdx.x, gridDim.x);
    if (STEP == 2) fork_settle(a, blockIdx.x, gridDim.x, s.warp_sum);
    if (STEP == 3) fork_assign(a, blockIdx.x, gridDim.x, s);
}

// All four by one cluster, its barrier between them: where there is little to do, four
// launches cost more than the step (64 beams with kv_copy: a call through Python 40 us, by four
// launches 49; in a graph, where launches cost less, 17.4 and 16.3).
constexpr int FK_CLUSTER = 8;
__global__ void __cluster_dims__(FK_CLUSTER, 1, 1) __launch_bounds__(FK_THREADS) fork_cluster_kernel(const ForkArgs a) {
    __shared__ AssignShared s;
    const int cta = blockIdx.x;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    auto all_done = [] {
        __threadfence();
        ptx::cluster_sync();
    };
    fork_count(a, cta, FK_CLUSTER);
    all_done();
    fork_claim(a, cta, FK_CLUSTER);
    all_done();
    fork_settle(a, cta, FK_CLUSTER, s.warp_sum);
    all_done();
    fork_assign(a, cta, FK_CLUSTER, s);
}

// ---------------------------------------------------------------- kv_copy
// A CTA looks through `each` rows and copies the pages of those that have one, in one
// pool, 16 bytes to a thread at a time, four of them on their way, in the order in which the
// page's tokens and heads lie.  Bound by memory where many rows copy (4096 beams, some 1150
// pages of one layer in part, 9300 tokens, 38 MB read and 38 written: 16 us), else by its launch
// and the chain from the list to the page (64 rows 5 us).
constexpr int CP_THREADS = 256, CP_ROWS = 32;
__global__ void __launch_bounds__(CP_THREADS) kv_copy_kernel(const PageCopyArgs a, int each) {
    const int lane = threadIdx.x & 31;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int r0 = blockIdx.x * each, mine = r0 + lane;
    const bool asked = lane < each && mine < a.n;
    const int to = asked ? a.to[mine] : -1, from = asked && to != -1 ? a.from[mine] : -1;
    int tokens = asked && a.tokens ? a.tokens[mine] : a.page_size;
    const bool out = (unsigned)from >= (unsigned)a.n_pages || (unsigned)to >= (unsigned)a.n_pages;
    if (to != -1 && (out || tokens < 0 || tokens > a.page_size) && threadIdx.x < 32 && blockIdx.y == 0) atomicOr(a.status, STATUS_PAGES);
    tokens = tokens < 0 ? 0 : min(tokens, a.page_size);
    char *const pool = static_cast<char *>(a.pool[blockIdx.y]);
    // rows of one token and head, the inner of the two the one with the smaller stride
    const bool token_in = a.token_bytes < a.head_bytes;
    const long long in_step = token_in ? a.token_bytes : a.head_bytes, out_step = token_in ? a.head_bytes : a.token_bytes;
    const unsigned pieces = a.row_bytes / 16;
    constexpr int U = 4;
    for (unsigned left = __ballot_sync(0xffffffffu, !out); left; left &= left - 1) {
        const int k = __ffs(left) - 1;
        const char *src = pool + __shfl_sync(0xffffffffu, from, k) * a.page_bytes;
        char *dst = pool + __shfl_sync(0xffffffffu, to, k) * a.page_bytes;
        const unsigned count = __shfl_sync(0xffffffffu, tokens, k), inner = token_in ? count : a.heads;
        const unsigned all = count * a.heads * pieces;              // (below 2^31, by the call's checks)
        for (unsigned e0 = threadIdx.x; e0 < all; e0 += U * CP_THREADS) {
            uint4 x[U];
            long long at[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const unsigned e = e0 + u * CP_THREADS;
                if (e >= all) continue;
                const unsigned row = e / pieces, o = row / inner;
                at[u] = o * out_step + (row - o * inner) * in_step + (e - row * pieces) * 16;
                x[u] = *reinterpret_cast<const uint4 *>(src + at[u]);
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (e0 + u * CP_THREADS < all) *reinterpret_cast<uint4 *>(dst + at[u]) = x[u];
        }
    }
}

}  // namespace

cudaError_t launch_kv_fork(const ForkArgs &args, int num_sms, int *launches, cudaStream_t st) {
    ForkArgs a = args;
    const int warps = FK_THREADS / 32;
    const long long rows = max(a.n_in, a.n_out), items = rows * ((a.cols - 1) / FK_SPAN + 1);
    const int most = min(num_sms, FORK_MAX_CTAS);
    const int row_grid = max(1, min(most, (a.n_out + FK_THREADS - 1) / FK_THREADS));
    const int span_grid = (int)max(1ll, min(4ll * most, (items + warps - 1) / warps));
    const int page_grid = max(row_grid, (int)min((long long)most, ((long long)a.n_pages + FK_THREADS - 1) / FK_THREADS));
    // the claiming step's CTAs: a thread to a row; and warps to a row's entries, two turns of all of
    // them for all rows (4096 rows of up to 32 pages in tables of 8192 columns 75 us, with four turns
    // 80, with a span of every row to each warp in turn 102; without the look 68)
    const auto claims = [&](int grid) {
        a.claiming = min(row_grid, grid - 1);
        a.parts = min((a.cols - 1) / FK_SPAN + 1, max(1, 2 * (grid - a.claiming) * warps / max(a.n_out, 1)));
        return grid;
    };
    // one cluster up to as many table spans and pages as its warps take in a few turns
    if (items <= 4 * FK_CLUSTER * warps && a.n_pages <= 16 * FK_CLUSTER * FK_THREADS) {
        *launches = 1;
        claims(FK_CLUSTER);
        return launch_chained(fork_cluster_kernel, FK_CLUSTER, FK_THREADS, 0, st, a);
    }
    *launches = 4;
    cudaError_t e = launch_chained(fork_step_kernel<0>, span_grid, FK_THREADS, 0, st, a);
    if (e == cudaSuccess) e = launch_chained(fork_step_kernel<1>, claims(row_grid + span_grid), FK_THREADS, 0, st, a);
    if (e == cudaSuccess) e = launch_chained(fork_step_kernel<2>, page_grid, FK_THREADS, 0, st, a);
    if (e == cudaSuccess) e = launch_chained(fork_step_kernel<3>, page_grid, FK_THREADS, 0, st, a);
    return e;
}

cudaError_t launch_kv_copy(const PageCopyArgs &a, int num_sms, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    // rows that copy nothing cost a look: many of them to a CTA where there are many
    const long long blocks = (long long)a.n * a.pools, wanted = 8ll * num_sms;
    const int each = (int)max(1ll, min((long long)CP_ROWS, blocks / wanted));
    cfg.gridDim = dim3((unsigned)((a.n + each - 1) / each), (unsigned)a.pools, 1);
    cfg.blockDim = dim3(CP_THREADS, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv_copy_kernel, a, each);
}

}  // namespace scute
