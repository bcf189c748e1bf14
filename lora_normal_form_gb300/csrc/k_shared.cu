// Attention of one new token of each request over the beginning that the requests of
// a group share: every request's query heads on one key/value head are rows of two
// matrix products with the same keys and values, so that these are read once for the
// group instead of once for each request:
//     S [rows x tokens] = Q K^T,   O [rows x D] = P V,   P = 2^(S - m).
// What it leaves is not an output but parts, a row's maximum m, sum l and unnormalised
// O over some of the tokens; the requests' own tokens leave theirs (k_attend_own.cu), and
// join_kernel below puts the parts of a row together.
//
// What bounds it.  A token costs 2 x D x size bytes and 2 x 2 x rows x D operations (the
// second product twice over, see below, so 3 x 2): with bf16 keys 1.5 x rows
// operations a byte, against the 286 where this GPU's tensor and memory rates
// balance: memory up to 190 rows (48 requests of 4 heads to a key), the products beyond.
//
// Layout.  Work rows are (group, key/value head, up to 2 x 128 rows), their tiles of 128
// tokens one sequence that is cut into equal contiguous ranges, one per CTA, as in
// k_attend.cuh.  In a CTA four warps bring keys and four values to shared memory, each to
// a ring of its own, and two warpgroups each run a stream of its own: scores in tensor
// memory (tcgen05.mma, issued by one of its threads), read back (a thread has a row), their
// weights written over them, the second product from there, into outputs that stay in
// tensor memory.  Up to 128 rows the streams take alternate tiles of the same rows, beyond
// each takes 128 rows of every tile; either way one stream's products run under the
// other's softmax.
//
// Weights go to the second product as two bf16 numbers, one rounded and what that left
// (16 bits of a weight, 2^-17 of it: as in k_attend.cuh with a bf16 cache, where an e4m3
// one's weights have 22), l sums them in 32 bits.  The
// reference m moves only when a score passes it by more than 2^8, so that outputs are
// seldom scaled.  Tokens behind the shared beginning's end are zero in shared memory and
// their scores minus infinity.
//
// Measured (this kernel alone, heads of 128, 32 on 8, us): 32 requests on 131072 tokens, bf16, 95 to
// 100 (5.4 to 5.7 TB/s, 80 to 84 % of the copy rate; tensor pipe 46 %); 64 on 8192, bf16, 21.5, of
// which 6 to 7 pass before the first product (the plan, the first rows, code that is cold) and 4
// with the parts' stores, the rest five tiles a CTA; 10 groups of 25 on 512 to 4032 tokens, e4m3,
// 28, the same with conversions between the copies and the products.  A least range of 3 or 4
// tiles and other row costs change nothing but the smallest calls, which they slow (2 requests
// on 1536 tokens: 15.5 us in all, 17 to 18).
#include <type_traits>

#include <cuda_fp8.h>

#include "internal.h"
#include "ptx.cuh"

namespace scute {

namespace {

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr int TT = 128;                    // tokens of a tile
constexpr int TILE = 128;                  // rows of a stream's tile
constexpr int SOFT = 256, LOAD = 256, THREADS = SOFT + LOAD;
constexpr int ROW_COST = 2;                // what a work row costs beside its tiles, in tiles
constexpr int MIN_TILES = 2;               // of a range
// Tiles whose tokens' marks are kept: a tile's are read by its softmax, which the keys
// SLOTS + 2 tiles on wait for (their slot is free when the products of two tiles on are
// done, and those follow it).
constexpr int OK_RING = 8;
constexpr uint64_t WAIT_NS = 2000000000ull;
constexpr unsigned ALL = 0xffffffffu;

// A whole warp's bounded wait, decided by the warp's votes alone.
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    const uint64_t t0 = ptx::globaltimer();
    for (;;) {
        if (__any_sync(ALL, *abort_flag != 0)) return false;
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (__all_sync(ALL, ptx::mbar_try_wait(bar, parity))) return true;
        if (__any_sync(ALL, ptx::globaltimer() - t0 > WAIT_NS)) {
            *abort_flag = 1;
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    return __all_sync(ALL, ptx::mbar_try_wait(bar, parity)) || wait_long(bar, parity, abort_flag);
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool real) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)), "r"(real ? 16 : 0)
                 : "memory");
}
template <int N>
__device__ __forceinline__ void copies_left() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// This thread's writes to shared memory before, as the tensor cores and their like read it.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void sts16(uint32_t p, uint4 x) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(p), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
}
__device__ __forceinline__ void store32(float *p, const uint32_t *x) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]),
                 "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
}
__device__ __forceinline__ float pow2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t y;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(hi), "f"(lo));
    return y;
}
__device__ __noinline__ float capped(float x, float cap) { return cap * LOG2E * tanhf(x / cap); }
// Two e4m3 values (16 bits of a word) as two bf16 ones, exactly: 4 bits of significand.
__device__ __forceinline__ uint32_t to_bf16(uint32_t pair) {
    uint32_t h;
    asm("{\n\t.reg .b16 lo;\n\tcvt.u16.u32 lo, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(pair));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    return pack_bf16(f.x, f.y);
}

// ---------------------------------------------------------------- tensor memory and products
// 32 columns of this warp's 32 lanes, without a wait.
__device__ __forceinline__ void tmem_load(uint32_t at, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at));
}
// The loads before have arrived (the registers pass through, so that no use moves above).
__device__ __forceinline__ void tmem_loaded(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                   "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                   "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}
__device__ __forceinline__ void tmem_store(uint32_t at, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// The products and their commits are issued by one elected thread of a whole warp (one
// that has branched off issues them three times as slowly where other warps compute: its
// operands go through the warp's own registers; measured, 16 products under FMAs 3.3
// against 0.9 thousand cycles).
// D (+)= A B^T from shared memory, and with A in tensor memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
    asm volatile(
        "{\n\t.reg .pred p, one;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|one, 0xffffffff;\n\t"
        "@one tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accum)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accum) {
    asm volatile(
        "{\n\t.reg .pred p, one;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|one, 0xffffffff;\n\t"
        "@one tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accum)
        : "memory");
}
// Arrive once on `bar` when the products before are done.
__device__ __forceinline__ void commit(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred one;\n\telect.sync _|one, 0xffffffff;\n\t"
        "@one tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar)
        : "memory");
}
// A slab is 64 elements (128 bytes) of each of 128 rows, 8 rows a 1024-byte atom whose
// 16-byte pieces are permuted within their row by the row's number.  Read along the 64
// elements (queries, keys: K-major) or across the rows (values: the inner index of the
// second product is the token, elements of a row lie along N; further slabs one SLAB on).
constexpr uint32_t SLAB = 128 * 128;
__device__ __forceinline__ uint32_t place_of(int row, int piece) {      // of a 16-byte piece in its slabs
    return (piece >> 3) * SLAB + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
}
__device__ __forceinline__ uint64_t slab_desc(uint32_t at, uint32_t lead_bytes) {
    uint64_t d = (uint64_t)((at & 0x3FFFFu) >> 4);
    d |= (uint64_t)(lead_bytes >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}
// fp32 sums of bf16 products, M = 128 rows, N columns; `across`: B read across its rows.
constexpr uint32_t instr_desc(int n, bool across) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (across ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(TILE >> 4) << 24);
}

// ---------------------------------------------------------------- the plan
// Groups, made by every CTA for itself: requests start[g] .. start[g + 1), the tokens
// they share (0 where that is not worth it), the first request that has them all (whose row of the table is read; no
// such request: no places), and the places of the groups before.
struct Plan {
    int start[SHARED_MAX_GROUPS + 1], tokens[SHARED_MAX_GROUPS], lead[SHARED_MAX_GROUPS], blocks[SHARED_MAX_GROUPS];
    long long at[SHARED_MAX_GROUPS + 1];
    long long warp_sum[THREADS / 32];
};
struct Bars {
    uint64_t kfull[4], kempty[4], vfull[4], vempty[4], qfull, qempty, sfull[2], pfull[2], ofull[2], turn[2], drain;
    uint32_t tmem;
    int abort;
    unsigned ok[OK_RING][TT / 32];         // tokens that count, of the last tiles' keys
};

// shared_group (internal.h) from the plan's copies.
__device__ __forceinline__ int group_of(const SharedArgs &a, const Plan &p, int r, int length) {
    int lo = 0, hi = a.n_groups - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.start[mid] <= r) lo = mid;
        else hi = mid - 1;
    }
    return p.tokens[lo] > 0 && length >= p.tokens[lo] && p.start[lo] <= r && r < p.start[lo + 1] ? lo : -1;
}
__device__ __forceinline__ int requests_of(const Plan &p, int g) { return p.start[g + 1] - p.start[g]; }
__device__ __forceinline__ int tiles_of(const Plan &p, int g) { return p.lead[g] == INT32_MAX ? 0 : (p.tokens[g] + TT - 1) / TT; }
__device__ __forceinline__ void make_plan(const SharedArgs &a, Plan &p) {
    static_assert(SHARED_MAX_GROUPS + 1 <= 3 * THREADS, "three groups of a thread");
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, G = a.n_groups;
    const int cap = a.kv.table_cols * a.kv.page_size;
    bool bad = false;
    // (everything that is read is asked for at once)
    int start[4], tokens[3], length = t < a.n_req ? a.kv_len[t] : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) start[i] = 3 * t + i <= G ? a.start[3 * t + i] : 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) tokens[i] = 3 * t + i < G ? a.shared_len[3 * t + i] : 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int g = 3 * t + i;
        if (g > G) break;
        bad |= start[i] < 0 || start[i] > a.n_req || (g < G && start[i + 1] < start[i]);
        p.start[g] = min(max(start[i], 0), a.n_req);
        if (g == G) break;
        bad |= tokens[i] < 0 || tokens[i] > cap;
        tokens[i] = min(max(tokens[i], 0), cap);
        p.tokens[g] = read_together(a, min(max(start[i + 1], 0), a.n_req) - p.start[g], tokens[i]) ? tokens[i] : 0;
        p.lead[g] = INT32_MAX;
    }
    __syncthreads();
    for (int r = t; r < a.n_req; r += THREADS) {
        if (r != t) length = a.kv_len[r];
        bad |= length < 0 || length > cap;
        const int g = group_of(a, p, r, min(max(length, 0), cap));
        if (g >= 0) atomicMin(&p.lead[g], r);
    }
    if (bad && blockIdx.x == 0) atomicOr(a.status, STATUS_PAGES);
    __syncthreads();
    long long mine[3], sum = 0;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int g = 3 * t + i;
        const int tiles = g < G ? tiles_of(p, g) : 0, blocks = tiles ? (requests_of(p, g) + 2 * a.tile_req - 1) / (2 * a.tile_req) : 0;
        if (g < G) p.blocks[g] = blocks;
        mine[i] = (long long)a.kv.heads * blocks * (tiles + ROW_COST);
        sum += mine[i];
    }
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(ALL, inc, o);
        if (lane >= o) inc += y;
    }
    long long at = inc - sum;
    if (G >= 96) {                         // (fewer are all the first warp's)
        if (lane == 31) p.warp_sum[warp] = inc;
        __syncthreads();
        for (int w = 0; w < warp; ++w) at += p.warp_sum[w];
    }
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const int g = 3 * t + i;
        if (g <= G) p.at[g] = at;
        at += mine[i];
    }
    __syncthreads();
}

__device__ __forceinline__ long long quotient(long long x, long long y) {
    return ((x | y) >> 32) == 0 ? (long long)((unsigned)x / (unsigned)y) : x / y;
}
// How the places are cut.
struct Cut {
    long long total;
    int ctas;
    __device__ __forceinline__ Cut(const SharedArgs &a, const Plan &p) {
        total = p.at[a.n_groups];
        ctas = (int)min((long long)gridDim.x, quotient(total + MIN_TILES - 1, MIN_TILES));
    }
    __device__ __forceinline__ long long start(int cta) const { return quotient(total * cta, ctas); }
    __device__ __forceinline__ int owner(long long x) const { return (int)quotient((x + 1) * ctas - 1, total); }
};
// A work row: its group, key/value head, block of requests, and where its parts go.
struct WorkRow {
    int g, hk, r0, requests;      // the block's first request and number of them
    bool twin;                    // both streams take the same rows
    int first_row;                // of its parts in the workspace, before the CTA's own offset
};
__device__ __forceinline__ WorkRow work_row(const SharedArgs &a, const Plan &p, int g, int row) {
    WorkRow w;
    const int blocks = p.blocks[g], all = requests_of(p, g);
    w.g = g;
    w.hk = blocks == 1 ? row : row / blocks;
    const int b = row - w.hk * blocks;
    w.r0 = p.start[g] + b * 2 * a.tile_req;
    w.requests = min(2 * a.tile_req, all - b * 2 * a.tile_req);
    w.twin = w.requests <= a.tile_req;
    // twice a row's room: a twin's streams each leave all of the rows
    w.first_row = a.first_row + 2 * a.group * (p.start[g] * a.kv.heads + w.hk * all + b * 2 * a.tile_req);
    return w;
}
__device__ __forceinline__ int stream_requests(const SharedArgs &a, const WorkRow &w, int x) {
    return w.twin ? w.requests : x == 0 ? a.tile_req : w.requests - a.tile_req;
}
// First row of a CTA's part of stream x.
__device__ __forceinline__ int part_row(const SharedArgs &a, const WorkRow &w, int cta, int x) {
    return w.first_row + 2 * TILE * cta + (x ? stream_requests(a, w, 0) * a.group : 0);
}

// Walks a CTA's range, work row by work row: tiles t0 .. t1 of each.
struct Walk {
    const SharedArgs &a;
    const Plan &p;
    long long base, end;
    int g, row, rows, tiles, t0, t1;
    WorkRow w;
    __device__ __forceinline__ Walk(const SharedArgs &args, const Plan &plan, const Cut &cut, int cta) : a(args), p(plan) {
        base = end = g = row = rows = tiles = t0 = t1 = 0;
        if (cta >= cut.ctas) return;
        const long long x = cut.start(cta);
        end = cut.start(cta + 1);
        g = 0;
        for (int hi = a.n_groups - 1; g < hi;) {          // the last group whose places begin at x or before
            const int mid = (g + hi + 1) >> 1;
            if (p.at[mid] <= x) g = mid;
            else hi = mid - 1;
        }
        group();
        row = tiles ? (int)quotient(x - p.at[g], tiles + ROW_COST) : 0;
        base = p.at[g] + (long long)row * (tiles + ROW_COST);
        set(x);
    }
    __device__ __forceinline__ void group() {
        tiles = tiles_of(p, g);
        rows = a.kv.heads * p.blocks[g];
    }
    __device__ __forceinline__ void set(long long from) {
        t0 = (int)max(0ll, from - base - ROW_COST);
        t1 = (int)min((long long)tiles, end - base - ROW_COST);
        if (more()) w = work_row(a, p, g, row);
    }
    __device__ __forceinline__ bool more() const { return tiles > 0 && base + ROW_COST < end; }
    __device__ __forceinline__ void next() {
        base += tiles + ROW_COST;
        if (++row == rows) {
            row = 0;
            do ++g;
            while (g < a.n_groups && tiles_of(p, g) == 0);
            if (g < a.n_groups) group();
            else tiles = 0;
        }
        set(base);
    }
};

// What the join needs of each request and key/value head, by the four warps that bring keys.
__device__ __forceinline__ void write_pieces(const SharedArgs &a, const Plan &p, const Cut &cut, int t) {
    const int H = a.kv.heads;
    for (long long i = (long long)blockIdx.x * (LOAD / 2) + t; i < (long long)a.n_req * H; i += (long long)gridDim.x * (LOAD / 2)) {
        const int r = (int)(i / H), hk = (int)(i - (long long)r * H);
        int4 piece = make_int4(0, -1, 0, 0);
        const int g = group_of(a, p, r, length_of(a, r));
        if (g >= 0) {
            const int tiles = tiles_of(p, g), b = (r - p.start[g]) / (2 * a.tile_req), blocks = p.blocks[g];
            const int row = hk * blocks + b;
            const WorkRow w = work_row(a, p, g, row);
            const int x = !w.twin && r - w.r0 >= a.tile_req;
            const long long base = p.at[g] + (long long)row * (tiles + ROW_COST) + ROW_COST;
            piece.x = cut.owner(base);
            piece.y = cut.owner(base + tiles - 1) | (w.twin ? SHARED_TWIN : 0);
            piece.z = part_row(a, w, 0, x);
            piece.w = stream_requests(a, w, x) * a.group | (r - w.r0 - x * a.tile_req) * a.group << 16;
        }
        a.piece[i] = piece;
    }
}

// ---------------------------------------------------------------- the kernel
template <bool FP8, int DC>
struct Shape {
    static constexpr int SLABS = DC / 64, TILE_BYTES = SLABS * SLAB;
    static constexpr int SLOTS = DC == 64 ? 4 : 2;             // of keys, and of values
    static constexpr int SMEM = 1024 + (2 + 2 * SLOTS) * TILE_BYTES + (int)sizeof(Plan) + (int)sizeof(Bars) + 64;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};

template <bool FP8, int DC>
__global__ void __launch_bounds__(THREADS, 1) shared_kernel(const SharedArgs a) {
    using S = Shape<FP8, DC>;
    constexpr int SLOTS = S::SLOTS, TB = S::TILE_BYTES, ESZ = FP8 ? 1 : 2;
    constexpr int S_COL = 0, O_COL = 2 * TT;                   // columns of tensor memory
    extern __shared__ uint8_t raw[];
    uint8_t *const tiles_at = raw + ((1024 - (ptx::smem_u32(raw) & 1023)) & 1023);
    const uint32_t q_at = ptx::smem_u32(tiles_at), k_at = q_at + 2 * TB, v_at = k_at + SLOTS * TB;
    Bars &b = *reinterpret_cast<Bars *>(tiles_at + (2 + 2 * SLOTS) * TB);
    Plan &p = *reinterpret_cast<Plan *>(reinterpret_cast<uint8_t *>(&b) + ((sizeof(Bars) + 15) & ~15));
    volatile int *const abort_flag = &b.abort;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, D = a.kv.dim, H = a.kv.heads, G = a.group;
    auto bar = [&](uint64_t &x) { return ptx::smem_u32(&x); };

    if (tid == 0) {
        b.abort = 0;
        for (int i = 0; i < SLOTS; ++i) {
            ptx::mbar_init(bar(b.kfull[i]), 4);
            ptx::mbar_init(bar(b.kempty[i]), 2 + a.hold);
            ptx::mbar_init(bar(b.vfull[i]), 4);
            ptx::mbar_init(bar(b.vempty[i]), 2);
        }
        ptx::mbar_init(bar(b.qfull), 8);
        ptx::mbar_init(bar(b.qempty), 2);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(bar(b.sfull[i]), 1);
            ptx::mbar_init(bar(b.pfull[i]), 4);
            ptx::mbar_init(bar(b.ofull[i]), 1);
            ptx::mbar_init(bar(b.turn[i]), 1);
        }
        ptx::mbar_init(bar(b.drain), 2);
        ptx::fence_mbar_init();
    }
    // behind a head's elements every row of a tile stays zero
    if (D < DC) {
        for (int i = tid; i < (2 + 2 * SLOTS) * TB / 16; i += THREADS) sts16(q_at + i * 16, make_uint4(0, 0, 0, 0));
        fence_async();
    }
    if (warp == 0) {
        ptx::tmem_alloc(ptx::smem_u32(&b.tmem), 512);
        ptx::tmem_relinquish();
        ptx::tc_fence_before();
    }
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    make_plan(a, p);                       // (its barriers order what was written above)
    ptx::tc_fence_after();
    // a number that every lane has, as one that the whole warp has
    auto same = [](auto y) { return __shfl_sync(ALL, y, 0); };
    const uint32_t tmem = same(b.tmem);
    const Cut cut(a, p);
    const int cta = blockIdx.x;
    Walk w(a, p, cut, cta);

    if (warp < SOFT / 32) {
        // ------------------------------------------------ a stream: its softmax, a thread to a row; its first
        // warp issues its products
        constexpr uint32_t QK = instr_desc(TT, false), PV = instr_desc(DC, true);
        const int x = same(warp >> 2), i = (warp & 3) * 32 + lane;
        const bool issues = (warp & 3) == 0;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t s_col = tmem + S_COL + x * TT, o_col = tmem + O_COL + x * DC, s_at = s_col + lanes, o_at = o_col + lanes;
        unsigned s_phase = 0, o_phase = 0, p_phase = 0, q_phase = 0, seq = 0;      // seq: tiles of the CTA before this work row's
        // The streams issue in turn, each the second product of its tile and the scores of
        // its next: one's run under the other's softmax.  (Side by side both would wait for
        // the products at once and for the softmax at once: 64 requests on 8192 tokens,
        // 3.8 us for a tile of each against 3.2.)
        unsigned turn_phase = x == 0 ? 1 : 0;
        auto my_turn = [&] {
            const bool yes = wait_bar(bar(b.turn[x]), turn_phase, abort_flag);
            turn_phase ^= 1;
            return yes;
        };
        auto pass_turn = [&] {
            if (lane == 0) ptx::mbar_arrive(bar(b.turn[1 - x]));
            __syncwarp();
        };
        bool live = true;
        for (; live && w.more(); w.next()) {
            const bool twin = w.w.twin;
            const int step = twin ? 2 : 1, t_first = w.t0 + (twin ? x : 0), uses = twin ? 2 : 1;
            // tile t's slot of a ring, and the parity of its filling
            auto slot_of = [&](int t) { return (seq + (t - w.t0)) % SLOTS; };
            auto phase_of = [&](int t) { return (seq + (t - w.t0)) / SLOTS & 1; };
            // scores of the stream's tile t (its weights before have been multiplied: the
            // products of one thread run in the order of their issue)
            auto scores = [&](int t) {
                const int slot = slot_of(t);
                live = wait_bar(bar(b.kfull[slot]), phase_of(t), abort_flag);
                if (!live) return;
                ptx::tc_fence_after();
                const uint64_t qd = same(slab_desc(q_at + (twin ? 0 : x) * TB, 16)), kd = same(slab_desc(k_at + slot * TB, 16));
#pragma unroll
                for (int k = 0; k < DC / 16; ++k) {
                    const uint32_t off = ((k / 4) * SLAB + (k % 4) * 32) >> 4;
                    mma_ss(s_col, qd + off, kd + off, QK, k > 0);
                }
                commit(bar(b.sfull[x]));
                for (int k = 0; k < uses; ++k) commit(bar(b.kempty[slot]));
                if (t + step >= w.t1) commit(bar(b.qempty));
            };
            // Tile t's values, which the other stream takes, have come.  Both streams see every
            // filling of a slot before it is given back: its barrier's parity tells only two
            // fillings apart.
            auto seen_values = [&](int t) {
                if (!wait_bar(bar(b.vfull[slot_of(t)]), phase_of(t), abort_flag)) return false;
                if (lane == 0) ptx::mbar_arrive(bar(b.vempty[slot_of(t)]));
                __syncwarp();
                return true;
            };
            if (issues) {
                live = wait_bar(bar(b.qfull), q_phase, abort_flag);
                if (!live) break;
                q_phase ^= 1;
                if (t_first < w.t1) scores(t_first);
                else if (lane == 0) ptx::mbar_arrive(bar(b.qempty));
                if (!live) break;
            }
            const float scale = (a.kv.k_scale ? a.kv.k_scale[w.w.hk] : 1.f) * a.scale;
            const float mul = a.softcap > 0.f ? scale : scale * LOG2E;
            float top = -INFINITY;
            uint64_t sum[2] = {0, 0};                          // of the even and the odd tokens' weights, each in two
            bool any = false;
            for (int t = t_first; t < w.t1; t += step) {
                live = (!issues || !twin || t == w.t0 || seen_values(t - 1)) && wait_bar(bar(b.sfull[x]), s_phase, abort_flag);
                if (!live) break;
                s_phase ^= 1;
                ptx::tc_fence_after();
                uint32_t r[32], r2[32];
                float f = mul;
                const volatile unsigned *ok = b.ok[(seq + (t - w.t0)) % OK_RING];
                if (a.softcap > 0.f || (ok[0] & ok[1] & ok[2] & ok[3]) != ALL) {     // scores as they count, put back
#pragma unroll 1
                    for (int c = 0; c < TT / 32; ++c) {
                        uint32_t y[32];
                        const unsigned count = ok[c];
                        tmem_load(s_at + c * 32, y);
                        tmem_loaded(y);
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            float z = __uint_as_float(y[k]) * mul;
                            if (a.softcap > 0.f) z = capped(z, a.softcap);
                            y[k] = __float_as_uint(count >> k & 1 ? z : -INFINITY);
                        }
                        __syncwarp();
                        tmem_store(s_at + c * 32, y);
                    }
                    tmem_stored();
                    f = 1.f;
                }
                // (a negative factor turns the scores' order round)
                const float sign = f < 0.f ? -1.f : 1.f;
                float most[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                auto take = [&](const uint32_t (&y)[32]) {
                    if (f < 0.f) {
#pragma unroll
                        for (int k = 0; k < 32; k += 2)
                            most[k / 2 & 3] = fmaxf(fmaxf(-__uint_as_float(y[k]), -__uint_as_float(y[k + 1])), most[k / 2 & 3]);
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; k += 2)
                            most[k / 2 & 3] = fmaxf(fmaxf(__uint_as_float(y[k]), __uint_as_float(y[k + 1])), most[k / 2 & 3]);
                    }
                };
                tmem_load(s_at, r);
#pragma unroll
                for (int c = 0; c < TT / 32; c += 2) {
                    tmem_loaded(r);
                    tmem_load(s_at + (c + 1) * 32, r2);
                    take(r);
                    tmem_loaded(r2);
                    if (c + 2 < TT / 32) tmem_load(s_at + (c + 2) * 32, r);
                    take(r2);
                }
                const float mx = fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3])) * (f * sign);
                if (__any_sync(ALL, mx > top + 8.f)) {
                    const float to = fmaxf(mx, top), al = to == top ? 1.f : exp2f(top - to);
                    top = to;
                    sum[0] = ptx::fma_two(sum[0], ptx::two(al, al), 0), sum[1] = ptx::fma_two(sum[1], ptx::two(al, al), 0);
                    if (any) {
#pragma unroll 1
                        for (int c = 0; c < DC / 32; ++c) {
                            tmem_load(o_at + c * 32, r);
                            tmem_loaded(r);
#pragma unroll
                            for (int k = 0; k < 32; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * al);
                            tmem_store(o_at + c * 32, r);
                        }
                        tmem_stored();
                    }
                }
                const bool adds = any;
                any = true;
                const float ref = top == -INFINITY ? 0.f : top;
                const uint64_t f2 = ptx::two(f, f), ref2 = ptx::two(-ref, -ref);
                auto weights = [&](const uint32_t (&y)[32], uint32_t at) {
                    uint32_t w2[32];
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float2 e = ptx::apart(ptx::fma_two(ptx::two(__uint_as_float(y[2 * k]), __uint_as_float(y[2 * k + 1])), f2, ref2));
                        const float p0 = pow2(e.x), p1 = pow2(e.y);
                        const uint64_t both = ptx::two(p0, p1);
                        sum[k & 1] = ptx::add_two(sum[k & 1], both);
                        const uint32_t hi = pack_bf16(p0, p1);
                        const float2 left = ptx::apart(ptx::add_two(both, ptx::two(-__uint_as_float(hi << 16), -__uint_as_float(hi & 0xffff0000u))));
                        w2[k] = hi;
                        w2[16 + k] = pack_bf16(left.x, left.y);
                    }
                    tmem_store(at, w2);
                };
                tmem_load(s_at, r);
#pragma unroll
                for (int c = 0; c < TT / 32; c += 2) {
                    tmem_loaded(r);
                    tmem_load(s_at + (c + 1) * 32, r2);
                    weights(r, s_at + c * 32);
                    tmem_loaded(r2);
                    if (c + 2 < TT / 32) tmem_load(s_at + (c + 2) * 32, r);
                    weights(r2, s_at + (c + 1) * 32);
                }
                tmem_stored();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(bar(b.pfull[x]));
                if (!issues) continue;
                const int slot = slot_of(t);
                live = wait_bar(bar(b.pfull[x]), p_phase, abort_flag) && wait_bar(bar(b.vfull[slot]), phase_of(t), abort_flag) && my_turn();
                if (!live) break;
                p_phase ^= 1;
                ptx::tc_fence_after();
                const uint64_t vd = same(slab_desc(v_at + slot * TB, SLAB));
#pragma unroll
                for (int k = 0; k < TT / 16; ++k) {
                    const uint32_t col = s_col + (k / 2) * 32 + (k % 2) * 8;
                    mma_ts(o_col, col, vd + k * (2048 >> 4), PV, adds || k > 0);
                    mma_ts(o_col, col + 16, vd + k * (2048 >> 4), PV, 1);
                }
                commit(bar(b.vempty[slot]));
                if (t + step >= w.t1) commit(bar(b.ofull[x]));
                if (t + step < w.t1) scores(t + step);
                if (!live) break;
                pass_turn();
            }
            if (live && issues && twin && x == 1 && (w.t1 - w.t0) % 2) {      // the other stream had one tile more
                live = my_turn();
                if (live) pass_turn();
            }
            if (!live) break;
            if (issues && twin && (w.t1 - w.t0 - 1) % 2 != x) live = seen_values(w.t1 - 1);
            if (!live) break;
            seq += w.t1 - w.t0;
            // the stream's part, 32 bytes of a row at a time
            const int n = stream_requests(a, w.w, x) * G, at = part_row(a, w.w, cta, x);
            const float2 l0 = ptx::apart(sum[0]), l1 = ptx::apart(sum[1]);
            const float l = (l0.x + l0.y) + (l1.x + l1.y);
            if (l != l && top == -INFINITY) top = 0.f;         // no number: not an empty part
            if (i < n) a.stat[at + i] = make_float2(any ? top : -INFINITY, any ? l : 0.f);
            if (any) {
                live = wait_bar(bar(b.ofull[x]), o_phase, abort_flag);
                if (!live) break;
                o_phase ^= 1;
                ptx::tc_fence_after();
                float *to = a.o + (long long)(at + i) * D;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t r[32];
                    tmem_load(o_at + c, r);
                    tmem_loaded(r);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (i < n && c + 8 * k < D) store32(to + c + 8 * k, &r[8 * k]);
                    }
                    __syncwarp();
                }
                ptx::tc_fence_before();
            }
        }
        if (issues) {
            // nothing may be under way when tensor and shared memory are given back
            commit(bar(b.drain));
            const uint64_t t0 = ptx::globaltimer();
            while (!__all_sync(ALL, ptx::mbar_try_wait(bar(b.drain), 0)) && __all_sync(ALL, ptx::globaltimer() - t0 < WAIT_NS)) {}
        }
        ptx::tc_fence_before();
    } else {
        // ------------------------------------------------ four warps bring keys, four values; each a tile of queries
        const bool keys = warp < SOFT / 32 + 4;
        const int lw = warp & 3;                               // rows 32 lw .. of a tile are this warp's
        // lanes of a row, rows of an instruction; a lane keeps its 16-byte piece
        constexpr int LR = DC * ESZ / 16, RI = 32 / LR, INSTR = 32 / RI;
        const int piece = lane % LR, row0 = lane / LR;
        const bool here = piece * 16 < D * ESZ;                // the others' pieces are zero for good
        const long long tok_bytes = a.kv.token_stride * ESZ;
        const uint32_t lane_at = place_of(lw * 32 + row0, FP8 ? 2 * piece : piece);
        // row n RI + row0 lies n RI rows from row0's place, but for the permutation
        constexpr int TURNS = 8 / RI;
        uint32_t turned[TURNS];
#pragma unroll
        for (int n = 0; n < TURNS; ++n) turned[n] = lane_at ^ (n * RI << 4);
        auto row_at = [&](int n) { return turned[n % TURNS] + n * RI * 128; };
        bool live = true, bad = false;
        uint32_t waiting = 0;                                  // the barrier of the filling on its way (0: none)
        auto told = [&](uint32_t x) {                          // a filling has landed
            fence_async();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(x);
        };
        auto sent = [&](uint32_t x) {
            ptx::cp_async_commit();
            if (waiting) {
                copies_left<1>();
                told(waiting);
            }
            waiting = x;
        };
        auto all_told = [&] {
            copies_left<0>();
            if (waiting) told(waiting);
            waiting = 0;
        };
        const uint32_t ring = keys ? k_at : v_at;
        uint64_t *const full = keys ? b.kfull : b.vfull, *const empty = keys ? b.kempty : b.vempty;
        int slot = 0;
        unsigned phase = 1, q_phase = 1, seq = 0;
        for (; live && w.more(); w.next()) {
            const int tokens = p.tokens[w.g];
            const int32_t *table = a.kv.table + p.lead[w.g] * a.kv.table_stride;
            const char *const from = reinterpret_cast<const char *>(keys ? a.kv.k : a.kv.v) + w.w.hk * a.kv.head_stride * ESZ;
            auto page_of = [&](int t) {                        // of this lane's token of tile t
                const int token = t * TT + lw * 32 + lane;
                return t < w.t1 && token < tokens ? table[a.page_shift >= 0 ? token >> a.page_shift : token / a.kv.page_size] : -1;
            };
            auto place_in = [&](int t, int page) -> long long {
                const int token = t * TT + lw * 32 + lane;
                if (token >= tokens) return -1;
                if (page < 0 || page >= a.kv.n_pages) {
                    bad = true;
                    return -1;
                }
                const int in = a.page_shift >= 0 ? token & (a.kv.page_size - 1) : token % a.kv.page_size;
                return ((long long)page * a.kv.page_stride + (long long)in * a.kv.token_stride) * ESZ;
            };
            // the tile's rows: every lane's own, and whether its halves of 16 step by the
            // token's stride (they lie in one page)
            struct Rows {
                long long place;
                unsigned steps;
            };
            auto rows_of = [&](int t, int page) {
                Rows y;
                y.place = place_in(t, page);
                y.steps = 0;
#pragma unroll
                for (int f = 0; f < 32; f += 16) {
                    const long long p0 = __shfl_sync(ALL, y.place, f);
                    if (__all_sync(ALL, (lane & 16) != f || (y.place >= 0 && y.place == p0 + (lane - f) * tok_bytes))) y.steps |= 1u << (f / 16);
                }
                return y;
            };
            // go(n, source, whether it counts) of every instruction
            auto each = [&](const Rows &y, auto &&go) {
#pragma unroll
                for (int f = 0; f < 32; f += 16) {
                    constexpr int N = 16 / RI;
                    if (y.steps >> (f / 16) & 1) {
                        const char *src = from + __shfl_sync(ALL, y.place, f) + row0 * tok_bytes + piece * 16;
                        if (here) {
#pragma unroll
                            for (int n = 0; n < N; ++n) {
                                go(f / RI + n, src, std::true_type{});
                                src += RI * tok_bytes;
                            }
                        }
                    } else {
#pragma unroll
                        for (int n = 0; n < N; ++n) {
                            const long long at = __shfl_sync(ALL, y.place, f + n * RI + row0);
                            if (here) go(f / RI + n, at >= 0 ? from + at + piece * 16 : from, at >= 0);
                        }
                    }
                }
            };
            auto copy = [&](uint32_t to, const Rows &y) {                           // 16-bit rows, asynchronously
                each(y, [&](int n, const char *src, auto real) {
                    if constexpr (std::is_same_v<decltype(real), std::true_type>) ptx::cp_async16(to + row_at(n), src);
                    else copy16(to + row_at(n), src, real);
                });
            };
            auto fetch = [&](uint4 (&x)[INSTR], const Rows &y) {                    // 8-bit rows, through registers
                each(y, [&](int n, const char *src, auto real) {
                    x[n] = real ? *reinterpret_cast<const uint4 *>(src) : make_uint4(0, 0, 0, 0);
                });
            };
            auto store = [&](uint32_t to, const uint4 (&x)[INSTR]) {
#pragma unroll
                for (int n = 0; n < INSTR; ++n) {
                    const uint32_t word[4] = {x[n].x, x[n].y, x[n].z, x[n].w}, at = to + row_at(n);
                    uint32_t out[8];
#pragma unroll
                    for (int k = 0; k < 4; ++k) out[2 * k] = to_bf16(word[k] & 0xffffu), out[2 * k + 1] = to_bf16(word[k] >> 16);
                    if (!here) continue;
                    sts16(at, make_uint4(out[0], out[1], out[2], out[3]));
                    sts16(at ^ 16, make_uint4(out[4], out[5], out[6], out[7]));
                }
            };
            int page = page_of(w.t0);
            // the queries: the block's rows, request by request
            all_told();
            live = wait_bar(bar(b.qempty), q_phase, abort_flag);
            if (!live) break;
            q_phase ^= 1;
            if (keys || !w.w.twin) {
                constexpr int QL = DC / 8, QR = 32 / QL;       // lanes of a row, rows of an instruction
                const int x = keys ? 0 : 1, n = stream_requests(a, w.w, x);
                const int row = lw * 32 + lane, in = row / G, r = w.w.r0 + x * a.tile_req + in;
                // in pieces of 16 bytes (rows of requests without the shared tokens are of no use, and no harm)
                const int own = in < n ? (int)((r * a.q_stride + (long long)(w.w.hk * G + row - in * G) * D) / 8) : -1;
                const int q_piece = lane % QL;
                const uint32_t to = q_at + x * TB;
                const uint4 *const q = reinterpret_cast<const uint4 *>(a.q);
#pragma unroll 8
                for (int k = 0; k < 32 / QR; ++k) {
                    const int in_tile = k * QR + lane / QL, at = __shfl_sync(ALL, own, in_tile);
                    if (q_piece * 8 < D) copy16(to + place_of(lw * 32 + in_tile, q_piece), at >= 0 ? q + at + q_piece : q, at >= 0);
                }
            }
            sent(bar(b.qfull));
            // (8-bit rows of a tile are on their way while the slot is waited for)
            Rows now = rows_of(w.t0, page);
            page = page_of(w.t0 + 1);
            uint4 x[FP8 ? INSTR : 1];
            if constexpr (FP8) fetch(x, now), all_told();      // (no later copy tells of the queries)
            for (int t = w.t0; t < w.t1; ++t) {
                live = wait_bar(bar(empty[slot]), phase, abort_flag);
                if (!live) break;
                if (keys) {
                    const unsigned ok = __ballot_sync(ALL, now.place >= 0);
                    if (lane == 0) *(volatile unsigned *)&b.ok[seq % OK_RING][lw] = ok;
                    ++seq;
                }
                if constexpr (FP8) {
                    store(ring + slot * TB, x);
                    if (t + 1 < w.t1) now = rows_of(t + 1, page), fetch(x, now);
                    told(bar(full[slot]));
                } else {
                    copy(ring + slot * TB, now);
                    if (t == w.t0) {                           // the first products wait for these
                        sent(bar(full[slot]));
                        if (t + 1 < w.t1) now = rows_of(t + 1, page);
                        all_told();
                    } else {
                        if (t + 1 < w.t1) now = rows_of(t + 1, page);
                        sent(bar(full[slot]));
                    }
                }
                page = page_of(t + 2);
                if (++slot == SLOTS) slot = 0, phase ^= 1;
            }
        }
        all_told();
        if (__any_sync(ALL, bad) && lane == 0) atomicOr(a.status, STATUS_PAGES);
        // while the last tiles are worked on (by the streams, before their first weights, it held
        // the first CTAs up by 4 thousand cycles: 64 requests on 8192 tokens 39.0 us, now 38.5)
        if (keys) write_pieces(a, p, cut, tid - SOFT);
    }
    __syncthreads();
    if (b.abort && tid == 0) atomicOr(a.status, STATUS_TIMEOUT);
    if (warp == 0) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

template <bool FP8, int DC>
cudaError_t launch_shape(const SharedArgs &a, int num_sms, cudaStream_t st) {
    using S = Shape<FP8, DC>;
    static std::atomic<unsigned long long> done{0};
    const auto kernel = shared_kernel<FP8, DC>;
    const cudaError_t e = allow_max_dynamic_smem(kernel, done);
    if (e != cudaSuccess) return e;
    return launch_chained(kernel, num_sms, THREADS, S::SMEM, st, a);
}

// ---------------------------------------------------------------- groups that no kernel reads
// The status of the groups' numbers (make_plan's), where each request is read alone.  Launched
// behind that attention, whose CTAs have all waited for what is read here, and beside it: 0.3 to
// 0.5 us of a call of 12 to 48.
__global__ void __launch_bounds__(256) check_groups_kernel(const int32_t *start, const int32_t *length, int groups, int n_req, int cap,
                                                           int *status) {
    ptx::grid_dep_launch();
    bool bad = false;
    for (int g = threadIdx.x; g <= groups; g += 256) {
        const int from = start[g];
        bad |= from < 0 || from > n_req || (g < groups && (start[g + 1] < from || length[g] < 0 || length[g] > cap));
    }
    if (bad) atomicOr(status, STATUS_PAGES);
    ptx::grid_dep_wait();
}

// ---------------------------------------------------------------- the parts of a request's heads, joined
// out = sum_i 2^(m_i - m) O_i / sum_i 2^(m_i - m) l_i over the parts of a head: that of
// its own tokens, and those of the tokens its group shares, in the order of their CTAs.
// JG threads share the parts of four elements, B loads of each on their way at once; a
// head's parts are then added up in shared memory in a fixed order.  Bound by the latency of
// two dependent loads and by L2: 7.5 us for the 22 MB of parts of 64 requests on 8192 tokens
// (38.8 us in all; four threads with eight loads 41.0, with six 39.0, eight with three 40.2).
constexpr int JOIN_THREADS = 256;
template <int JG, int B>
__global__ void __launch_bounds__(JOIN_THREADS) join_kernel(const JoinArgs a) {
    __shared__ float s_m[JG > 1 ? JOIN_THREADS : 1], s_l[JG > 1 ? JOIN_THREADS : 1];
    __shared__ float4 s_o[JG > 1 ? JOIN_THREADS : 1];
    const int quads = a.dim / 4, per = JOIN_THREADS / (JG * quads), t = threadIdx.x;
    const int in = t / (JG * quads), rest = t - in * JG * quads, part0 = rest / quads, d = (rest - part0 * quads) * 4;
    const int row = blockIdx.x * per + in;
    const bool real = in < per && row < a.rows;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    float m = -INFINITY, l = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    const int r = real ? row / a.q_heads : 0, h = row - r * a.q_heads, hk = h / a.group;
    if (real) {
        const int4 piece = a.piece ? a.piece[(long long)r * (a.q_heads / a.group) + hk] : make_int4(0, -1, 0, 0);
        const int twin = piece.y >= 0 && piece.y & SHARED_TWIN ? 1 : 0, n = piece.w & 0xffff, i = (piece.w >> 16) + h - hk * a.group;
        const int2 its = a.own_at[r];
        const int own = its.x, owns = its.y;
        const int parts = owns + (piece.y < 0 ? 0 : ((piece.y & ~SHARED_TWIN) - piece.x + 1) << twin);
#pragma unroll 1
        for (int k0 = part0; k0 < parts; k0 += JG * B) {
            float2 s[B];
            float4 y[B];
#pragma unroll
            for (int k = 0; k < B; ++k) {
                const int at = k0 + k * JG;
                s[k] = make_float2(-INFINITY, 0.f);
                if (at >= parts) continue;
                // the parts of its own tokens are the first ones
                const int shared = at - owns;
                const int from = shared < 0 ? (own + at) * a.q_heads + h
                                            : piece.z + 256 * (piece.x + (shared >> twin)) + (shared & twin) * n + i;
                s[k] = a.stat[from];
                y[k] = *reinterpret_cast<const float4 *>(a.o + (long long)from * a.dim + d);
            }
            float top = m;
#pragma unroll
            for (int k = 0; k < B; ++k) top = fmaxf(top, s[k].x);
            const float ref = top == -INFINITY ? 0.f : top, f = pow2(m - ref);
            l *= f, x.x *= f, x.y *= f, x.z *= f, x.w *= f;
            m = top;
#pragma unroll
            for (int k = 0; k < B; ++k) {
                if (s[k].x == -INFINITY) continue;           // no token: its outputs may hold anything
                const float g = pow2(s[k].x - ref);
                l += s[k].y * g;
                x.x += y[k].x * g, x.y += y[k].y * g, x.z += y[k].z * g, x.w += y[k].w * g;
            }
        }
    }
    if constexpr (JG > 1) {
        s_m[t] = m, s_l[t] = l, s_o[t] = x;
        __syncthreads();
        if (!real || part0 != 0) return;
#pragma unroll
        for (int k = 1; k < JG; ++k) m = fmaxf(m, s_m[t + k * quads]);
        const float ref = m == -INFINITY ? 0.f : m, f = pow2(s_m[t] - ref);
        l *= f, x.x *= f, x.y *= f, x.z *= f, x.w *= f;
#pragma unroll
        for (int k = 1; k < JG; ++k) {
            const float g = pow2(s_m[t + k * quads] - ref);
            const float4 y = s_o[t + k * quads];
            l += s_l[t + k * quads] * g;
            x.x += y.x * g, x.y += y.y * g, x.z += y.z * g, x.w += y.w * g;
        }
    }
    if (!real) return;
    const float vs = a.v_scale ? a.v_scale[hk] : 1.f, div = l == 0.f ? 0.f : vs / l;
    __nv_bfloat16 *out = reinterpret_cast<__nv_bfloat16 *>(a.out) + r * a.out_stride + (long long)h * a.dim + d;
    *reinterpret_cast<uint2 *>(out) = make_uint2(pack_bf16(x.x * div, x.y * div), pack_bf16(x.z * div, x.w * div));
    if (a.lse && d == 0) a.lse[row] = (m + log2f(l)) * LN2;
}

}  // namespace

cudaError_t launch_check_groups(const AttendArgs &a, cudaStream_t st) {
    return launch_chained(check_groups_kernel, 1, 256, 0, st, a.start, a.shared_len, a.n_groups, a.n_req, a.kv.table_cols * a.kv.page_size, a.status);
}

cudaError_t launch_join(const JoinArgs &a, int parts, cudaStream_t st) {
    const auto run = [&](auto kernel, int groups) {
        const int per = JOIN_THREADS / (groups * (a.dim / 4));
        return launch_chained(kernel, (a.rows + per - 1) / per, JOIN_THREADS, 0, st, a);
    };
    return parts > 8 ? run(join_kernel<2, 8>, 2) : run(join_kernel<1, 4>, 1);
}

// The parts of a work row: as many as CTAs share it, of two streams; few with many groups.
int shared_parts(int n_groups, int kv_heads, int num_sms) { return 2 * (num_sms / (n_groups * kv_heads) + 1); }

cudaError_t launch_shared(const SharedArgs &a, int num_sms, cudaStream_t st) {
    const bool wide = a.kv.dim > 64;
    if (a.kv.dtype == KV_E4M3) return wide ? launch_shape<true, 128>(a, num_sms, st) : launch_shape<true, 64>(a, num_sms, st);
    return wide ? launch_shape<false, 128>(a, num_sms, st) : launch_shape<false, 64>(a, num_sms, st);
}

}  // namespace scute
