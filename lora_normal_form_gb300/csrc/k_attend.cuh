// Attention of one new token of each request over its paged cache:
//     out = sum_t p_t v_t,   p_t = exp(s_t - m) / sum_u exp(s_u - m),
// s_t the score of token t and m any number near the scores' maximum.  One pass:
// every warp keeps a reference m, the sum l of its weights and the unnormalised
// outputs o; two such triples join as m = max(m1, m2), l = l1 e^(m1 - m) + l2
// e^(m2 - m), o likewise.  Exponents are taken in powers of two.
//
// What bounds it: the cache, 2 x tokens x heads x dim elements read once, and for
// each byte 2 x group / element size operations (4 with 4 bf16 heads to a key, 32
// with 16 e4m3 ones).  Up to 8 heads to a key and 128 elements to a head that is
// memory, as measured here; beyond, and in fp32 from 4 heads on, the products, the
// conversions and the softmax of each (token, head).  On a GB300 whose copy rate is
// 6775 GB/s, 32 query heads on 8 key/value heads of 128 (device time of a graph's
// launch):
//     4 requests of 100003 to 131072 tokens, bf16   278 us, 6830 GB/s
//     64 requests of 200 to 8192 tokens, bf16        90 us, 6260 GB/s
//     64 of 500 to 16384, e4m3, 64 query heads      102 us, 5880 GB/s
//     256 requests of up to 1000 tokens, bf16        40 us, 3690 GB/s (the rows' ends)
//     1 request of 777 tokens                       9.7 us (the dependent steps: lengths
//         1.7, pages and cache rows 3.3, arrival 1.0, joining and storing 2.1)
//
// The work is one sequence of tiles (TT tokens of one request and head row),
// with ROW_COST places before each row's first for what a row costs beside its
// tiles, cut into equal contiguous ranges, one per CTA, whatever rows they fall
// in: any batch, one long request or many short ones, fills the GPU alike.  In a
// CTA one or two warps look the pages up and bring the tokens' key and value rows
// into a ring of stages by 16-byte asynchronous copies, running ahead over the
// ends of rows (a page may end anywhere in a tile); the others take the tiles in
// turn, each with its own triple, and join them in shared memory where a row
// ends.  Of a row that several CTAs share each leaves its triple in the workspace,
// arrives at the row's counter when its whole range is done, and the last to
// arrive joins them in the order of the CTAs, so that results do not depend on
// which that is.
//
// Instead of the copies, one bulk copy for each token row costs about 20 ns of
// its SM each (64 requests: 322 us), and cache rows loaded straight to registers
// leave the warps waiting (145 us).
#pragma once

#include <cuda_fp8.h>

#include "internal.h"
#include "ptx.cuh"

namespace scute {

namespace {

// What a request sees, a kernel for each: its tokens from first on (all, or a window's);
// a window's and the first few (sinks); those behind what its group shares (k_shared.cu;
// k_attend_own.cu alone).
enum { PLAIN, SINKS, SHARED };

constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;
constexpr int ATT_CTAS = 6;               // CTAs of an SM, at most
constexpr int QS = 2;                     // rows whose queries may be waiting
constexpr int MAX_STAGES = 32;
// What a row costs beside its tiles, in tiles: with 1, 256 short requests take
// 44.2 us and one request 12.2, with 3 40.2 and 9.7, with 6 42.2 and 9.6.
constexpr int ROW_COST = 3;
// The least places of a range, so that a small batch is not cut to parts whose
// joining costs more: one request takes 11.1 us with 2, 9.7 with 4, 11.9 with 8.
constexpr int MIN_TILES = 4;
constexpr uint64_t WAIT_NS = 2000000000ull;

// A whole warp's wait, ended by the warp's votes alone.  Lanes that poll each for
// itself see the barrier complete, the time pass and the CTA's abort at their own
// moments: one could be past the wait while another gave up, and neither would come
// to the other's next shuffle.  (Polled again, a completed barrier is still complete:
// it goes on only after this warp's own arrival or filling.)
__device__ __noinline__ bool wait_long(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    constexpr unsigned ALL_LANES = 0xffffffffu;
    const uint64_t t0 = ptx::globaltimer();
    for (;;) {
        if (__any_sync(ALL_LANES, *abort_flag != 0)) return false;
#pragma unroll 1
        for (int i = 0; i < 32; ++i)
            if (__all_sync(ALL_LANES, ptx::mbar_try_wait(bar, parity))) return true;
        if (__any_sync(ALL_LANES, ptx::globaltimer() - t0 > WAIT_NS)) {
            *abort_flag = 1;
            return false;
        }
    }
}
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, volatile int *abort_flag) {
    return __all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity)) || wait_long(bar, parity, abort_flag);
}
__device__ __forceinline__ uint4 lds16(uint32_t p) {
    uint4 r;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(p));
    return r;
}
__device__ __forceinline__ uint2 lds8(uint32_t p) {
    uint2 r;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(p));
    return r;
}
// 16 bytes from global to shared memory, or 16 zero bytes; of the cache's rows
// with an L2 policy (they are read once: what else a step keeps in L2, its code
// among it, shall stay there).
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool real, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(real ? 16 : 0), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}
// One of the barrier's arrivals, when this thread's copies so far have arrived.
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
template <int THREADS>
__device__ __forceinline__ void sync_threads() { asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory"); }
__device__ __forceinline__ float reduce_max(float x) {        // over the lanes of one column
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float reduce_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
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
// 2^x; results below the normal range are zero.
__device__ __forceinline__ float pow2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// Two e4m3 values, the low or the high 16 bits of a word, as two halves.
__device__ __forceinline__ uint32_t halves_lo(uint32_t x) {
    uint32_t y;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t halves_hi(uint32_t x) {
    uint32_t y;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(y) : "r"(x));
    return y;
}
// A capped score, in powers of two (kept out of the loop's code).
__device__ __noinline__ float capped(float x, float cap) { return cap * LOG2E * tanhf(x / cap); }
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

// A stage holds a tile's key rows, then its value rows (ROW bytes each).  The
// 16-byte pieces of a row are permuted within 128 bytes so that the lanes of a
// quarter warp read different banks, of the keys (rows 2i and 2i + 1, four
// neighbouring pieces of each) as of the values (rows 0, 2, 4, 6, two pieces of each).
template <int ROW>
__device__ __forceinline__ constexpr uint32_t turn_of(int row) {
    return ROW == 64 ? (row >> 1 & 3) << 5 : ((row & 1) << 6) ^ ((row >> 1 & 3) << 5);
}
template <int ROW>
__device__ __forceinline__ uint32_t place_of(int row, int piece) {
    return (row * ROW + piece * 16) ^ turn_of<ROW>(row);
}

// ---------------------------------------------------------------- 16- and 8-bit caches
// The products run on the warp-wide matrix instructions with the cache as the
// operand of 16 rows and the query heads as the one of 8 columns:
//     S^T [16 tokens x 8 heads] = K [16 x D] Q^T,
//     O^T [D x 8 heads] += V^T [D x 16 tokens] P^T,
// so a group of 4 or 8 query heads wastes little.  A product's inner index may
// be numbered in any way that both operands share, so lane (g, c) = (lane / 4,
// lane % 4) takes 16 consecutive bytes of token g's (and g + 8's) key and the
// query's fragment the same elements; and 16 consecutive bytes of the values of
// tokens 2c, 2c + 1, 2c + 8, 2c + 9, of which pairs of tokens are interleaved by
// byte permutes.  The work per byte is small up to 8 heads (8 products for each
// element of a key, 2 x 8 for one of a value, whose weights come in two parts: about
// a tenth of these instructions' rate at full memory bandwidth; the tensor pipe is
// 13 % busy), so the larger tiles of the asynchronous matrix unit, 128 rows of which
// one new token fills at most 16, would gain nothing here.  A tile's values are read
// from shared memory piece by piece, behind the weights: all of them at once beside
// the keys costs registers (64 requests 91.2 against 89.9 us, e4m3, its weights in
// one part then, 101.9 against 98.5).
//
// Weights.  l sums them in 32 bits.  The second product takes them in two parts of
// the cache's own width, a number rounded and what that left, each in a product of
// its own: 16 bits of a weight with bf16 parts, 22 with the e4m3 cache's halves (and
// down to 2^-24 beside weights up to 2^15).  One part would keep 8 and 11 bits.  It
// costs nothing where memory bounds (bf16) and little with e4m3: 64 requests 102.2
// us against 99.1, heads of 64 79.5 against 75.1, 16 heads to a key 105.5 against
// 98.7.  A third bf16 part brings the outputs no nearer to 64 bits, whose distance
// is then the products' accumulation (1e-6 of the output before its rounding).
template <bool FP8, int DC, int NT>
struct MmaMath {
    using IO = __nv_bfloat16;
    static constexpr int ESZ = FP8 ? 1 : 2, ROW = DC * ESZ;
    static constexpr int MT = ROW <= 128 ? 2 : 1;         // 16-token steps of a tile
    static constexpr int TT = 16 * MT, HC = 8 * NT;
    static constexpr int P_BYTES = 0;
    static constexpr int KE = FP8 ? 16 : 8;               // elements of 16 bytes
    static constexpr int NQ = NT;
    static constexpr int KP = DC / (4 * KE);              // key pieces of a lane, each four lanes wide
    static constexpr int VE = FP8 && DC > 64 ? 16 : 8;    // elements of a value piece, eight lanes wide
    static constexpr int VP = DC / (8 * VE);
    static constexpr int VW = VE * ESZ / 4;               // its words
    // How far below the largest score the reference is set, in powers of two.  16-bit
    // weights of an 8-bit cache end at 2^-24: set 2^7 below, with weights up to 2^15,
    // tokens count down to 2^-31 of the largest weight, of which a million are 2^-11.
    static constexpr float ABOVE = FP8 ? 7.f : 0.f;
    static constexpr int OT = VE / 2;                     // 16-row output tiles of a value piece

    const int lane, g, c;
    uint32_t qf[NT][KP][KE / 2];
    float mul[NT][2];             // product to score, per head of this lane's columns
    float o[NT][VP][OT][4], top[NT][2], sum[NT][2];

    __device__ __forceinline__ MmaMath(int l, uint32_t) : lane(l), g(l >> 2), c(l & 3) {}
    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            top[nt][0] = top[nt][1] = -INFINITY;
            sum[nt][0] = sum[nt][1] = 0.f;
#pragma unroll
            for (int j = 0; j < VP; ++j)
#pragma unroll
                for (int i = 0; i < OT; ++i) o[nt][j][i][0] = o[nt][j][i][1] = o[nt][j][i][2] = o[nt][j][i][3] = 0.f;
        }
    }
    // The row's queries, [nh][D] in shared memory: the fragments' elements are those
    // of the keys' pieces.
    static constexpr int QE = KE / 8;                     // 16-byte pieces of a query for each of a key
    __device__ __forceinline__ void queries(uint32_t qs, int nh, int D, float scale) {
        uint4 x[NT][KP][QE];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int p = 0; p < KP; ++p)
#pragma unroll
                for (int e = 0; e < QE; ++e) {
                    const int h = nt * 8 + g, d = (p * 4 + c) * KE + e * 8;
                    x[nt][p][e] = make_uint4(0, 0, 0, 0);
                    if (h < nh && d < D) x[nt][p][e] = lds16(qs + (h * D + d) * 2);
                }
        queries(x, scale);
    }
    // The same from memory, read ahead.
    __device__ __forceinline__ void read_queries(const IO *q, int nh, int D, uint4 (&x)[NT][KP][QE]) const {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int p = 0; p < KP; ++p)
#pragma unroll
                for (int e = 0; e < QE; ++e) {
                    const int h = nt * 8 + g, d = (p * 4 + c) * KE + e * 8;
                    x[nt][p][e] = make_uint4(0, 0, 0, 0);
                    if (h < nh && d < D) x[nt][p][e] = *reinterpret_cast<const uint4 *>(q + (long long)h * D + d);
                }
    }
    __device__ __forceinline__ void queries(const uint4 (&x)[NT][KP][QE], float scale) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int p = 0; p < KP; ++p)
#pragma unroll
                for (int e = 0; e < QE; ++e) {
                    qf[nt][p][e * 4 + 0] = x[nt][p][e].x;
                    qf[nt][p][e * 4 + 1] = x[nt][p][e].y;
                    qf[nt][p][e * 4 + 2] = x[nt][p][e].z;
                    qf[nt][p][e * 4 + 3] = x[nt][p][e].w;
                }
            float back = 1.f;
            if constexpr (FP8) {
                // 16-bit halves have 11 bits where bf16 has 8: scaled by a power of
                // two that takes the head's largest element below 2^8, every element
                // down to 2^-22 of it stays exact
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
            mul[nt][0] = __shfl_sync(0xffffffffu, back, (2 * c) * 4) * scale;
            mul[nt][1] = __shfl_sync(0xffffffffu, back, (2 * c + 1) * 4) * scale;
        }
    }
    // One tile: keys at kd, values at vd, bit i of ok whether token i counts;
    // release() when the stage is in registers.
    template <typename F>
    __device__ __forceinline__ void tile(uint32_t kd, uint32_t vd, unsigned ok, float softcap, F release) {
        // two chains of products, so that one seldom waits for the one before it
        constexpr int TWO = NT == 1;
        float sc[MT][NT][4] = {}, sd[MT][TWO ? NT : 1][4] = {};
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < KP; ++j) {
                const uint4 x = lds16(kd + place_of<ROW>(m * 16 + g, j * 4 + c));
                const uint4 y = lds16(kd + place_of<ROW>(m * 16 + g + 8, j * 4 + c));
                const uint32_t w0[4] = {x.x, x.y, x.z, x.w}, w1[4] = {y.x, y.y, y.z, y.w};
                if constexpr (FP8) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t a0 = halves_lo(w0[e]), a2 = halves_hi(w0[e]);
                        const uint32_t a1 = halves_lo(w1[e]), a3 = halves_hi(w1[e]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816<true>(TWO && (e & 1) ? sd[m][TWO ? nt : 0] : sc[m][nt], a0, a1, a2, a3, qf[nt][j][2 * e],
                                           qf[nt][j][2 * e + 1]);
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 2; ++e)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816<false>(TWO && (e & 1) ? sd[m][TWO ? nt : 0] : sc[m][nt], w0[2 * e], w1[2 * e], w0[2 * e + 1],
                                            w1[2 * e + 1], qf[nt][j][2 * e], qf[nt][j][2 * e + 1]);
                }
            }
        uint32_t vr[4][VW];
        auto values = [&](int m, int k, int j) {
            const int tok = m * 16 + 2 * c + (k & 1) + (k >> 1) * 8;
            uint32_t *to = vr[k];
            if constexpr (VW == 4) {
                const uint4 x = lds16(vd + place_of<ROW>(tok, j * 8 + g));
                to[0] = x.x, to[1] = x.y, to[2] = x.z, to[3] = x.w;
            } else {
                const uint2 x = lds8(vd + place_of<ROW>(tok, g >> 1) + (g & 1) * 8);
                to[0] = x.x, to[1] = x.y;
            }
        };
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int k = 0; k < 4; ++k) sc[m][nt][k] = (TWO ? sc[m][nt][k] + sd[m][TWO ? nt : 0][k] : sc[m][nt][k]) * mul[nt][k & 1];
        if (softcap > 0.f) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int k = 0; k < 4; ++k) sc[m][nt][k] = capped(sc[m][nt][k], softcap);
        }
        if (ok != (TT == 32 ? 0xffffffffu : 0xffffu)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (!(ok >> (m * 16 + (k >> 1) * 8 + g) & 1)) sc[m][nt][k] = -INFINITY;
        }
        // scores in powers of two; the reference of the weights moves only when a
        // score passes where it was set by more than 2^8, so that the outputs are
        // seldom scaled
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int k = 0; k < 4; ++k) mx[k & 1] = fmaxf(mx[k & 1], sc[m][nt][k]);
            if (__any_sync(0xffffffffu, mx[0] > top[nt][0] + (ABOVE + 8.f) || mx[1] > top[nt][1] + (ABOVE + 8.f))) {
                float al[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float x = fmaxf(reduce_max(mx[k]) - ABOVE, top[nt][k]);
                    al[k] = x == top[nt][k] ? 1.f : exp2f(top[nt][k] - x);
                    top[nt][k] = x;
                    sum[nt][k] *= al[k];
                }
#pragma unroll
                for (int j = 0; j < VP; ++j)
#pragma unroll
                    for (int k = 0; k < OT; ++k) {
                        o[nt][j][k][0] *= al[0];
                        o[nt][j][k][1] *= al[1];
                        o[nt][j][k][2] *= al[0];
                        o[nt][j][k][3] *= al[1];
                    }
            }
        }
        uint32_t pf[MT][NT][2][2];            // [tokens 0-7, 8-15][weights, what their rounding left]
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float ref[2] = {top[nt][0] == -INFINITY ? 0.f : top[nt][0], top[nt][1] == -INFINITY ? 0.f : top[nt][1]};
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float p[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    p[k] = pow2(sc[m][nt][k] - ref[k & 1]);
                    sum[nt][k & 1] += p[k];
                }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    if constexpr (FP8) {
                        // a half keeps 11 bits of a weight (and none below 2^-24), two 22
                        const uint32_t hi = pack_f16(p[2 * k], p[2 * k + 1]);
                        const float2 back = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                        pf[m][nt][k][0] = transpose8(hi);
                        pf[m][nt][k][1] = transpose8(pack_f16(p[2 * k] - back.x, p[2 * k + 1] - back.y));
                    } else {
                        // bf16 keeps 8 bits of a weight, two parts 16
                        const uint32_t hi = pack_bf16(p[2 * k], p[2 * k + 1]);
                        const float r0 = p[2 * k] - __uint_as_float(hi << 16);
                        const float r1 = p[2 * k + 1] - __uint_as_float(hi & 0xffff0000u);
                        pf[m][nt][k][0] = transpose8(hi);
                        pf[m][nt][k][1] = transpose8(pack_bf16(r0, r1));
                    }
                }
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < VP; ++j) {
#pragma unroll
                for (int k = 0; k < 4; ++k) values(m, k, j);
#pragma unroll
                for (int i = 0; i < VW; ++i) {
                    const uint32_t x0 = vr[0][i], x1 = vr[1][i], x2 = vr[2][i], x3 = vr[3][i];
                    if constexpr (FP8) {
                        const uint32_t y0 = __byte_perm(x0, x1, 0x5140), y1 = __byte_perm(x0, x1, 0x7362);
                        const uint32_t y2 = __byte_perm(x2, x3, 0x5140), y3 = __byte_perm(x2, x3, 0x7362);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const uint32_t ya = k ? y1 : y0, yb = k ? y3 : y2;
                            const uint32_t a0 = halves_lo(ya), a1 = halves_hi(ya);
                            const uint32_t a2 = halves_lo(yb), a3 = halves_hi(yb);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) {
                                mma16816<true>(o[nt][j][2 * i + k], a0, a1, a2, a3, pf[m][nt][0][0], pf[m][nt][1][0]);
                                mma16816<true>(o[nt][j][2 * i + k], a0, a1, a2, a3, pf[m][nt][0][1], pf[m][nt][1][1]);
                            }
                        }
                    } else {
                        const uint32_t a0 = __byte_perm(x0, x1, 0x5410), a1 = __byte_perm(x0, x1, 0x7632);
                        const uint32_t a2 = __byte_perm(x2, x3, 0x5410), a3 = __byte_perm(x2, x3, 0x7632);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma16816<false>(o[nt][j][i], a0, a1, a2, a3, pf[m][nt][0][0], pf[m][nt][1][0]);
                            mma16816<false>(o[nt][j][i], a0, a1, a2, a3, pf[m][nt][0][1], pf[m][nt][1][1]);
                        }
                    }
                }
            }
        release();
    }
    // The warp's maximum and sum of every head, to m and l.
    __device__ __forceinline__ void stats(float *m, float *l) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float x = reduce_sum(sum[nt][i]);
                if (x != x && top[nt][i] == -INFINITY) top[nt][i] = 0.f;      // no number: not an empty share
                if (g == 0) {
                    m[nt * 8 + 2 * c + i] = top[nt][i];
                    l[nt * 8 + 2 * c + i] = x;
                }
            }
    }
    // The warp's outputs, [HC] rows of `ld` floats, relative to the maxima `all`.
    __device__ __forceinline__ void outputs(float *to, int ld, const float (&all)[NT][2]) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float f[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) f[i] = all[nt][i] > -INFINITY ? exp2f(top[nt][i] - all[nt][i]) : 0.f;
            float *p0 = to + (nt * 8 + 2 * c) * ld, *p1 = p0 + ld;
#pragma unroll
            for (int j = 0; j < VP; ++j)
#pragma unroll
                for (int i = 0; i < OT; i += 2) {
                    const int d = (j * 8 + g) * VE + 2 * i;
                    *reinterpret_cast<float4 *>(p0 + d) = make_float4(o[nt][j][i][0] * f[0], o[nt][j][i][2] * f[0],
                                                                      o[nt][j][i + 1][0] * f[0], o[nt][j][i + 1][2] * f[0]);
                    *reinterpret_cast<float4 *>(p1 + d) = make_float4(o[nt][j][i][1] * f[1], o[nt][j][i][3] * f[1],
                                                                      o[nt][j][i + 1][1] * f[1], o[nt][j][i + 1][3] * f[1]);
                }
        }
    }
    // The outputs of the first nh heads as they are, relative to the warp's own maxima.
    __device__ __forceinline__ void part(float *to, int D, int nh) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int h = nt * 8 + 2 * c + k;
                if (h >= nh) continue;
#pragma unroll
                for (int j = 0; j < VP; ++j)
#pragma unroll
                    for (int i = 0; i < OT; i += 2) {
                        const int d = (j * 8 + g) * VE + 2 * i;
                        if (d < D)
                            *reinterpret_cast<float4 *>(to + (long long)h * D + d) =
                                make_float4(o[nt][j][i][k], o[nt][j][i][k + 2], o[nt][j][i + 1][k], o[nt][j][i + 1][k + 2]);
                    }
            }
    }
    // Merge the maxima of CW warps and write this warp's outputs.
    template <int CW>
    __device__ __forceinline__ void finish(const float *s_m, float *to, int ld) {
        float all[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                all[nt][i] = -INFINITY;
#pragma unroll
                for (int x = 0; x < CW; ++x) all[nt][i] = fmaxf(all[nt][i], s_m[x * HC + nt * 8 + 2 * c + i]);
            }
        outputs(to, ld, all);
    }
};

// ---------------------------------------------------------------- 32-bit caches
// Sums in 32 bits throughout, NH heads at a time, on fp32 FMAs (16-bit products
// would not keep 32 bits; three-part ones on the matrix instructions would, and are
// not tried).  With one to two heads a key bound by memory (64 requests of one head
// of 64: 111 us, 6470 GB/s), from eight on by the FMAs and the shared memory that
// feeds them (32 requests, 8 heads of 128: 213 us, 3410 GB/s; 16 heads read every key
// twice: 213 us, 1700 GB/s).  Scores: lane (g, c) multiplies every fourth 16-byte
// piece of token g's key, and the four lanes of a token add up.  Outputs: a lane owns
// DC / 32 neighbouring elements and takes the tile's tokens one after another, their
// weights from shared memory.
template <int DC, int NH>
struct FmaMath {
    using IO = float;
    static constexpr int ESZ = 4, ROW = DC * 4;
    static constexpr int TT = DC <= 64 ? 16 : 8, MT = TT / 8, HC = NH;
    static constexpr int P_BYTES = HC * TT * 4;
    static constexpr int KP = DC / 16;                    // key pieces of a lane
    static constexpr int E = DC / 32;                     // outputs of a lane

    const int lane, g, c;
    const uint32_t ps;            // this warp's weights, [HC][TT]
    uint32_t qs;
    int D;
    float mul, o[NH][E], top[NH], sum[NH];

    __device__ __forceinline__ FmaMath(int l, uint32_t weights) : lane(l), g(l >> 2), c(l & 3), ps(weights) {}
    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            top[h] = -INFINITY, sum[h] = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[h][e] = 0.f;
        }
    }
    __device__ __forceinline__ void queries(uint32_t q, int, int dim, float scale) { qs = q, D = dim, mul = scale; }
    template <typename F>
    __device__ __forceinline__ void tile(uint32_t kd, uint32_t vd, unsigned ok, float softcap, F release) {
        float s[MT][NH] = {};
#pragma unroll
        for (int j = 0; j < KP; ++j) {
            const int d = (j * 4 + c) * 4;
            float k[MT][4];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const uint4 x = lds16(kd + place_of<ROW>(m * 8 + g, j * 4 + c));
                k[m][0] = __uint_as_float(x.x), k[m][1] = __uint_as_float(x.y);
                k[m][2] = __uint_as_float(x.z), k[m][3] = __uint_as_float(x.w);
            }
            if (d < D)
#pragma unroll
                for (int h = 0; h < NH; ++h) {      // rows behind the last head are not read back
                    const uint4 x = lds16(qs + (h * D + d) * 4);
                    const float q[4] = {__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w)};
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[m][h] = fmaf(k[m][e], q[e], s[m][h]);
                }
        }
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            float mx = -INFINITY;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float x = s[m][h];
                x += __shfl_xor_sync(0xffffffffu, x, 1);
                x += __shfl_xor_sync(0xffffffffu, x, 2);
                x *= mul;
                if (softcap > 0.f) x = capped(x, softcap);
                if (!(ok >> (m * 8 + g) & 1)) x = -INFINITY;
                s[m][h] = x;
                mx = fmaxf(mx, x);
            }
            if (__any_sync(0xffffffffu, mx > top[h] + 8.f)) {
                const float x = fmaxf(reduce_max(mx), top[h]);
                const float al = x == top[h] ? 1.f : exp2f(top[h] - x);
                top[h] = x;
                sum[h] *= al;
#pragma unroll
                for (int e = 0; e < E; ++e) o[h][e] *= al;
            }
            const float ref = top[h] == -INFINITY ? 0.f : top[h];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const float p = exp2f(s[m][h] - ref);
                sum[h] += p;
                if (c == 0) asm volatile("st.shared.f32 [%0], %1;" ::"r"(ps + (h * TT + m * 8 + g) * 4), "f"(p) : "memory");
            }
        }
        __syncwarp();
        constexpr int B = 4;                 // tokens at a time
#pragma unroll
        for (int t0 = 0; t0 < TT; t0 += B) {
            float v[B][E];
#pragma unroll
            for (int i = 0; i < B; ++i) {
                if constexpr (E == 2) {
                    const uint2 x = lds8(vd + place_of<ROW>(t0 + i, lane >> 1) + (lane & 1) * 8);
                    v[i][0] = __uint_as_float(x.x), v[i][1] = __uint_as_float(x.y);
                } else {
#pragma unroll
                    for (int e = 0; e < E / 4; ++e) {
                        const uint4 x = lds16(vd + place_of<ROW>(t0 + i, lane * (E / 4) + e));
                        v[i][4 * e] = __uint_as_float(x.x), v[i][4 * e + 1] = __uint_as_float(x.y);
                        v[i][4 * e + 2] = __uint_as_float(x.z), v[i][4 * e + 3] = __uint_as_float(x.w);
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < NH; ++h) {
                const uint4 x = lds16(ps + (h * TT + t0) * 4);
                const float p[4] = {__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w)};
#pragma unroll
                for (int i = 0; i < B; ++i)
#pragma unroll
                    for (int e = 0; e < E; ++e) o[h][e] = fmaf(p[i], v[i][e], o[h][e]);
            }
        }
        release();
    }
    __device__ __forceinline__ void stats(float *m, float *l) {
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            const float x = reduce_sum(sum[h]);
            if (x != x && top[h] == -INFINITY) top[h] = 0.f;
            if (lane == 0) m[h] = top[h], l[h] = x;
        }
    }
    template <int CW>
    __device__ __forceinline__ void finish(const float *s_m, float *to, int ld) {
#pragma unroll
        for (int h = 0; h < NH; ++h) {
            float all = -INFINITY;
#pragma unroll
            for (int x = 0; x < CW; ++x) all = fmaxf(all, s_m[x * HC + h]);
            const float f = all > -INFINITY ? exp2f(top[h] - all) : 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) to[h * ld + lane * E + e] = o[h][e] * f;
        }
    }
};

// The batch's work list.  Row (request r, key/value head and head chunk) takes
// ROW_COST places and then one for each of its tiles, an empty request's row one
// tile all the same; places_at[r] = places of one row of each request before r.
//
// Which tokens a request sees.  A row's tiles run over positions first .. len - 1, each a
// token's.  Without tokens that stay visible before a window (sinks) position and token
// are one and first is the window's first token f.  With them, S = min(sinks, f) tokens in
// front, the window's positions are its tokens' from wa on, f rounded down to a tile, and
// those of the S tokens, rounded up to a tile, lie directly before wa; positions of tokens
// between S and f do not count.  So tiles begin where tiles of the whole context would, and
// lie in whole pages where those do, at the price of up to two tiles in part (200 requests
// of 30 to 5000 tokens, window 1000, 24 in front, e4m3, pages of 16: 72.8 us against 85.1
// with the S tokens directly before f).
struct Seen {
    int first, len;
    int wa, f, s;            // (with sinks)
};
template <int MODE>
__device__ __forceinline__ Seen seen_of(const AttendArgs &a, int r, int tt, bool *bad) {
    const int cap = a.kv.table_cols * a.kv.page_size;
    int n = a.kv_len[r];
    *bad = n < 0 || n > cap;
    n = n < 0 ? 0 : n > cap ? cap : n;
    Seen y = {0, n, 0, 0, 0};
    if constexpr (MODE == SHARED) {
        int tokens;
        y.first = shared_group(a, r, n, &tokens) >= 0 ? tokens : 0;
    } else {
        y.first = a.window > 0 ? max(0, n - a.window) : 0;
        if constexpr (MODE == SINKS) {
            y.f = y.first;
            y.s = min(a.sinks, y.f);
            y.wa = y.f - y.f % tt;
            y.first = max(0, y.wa - (y.s + tt - 1) / tt * tt);
        }
    }
    return y;
}
// The token at position i (-1: none that counts).
template <int MODE>
__device__ __forceinline__ int token_of(const Seen &y, int i) {
    if constexpr (MODE != SINKS) return i;
    const int token = i < y.wa ? i - y.first : i;
    return token < y.s || token >= y.f ? token : -1;
}
template <int MODE>
__device__ __forceinline__ void plan_places(const AttendArgs &a, int tt, int *places_at, int *warp_sum) {
    const int t = threadIdx.x, lane = t & 31, warp = t >> 5, n = a.n_req, threads = blockDim.x;
    const int per = (n + threads - 1) / threads, r0 = min(n, t * per), r1 = min(n, r0 + per);
    int mine = 0;
    bool any = false;
#pragma unroll 8
    for (int r = r0; r < r1; ++r) {
        bool bad;
        const Seen y = seen_of<MODE>(a, r, tt, &bad);
        any |= bad;
        mine += ROW_COST + max(1, (y.len - y.first + tt - 1) / tt);
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
    for (int w = 0; w < warp; ++w) at += warp_sum[w];
    for (int r = r0; r < r1; ++r) {
        bool bad;
        const Seen y = seen_of<MODE>(a, r, tt, &bad);
        places_at[r] = at;
        at += ROW_COST + max(1, (y.len - y.first + tt - 1) / tt);
    }
    if (t == threads - 1) places_at[n] = at;
    __syncthreads();
}

// x / y of numbers that mostly fit 32 bits (a 64-bit division is a long routine).
__device__ __forceinline__ long long quotient(long long x, long long y) {
    return ((x | y) >> 32) == 0 ? (long long)((unsigned)x / (unsigned)y) : x / y;
}

// Walks a CTA's range of places, row by row.
template <int MODE>
struct Walk {
    const AttendArgs &a;
    const int *places_at;
    int hz, Z, tt;
    long long total, end;
    int ctas;
    // the row: its first place, request, head and chunk, tiles; positions [first, len)
    long long base;
    int r, hk, z, tiles;
    Seen seen;
    int t0, t1;              // the range's tiles of it

    __device__ __forceinline__ Walk(const AttendArgs &args, const int *at, int heads_chunk, int tile, int min_tiles)
        : a(args), places_at(at), tt(tile) {
        Z = (a.group + heads_chunk - 1) / heads_chunk;
        hz = a.kv.heads * Z;
        total = (long long)at[a.n_req] * hz;
        ctas = (int)min((long long)gridDim.x, quotient(total + min_tiles - 1, min_tiles));
    }
    __device__ __forceinline__ long long start(int cta) const { return quotient(total * cta, ctas); }
    // The CTA whose range holds place x.
    __device__ __forceinline__ int owner(long long x) const { return (int)quotient((x + 1) * ctas - 1, total); }
    __device__ __forceinline__ int first_owner() const { return owner(base + ROW_COST); }
    __device__ __forceinline__ int last_owner() const { return owner(base + ROW_COST + tiles - 1); }
    __device__ __forceinline__ void request() {
        bool bad;
        seen = seen_of<MODE>(a, r, tt, &bad);
        tiles = places_at[r + 1] - places_at[r] - ROW_COST;
    }
    __device__ __forceinline__ void cut(long long from) {
        t0 = (int)max(0ll, from - base - ROW_COST);
        t1 = (int)min((long long)tiles, end - base - ROW_COST);
    }
    // At the first row of CTA cta's range that has tiles in it.
    __device__ __forceinline__ void open(int cta) {
        const long long x = start(cta);
        end = start(cta + 1);
        r = 0;
        for (int hi = a.n_req - 1; r < hi;) {
            const int mid = (r + hi + 1) >> 1;
            if ((long long)places_at[mid] * hz <= x) r = mid;
            else hi = mid - 1;
        }
        request();
        const long long in = x - (long long)places_at[r] * hz;
        const int row = (int)quotient(in, tiles + ROW_COST);
        base = (long long)places_at[r] * hz + (long long)row * (tiles + ROW_COST);
        hk = row / Z;
        z = row - hk * Z;
        cut(x);
    }
    // Whether there is a row left; next() goes on to the next one.
    __device__ __forceinline__ bool more() const { return base + ROW_COST < end; }
    __device__ __forceinline__ void next() {
        base += tiles + ROW_COST;
        if (++z == Z) {
            z = 0;
            if (++hk == a.kv.heads) {
                hk = 0;
                if (++r < a.n_req) request();
            }
        }
        cut(base);
    }
    __device__ __forceinline__ int from() const { return seen.first + t0 * tt; }
    __device__ __forceinline__ int to() const { return (int)min((long long)seen.len, seen.first + (long long)t1 * tt); }
    __device__ __forceinline__ bool whole() const { return t0 == 0 && t1 == tiles; }
};

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

// Four elements of the output of one head, times f.
template <typename IO>
__device__ __forceinline__ void put(const AttendArgs &a, int r, int h, int d, float4 x, float f) {
    IO *out = reinterpret_cast<IO *>(a.out) + r * a.out_stride + (long long)h * a.kv.dim + d;
    if constexpr (sizeof(IO) == 4) {
        *reinterpret_cast<float4 *>(out) = make_float4(x.x * f, x.y * f, x.z * f, x.w * f);
    } else {
        uint2 y;
        y.x = pack_bf16(x.x * f, x.y * f);
        y.y = pack_bf16(x.z * f, x.w * f);
        *reinterpret_cast<uint2 *>(out) = y;
    }
}

// A row that several CTAs share, as its joiner needs it.
struct SharedRow {
    int r, hk, h0, nh, c0, c1;          // request, heads; its first and last CTA
};
// Join the parts of up to two rows, as many parts at a time as `room` bytes of
// shared memory hold, brought there at once; those of both rows where they fit.
// How a row's parts are grouped depends on that row alone (its parts, heads and the
// room): which CTA is the last of a row, and whether it joins another one beside it,
// is a race, and a row joined in other groups has other bits.  A row whose parts fit
// is joined in one group, alone or beside another; one whose parts do not, in groups
// of as many as fit alone.
template <typename IO, int THREADS>
__device__ __forceinline__ void join_parts(const AttendArgs &a, const SharedRow &head, const SharedRow &tail, bool last_head,
                                           bool last_tail, uint8_t *buf, int room, int t) {
    constexpr int IT = 2;                // groups of four outputs of a thread at a time
    const int D = a.kv.dim;
    auto parts_of = [&](const SharedRow &row, bool last) { return last ? row.c1 - row.c0 + 1 : 0; };
    auto bytes_of = [&](const SharedRow &row) { return (2 * ATT_HEADS + row.nh * D) * 4; };      // of a part
    auto bring_row = [&](const SharedRow &row, int k0, int k1, uint32_t to) {      // a row's parts k0 .. k1
        const int bytes = bytes_of(row), pieces = bytes / 16;
        for (int e = t; e < pieces; e += THREADS) {
            const float *from = part_of(a, 2 * (row.c0 + k0)).m + e * 4;
            uint32_t at = to + e * 16;
#pragma unroll 4
            for (int k = k0; k < k1; ++k) {
                copy16(at, k ? from : from + PART_FLOATS);           // the first one's is its CTA's second slot
                at += bytes;
                from += 2 * PART_FLOATS;
            }
        }
    };
    const uint32_t room_at = ptx::smem_u32(buf);
    const int n_head = parts_of(head, last_head), n_tail = parts_of(tail, last_tail);
    const int head_bytes = n_head ? n_head * bytes_of(head) : 0, tail_bytes = n_tail ? n_tail * bytes_of(tail) : 0;
    const bool once = head_bytes + tail_bytes <= room;
    if (once) {
        sync_threads<THREADS>();
        if (n_head) bring_row(head, 0, n_head, room_at);
        if (n_tail) bring_row(tail, 0, n_tail, room_at + head_bytes);
        asm volatile("cp.async.wait_all;" ::: "memory");
        sync_threads<THREADS>();
    }
#pragma unroll 1
    for (int w = 0; w < 2; ++w) {
        if (!(w ? last_tail : last_head)) continue;
        const SharedRow &row = w ? tail : head;
        const int count = w ? n_tail : n_head, items = row.nh * (D / 4);
        const int bytes = bytes_of(row), ld = bytes / 4, cap = once ? count : room / bytes;
        const float vs = a.kv.v_scale ? a.kv.v_scale[row.hk] : 1.f;
#pragma unroll 1
        for (int g0 = 0; g0 < items; g0 += IT * THREADS) {
            float m[IT], l[IT];
            float4 x[IT];
#pragma unroll
            for (int i = 0; i < IT; ++i) m[i] = -INFINITY, l[i] = 0.f, x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
            for (int p0 = 0; p0 < count; p0 += cap) {
                const int p1 = min(p0 + cap, count);
                if (!once) {
                    sync_threads<THREADS>();
                    bring_row(row, p0, p1, room_at);
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    sync_threads<THREADS>();
                }
                const float *parts = reinterpret_cast<const float *>(buf + (once && w ? head_bytes : 0));
                // the groups side by side, so that their loads overlap (past the row's
                // end the last one's again)
                const int k1 = p1 - p0;
                const float *pm[IT];
                float top[IT];
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    const int e = min(g0 + t + i * THREADS, items - 1);
                    pm[i] = parts + e / (D / 4);
                    top[i] = m[i];
                }
#pragma unroll 4
                for (int k = 0; k < k1; ++k)
#pragma unroll
                    for (int i = 0; i < IT; ++i) top[i] = fmaxf(top[i], pm[i][k * ld]);
                float ref[IT];
                const float4 *py[IT];
#pragma unroll
                for (int i = 0; i < IT; ++i) {
                    ref[i] = top[i] == -INFINITY ? 0.f : top[i];
                    py[i] = reinterpret_cast<const float4 *>(parts + 2 * ATT_HEADS) + min(g0 + t + i * THREADS, items - 1);
                    const float f = pow2(m[i] - ref[i]);
                    l[i] *= f, x[i].x *= f, x[i].y *= f, x[i].z *= f, x[i].w *= f;
                    m[i] = top[i];
                }
#pragma unroll 4
                for (int k = 0; k < k1; ++k)
#pragma unroll
                    for (int i = 0; i < IT; ++i) {
                        const float g = pow2(pm[i][k * ld] - ref[i]);
                        const float4 y = py[i][k * (ld / 4)];
                        l[i] += pm[i][k * ld + ATT_HEADS] * g;
                        x[i].x += y.x * g, x[i].y += y.y * g, x[i].z += y.z * g, x[i].w += y.w * g;
                    }
            }
#pragma unroll
            for (int i = 0; i < IT; ++i) {
                const int e = g0 + t + i * THREADS;
                if (e >= items) break;
                const int h = e / (D / 4), d = 4 * (e - h * (D / 4));
                put<IO>(a, row.r, row.h0 + h, d, x[i], l[i] == 0.f ? 0.f : vs / l[i]);
                if (a.lse && d == 0) a.lse[(long long)row.r * a.q_heads + row.h0 + h] = (m[i] + log2f(l[i])) * LN2;
            }
        }
    }
}

// Sizes of one instance: CW warps of a CTA compute, PW fetch, CTAS of them share an SM.
template <typename M, int DC, int CW, int PW, int CTAS>
struct Shape {
    static constexpr int THREADS = 32 * (CW + PW);
    static constexpr int STAGE = 2 * M::TT * M::ROW;
    static constexpr int O_LD = DC + 4;                   // floats between heads
    static constexpr int O_BYTES = CW * M::HC * O_LD * 4, Q_BYTES = M::HC * DC * (int)sizeof(typename M::IO);
    static constexpr int FIXED = O_BYTES + QS * Q_BYTES + CW * M::P_BYTES + CW * M::HC * 8 + M::HC * 8 +
                                 (2 * MAX_STAGES + 2 * QS) * 8 + MAX_STAGES * 4 + 64;
    static_assert(CW * STAGE >= (2 * ATT_HEADS + M::HC * DC) * 4, "the ring holds a part");
    static_assert(STAGE % 128 == 0 && O_BYTES % 16 == 0 && Q_BYTES % 16 == 0 && M::P_BYTES % 16 == 0, "alignment");
    static size_t smem(int stages, int n_req) { return FIXED + (size_t)stages * STAGE + 4 * ((size_t)n_req + 1); }
};

template <typename M, int DC, int CW, int PW, int CTAS, int MODE>
__global__ void __launch_bounds__(32 * (CW + PW), CTAS) attend_kernel(const AttendArgs a, int stages) {
    using S = Shape<M, DC, CW, PW, CTAS>;
    using IO = typename M::IO;
    constexpr int TT = M::TT, HC = M::HC, ESZ = M::ESZ;
    constexpr unsigned ALL = TT == 32 ? 0xffffffffu : (1u << TT) - 1;

    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *const s_ring = smem;
    float *const s_o = reinterpret_cast<float *>(smem + (size_t)stages * S::STAGE);   // [CW][HC][O_LD]
    uint8_t *const s_q = reinterpret_cast<uint8_t *>(s_o) + S::O_BYTES;               // [QS][HC][D]
    uint8_t *const s_p = s_q + QS * S::Q_BYTES;                                       // [CW] weights of a tile
    float *const s_m = reinterpret_cast<float *>(s_p + CW * M::P_BYTES);              // [CW][HC]
    float *const s_l = s_m + CW * HC;                                                 // [CW][HC]
    float *const s_top = s_l + CW * HC, *const s_sum = s_top + HC;                    // [HC]
    uint64_t *const s_bar = reinterpret_cast<uint64_t *>(s_sum + HC);
    unsigned *const s_ok = reinterpret_cast<unsigned *>(s_bar + 2 * MAX_STAGES + 2 * QS);   // [stage] tokens that count
    int *const s_misc = reinterpret_cast<int *>(s_ok + MAX_STAGES);
    volatile int *const s_abort = s_misc, *const s_last = s_misc + 1;      // [2]
    int *const s_warp = s_misc + 3;
    int *const places_at = s_misc + 16;
    auto full = [&](int i) { return ptx::smem_u32(s_bar + i); };
    auto empty = [&](int i) { return ptx::smem_u32(s_bar + MAX_STAGES + i); };
    auto q_full = [&](int i) { return ptx::smem_u32(s_bar + 2 * MAX_STAGES + i); };
    auto q_empty = [&](int i) { return ptx::smem_u32(s_bar + 2 * MAX_STAGES + QS + i); };

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int D = a.kv.dim, row_bytes = D * ESZ;
    if (threadIdx.x == 0) {
        *s_abort = 0;
        for (int i = 0; i < stages; ++i) {
            ptx::mbar_init(full(i), 33);      // the copies of 32 lanes, and the count of tokens
            ptx::mbar_init(empty(i), 1 + a.hold);
        }
        for (int i = 0; i < QS; ++i) {
            ptx::mbar_init(q_full(i), 32);
            ptx::mbar_init(q_empty(i), CW);
        }
        ptx::fence_mbar_init();
    }
    // behind a head's elements every row of a stage stays zero
    if (row_bytes < M::ROW)
        for (int i = threadIdx.x; i < stages * S::STAGE / 16; i += S::THREADS)
            reinterpret_cast<uint4 *>(s_ring)[i] = make_uint4(0, 0, 0, 0);
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    plan_places<MODE>(a, TT, places_at, s_warp);
    Walk<MODE> w(a, places_at, HC, TT, MIN_TILES);
    const int cta = blockIdx.x;
    if (cta >= w.ctas) return;
    w.open(cta);

    if (warp < PW) {
        // ------------------------------------------------ the warp that fetches
        // Spans of up to 128 tokens; the pages of the next span are looked up
        // before this one's rows are sent for.
        constexpr int SPAN = 128;
        const uint64_t policy = ptx::make_policy_evict_first();
        // pages in which a tile of 32 tokens lies at once: one check and one base for
        // it (e4m3, pages of 32 or 256 tokens: 98.6 us against 102.9 by halves); in
        // others the check is lost (pages of 16: 111.8 us, by halves 107.7)
        const bool whole_tiles = TT <= 16 || a.kv.page_size % TT == 0;
        const long long tok_bytes = a.kv.token_stride * ESZ;
        int hk = w.hk, z = w.z, r = w.r, stop = w.to(), pos = w.from();
        Seen seen = w.seen;
        bool opens = true, more = w.more();
        auto look_up = [&](int of, const Seen &y, int from, int until, int *page) {
            const int32_t *table = a.kv.table + of * a.kv.table_stride;
#pragma unroll
            for (int k = 0; k < SPAN / 32; ++k) {
                const int i = from + k * 32 + lane, token = token_of<MODE>(y, i);
                page[k] = i < until && token >= 0 ? table[a.page_shift >= 0 ? token >> a.page_shift : token / a.kv.page_size] : -1;
            }
        };
        int page[SPAN / 32];
        if (more) look_up(r, seen, pos, stop, page);
        bool bad = false;
        int st = 0, turn = 0, qst = 0;          // the next stage, whose it is to fill, the next slot of queries
        unsigned ph = 1, qph = 1;
        // (a wait that ran out ends this warp's work; another warp's ends at this one's next wait)
        while (more) {
            const bool last = pos + SPAN >= stop;
            if (last) w.next();
            const int next_pos = last ? w.from() : pos + SPAN, next_stop = last ? w.to() : stop;
            int next_page[SPAN / 32];
            if (last) more = w.more();
            if (more) look_up(w.r, w.seen, next_pos, next_stop, next_page);
            if (opens && pos < stop) {
                if (warp == 0) {
                    if (!wait_bar(q_empty(qst), qph, s_abort)) break;
                    const int h0 = hk * a.group + z * HC, nh = min(HC, a.group - z * HC);
                    constexpr int QE = 16 / sizeof(IO);
                    const IO *q = reinterpret_cast<const IO *>(a.q) + r * a.q_stride + (long long)h0 * D;
                    for (int i = lane; i < nh * D / QE; i += 32)
                        copy16(ptx::smem_u32(s_q + qst * S::Q_BYTES) + i * 16, q + i * QE);
                    copies_arrive(q_full(qst));
                }
                if (++qst == QS) qst = 0, qph ^= 1;
            }
            const char *kb = reinterpret_cast<const char *>(a.kv.k) + hk * a.kv.head_stride * ESZ;
            const char *vb = reinterpret_cast<const char *>(a.kv.v) + hk * a.kv.head_stride * ESZ;
            bool gone = false;
#pragma unroll
            for (int k = 0; k < SPAN / 32; ++k) {
                if (pos + k * 32 >= stop || gone) break;
                const int i = pos + k * 32 + lane;
                long long place = -1;
                const int token = token_of<MODE>(seen, i);
                if (i < stop && token >= 0) {
                    if (page[k] < 0 || page[k] >= a.kv.n_pages) {
                        bad = true;
                    } else {
                        const int in = a.page_shift >= 0 ? token & (a.kv.page_size - 1) : token % a.kv.page_size;
                        place = ((long long)page[k] * a.kv.page_stride + (long long)in * a.kv.token_stride) * ESZ;
                    }
                }
                const unsigned all = __ballot_sync(0xffffffffu, place >= 0);
#pragma unroll
                for (int m = 0; m < 32 / TT; ++m) {
                    if (pos + k * 32 + m * TT >= stop) break;
                    if (turn == warp) {
                        if (!wait_bar(empty(st), ph, s_abort)) {
                            gone = true;
                            break;
                        }
                        const unsigned ok = all >> (m * TT) & ALL;
                        const uint32_t kd = ptx::smem_u32(s_ring + (size_t)st * S::STAGE), vd = kd + TT * M::ROW;
                        // lanes of a row, rows of an instruction, and its instructions where it is longer
                        constexpr int LR = M::ROW >= 512 ? 32 : M::ROW / 16, RI = 32 / LR, CS = M::ROW / 16 / LR;
                        const int row0 = lane / LR;
                        // rows of the tile that lie in one page step by the token's stride
                        auto one_page = [&](int f, int count) {        // tokens f .. of the 32
                            const long long place0 = __shfl_sync(0xffffffffu, place, f);
                            return place0 >= 0 && pos + k * 32 + f + count <= stop &&
                                   __all_sync(0xffffffffu, lane / count != f / count ||
                                                               place == place0 + (lane - f) * tok_bytes);
                        };
                        auto send = [&](int f, int n0, int n1) {
                            const long long from = __shfl_sync(0xffffffffu, place, f) + row0 * tok_bytes;
#pragma unroll
                            for (int cs = 0; cs < CS; ++cs) {
                                const int piece = cs * LR + lane % LR;
                                if (piece * 16 >= row_bytes) continue;           // zero for good
                                // row n * RI + row0 lies n * RI rows from row0's place, but for
                                // the permutation, whose bits of the two add up
                                const uint32_t lane_at = place_of<M::ROW>(row0, piece);
                                const char *ks = kb + from + piece * 16, *vs = vb + from + piece * 16;
#pragma unroll
                                for (int n = n0; n < n1; ++n) {
                                    const uint32_t to = n * RI * M::ROW + (lane_at ^ turn_of<M::ROW>(n * RI));
                                    copy16(kd + to, ks, policy);
                                    copy16(vd + to, vs, policy);
                                    ks += RI * tok_bytes;
                                    vs += RI * tok_bytes;
                                }
                            }
                        };
                        constexpr int SUB = TT < 16 ? TT : 16;
                        if (whole_tiles && one_page(m * TT, TT)) {
                            send(m * TT, 0, TT / RI);
                        } else {
#pragma unroll
                            for (int u = 0; u < TT / SUB; ++u) {
                                if ((TT > SUB || !whole_tiles) && one_page(m * TT + u * SUB, SUB)) {
                                    send(m * TT + u * SUB, u * SUB / RI, (u + 1) * SUB / RI);
                                    continue;
                                }
#pragma unroll 2
                                for (int n = u * SUB / RI; n < (u + 1) * SUB / RI; ++n) {
                                    const int row = n * RI + row0;
                                    const long long p = __shfl_sync(0xffffffffu, place, m * TT + row);
#pragma unroll
                                    for (int cs = 0; cs < CS; ++cs) {
                                        const int piece = cs * LR + lane % LR;
                                        if (piece * 16 >= row_bytes) continue;
                                        const uint32_t to = place_of<M::ROW>(row, piece);
                                        copy16(kd + to, p >= 0 ? kb + p + piece * 16 : kb, p >= 0, policy);
                                        copy16(vd + to, p >= 0 ? vb + p + piece * 16 : vb, p >= 0, policy);
                                    }
                                }
                            }
                        }
                        copies_arrive(full(st));
                        if (lane == 0) {
                            s_ok[st] = ok;
                            ptx::mbar_arrive(full(st));
                        }
                    }
                    if (++turn == PW) turn = 0;
                    if (++st == stages) st = 0, ph ^= 1;
                }
            }
            if (gone) break;
            opens = last;
            r = w.r, hk = w.hk, z = w.z, seen = w.seen;
            pos = next_pos;
            stop = next_stop;
#pragma unroll
            for (int k = 0; k < SPAN / 32; ++k) page[k] = next_page[k];
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(a.status, STATUS_PAGES);
        // nothing of this warp's may be on its way when the CTA ends
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (*s_abort && lane == 0) atomicOr(a.status, STATUS_TIMEOUT);
        return;
    }

    // ---------------------------------------------------- the warps that compute
    const int cw = warp - PW, t = threadIdx.x - 32 * PW;
    int st = cw, qst = 0;                   // this warp's next stage, the next row's queries
    unsigned ph = 0, qph = 0, seq = 0;      // tiles of the CTA so far
    bool live = true;                       // until a wait ran out: then no tile is there to be read
    // what the end joins: the rows that began before this range, and go on behind it
    SharedRow head = {-1}, tail = {-1};
    M math(lane, ptx::smem_u32(s_p + cw * M::P_BYTES));
    for (; w.more(); w.next()) {
        const int h0 = w.hk * a.group + w.z * HC, nh = min(HC, a.group - w.z * HC);
        const int tiles = w.to() > w.from() ? (w.to() - w.from() + TT - 1) / TT : 0;
        math.reset();
        if (tiles) {
            const float scale = (a.kv.k_scale ? a.kv.k_scale[w.hk] : 1.f) * a.scale;
            live = live && wait_bar(q_full(qst), qph, s_abort);
            if (live) math.queries(ptx::smem_u32(s_q + qst * S::Q_BYTES), nh, D, a.softcap > 0.f ? scale : scale * LOG2E);
            // tile n of the CTA is warp n mod CW's, and the ring a multiple of CW
            // long: a stage has one reader for good, which has seen every earlier
            // filling of it, so that the parity it waits for is never ambiguous
            for (unsigned n = seq + ((unsigned)(cw - (int)(seq % CW) + CW) % CW); live && n < seq + tiles; n += CW) {
                live = wait_bar(full(st), ph, s_abort);
                if (!live) break;
                const unsigned ok = *(volatile unsigned *)(s_ok + st);
                const uint32_t kd = ptx::smem_u32(s_ring + (size_t)st * S::STAGE);
                math.tile(kd, kd + TT * M::ROW, ok, a.softcap, [&] {
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(empty(st));
                });
                if ((st += CW) >= stages) st = cw, ph ^= 1;
            }
            seq += tiles;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(q_empty(qst));
            if (++qst == QS) qst = 0, qph ^= 1;
        }

        // the warps' shares of the row
        math.stats(s_m + cw * HC, s_l + cw * HC);
        sync_threads<CW * 32>();
        math.template finish<CW>(s_m, s_o + cw * HC * S::O_LD, S::O_LD);
        if (t < HC) {
            float m = -INFINITY, l = 0.f;
#pragma unroll
            for (int x = 0; x < CW; ++x) m = fmaxf(m, s_m[x * HC + t]);
            if (m > -INFINITY)
#pragma unroll
                for (int x = 0; x < CW; ++x) l += s_l[x * HC + t] * exp2f(s_m[x * HC + t] - m);
            s_top[t] = m;
            s_sum[t] = l;
        }
        sync_threads<CW * 32>();
        auto merged = [&](int h, int d) {
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int x = 0; x < CW; ++x) {
                const float4 v = *reinterpret_cast<const float4 *>(s_o + (x * HC + h) * S::O_LD + d);
                y.x += v.x, y.y += v.y, y.z += v.z, y.w += v.w;
            }
            return y;
        };
        if (w.whole()) {
            const float vs = a.kv.v_scale ? a.kv.v_scale[w.hk] : 1.f;
            for (int i = t; i < nh * (D / 4); i += CW * 32) {
                const int h = i / (D / 4), d = 4 * (i - h * (D / 4));
                put<IO>(a, w.r, h0 + h, d, merged(h, d), s_sum[h] == 0.f ? 0.f : vs / s_sum[h]);
            }
            if (a.lse && t < nh) a.lse[(long long)w.r * a.q_heads + h0 + t] = (s_top[t] + log2f(s_sum[t])) * LN2;
        } else {
            const PartView p = part_of(a, 2 * cta + (w.t0 == 0 ? 1 : 0));
            for (int i = t; i < nh * (D / 4); i += CW * 32) {
                const int h = i / (D / 4), d = 4 * (i - h * (D / 4));
                *reinterpret_cast<float4 *>(p.o + h * D + d) = merged(h, d);
            }
            if (t < nh) p.m[t] = s_top[t], p.l[t] = s_sum[t];
            (w.t0 == 0 ? tail : head) = SharedRow{w.r, w.hk, h0, nh, w.first_owner(), w.last_owner()};
        }
    }

    // a fetching warp may have ended before the wait that ran out
    if (!live && lane == 0) atomicOr(a.status, STATUS_TIMEOUT);
    // arrive at the shared rows; the last to arrive joins
    if (head.r < 0 && tail.r < 0) return;
    sync_threads<CW * 32>();
    if (t < 2) {
        const SharedRow &row = t ? tail : head;
        int last = 0;
        if (row.r >= 0) {
            __threadfence();          // the CTA's parts, which the barrier above has ordered before this
            last = atomicAdd(a.ctr + row.c0, 1) == row.c1 - row.c0;
            if (last) a.ctr[row.c0] = 0;
            __threadfence();
        }
        s_last[t] = last;
    }
    sync_threads<CW * 32>();
    const bool last_head = s_last[0], last_tail = s_last[1];
    if (last_head || last_tail)          // the ring is empty by now
        join_parts<IO, CW * 32>(a, head, tail, last_head, last_tail, s_ring, stages * S::STAGE, t);
}

template <typename M, int DC, int CW, int PW, int CTAS, int MODE>
cudaError_t launch_shape(const AttendArgs &a, int num_sms, cudaStream_t st) {
    using S = Shape<M, DC, CW, PW, CTAS>;
    static_assert(CTAS <= ATT_CTAS, "workspace");
    static std::atomic<unsigned long long> done{0};
    const auto kernel = attend_kernel<M, DC, CW, PW, CTAS, MODE>;
    const cudaError_t e = allow_max_dynamic_smem(kernel, done);
    if (e != cudaSuccess) return e;
    // as many CTAs on an SM as its registers allow; fewer where a large batch's
    // list leaves too little room for their rings
    int per_sm = CTAS;
    long long stages = 0;
    for (; per_sm >= 1; --per_sm) {
        stages = ((228 / per_sm - 1) * 1024 - (long long)S::smem(0, a.n_req)) / S::STAGE / CW * CW;
        if (stages >= CW) break;
    }
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    if (stages > MAX_STAGES) stages = MAX_STAGES / CW * CW;
    return launch_chained(kernel, num_sms * per_sm, S::THREADS, S::smem((int)stages, a.n_req), st, a, (int)stages);
}

// Shapes: (computing warps, fetching warps, CTAs of an SM), each the fastest of those
// measured.  Few warps in many small CTAs end their rows independently of each other;
// many heads or long ones take more registers or more products for each byte that is
// fetched.  Not all of them hold their values in the registers that their CTAs leave:
// per thread, bf16 spills 148 bytes in the shape of 16 heads of 128 and 76 in that of
// dim > 128, e4m3 256 and 112, and 48 with heads of 64.  Device times in us, 64
// requests of up to 8192 tokens (e4m3: to 16384) where not said:
//     group <= 8, dim <= 128   2,1,4: 90.5, 256 short requests 40.2; 4,2,2: 100.3, 59.5
//                              e4m3 2,1,4: 101.8, 4,2,2: 118.1
//       dim <= 64              bf16 2,1,4: 62.0, 2,1,5: 63.6
//                              e4m3 2,1,6: 79.6, 2,1,5: 82.1, 2,1,4: 90.0
//     group > 8: 16 heads at a time, each key fetched once: 76.4 (4,2,2); in eights
//       with the shape above 105.2; 16 with 2,1,4: 131.1 (e4m3 105.2, 109.8, 159.9;
//       40 heads on one key, in eights 55.7 and 58.0 in sixteens)
//       dim <= 64              2,1,4: 69.7, 4,2,2: 90.6 (e4m3 98.3, 129.9)
//     dim > 128                4,2,2: 72.0, 2,2,2: 80.1, 2,1,3: 101.5 (32 requests);
//                              e4m3, 4 heads 138.6, 144.8, 136.3
template <bool FP8, int MODE>
cudaError_t launch_mma(const AttendArgs &a, int num_sms, cudaStream_t st) {
    const int D = a.kv.dim;
    const bool wide = a.group > 8;
    if (D > 128) return launch_shape<MmaMath<FP8, 256, 1>, 256, 4, 2, 2, MODE>(a, num_sms, st);
    if (D > 64)
        return wide ? launch_shape<MmaMath<FP8, 128, 2>, 128, 4, 2, 2, MODE>(a, num_sms, st)
                    : launch_shape<MmaMath<FP8, 128, 1>, 128, 2, 1, 4, MODE>(a, num_sms, st);
    return wide ? launch_shape<MmaMath<FP8, 64, 2>, 64, 2, 1, 4, MODE>(a, num_sms, st)
                : launch_shape<MmaMath<FP8, 64, 1>, 64, 2, 1, FP8 ? 6 : 4, MODE>(a, num_sms, st);
}
// 32-bit caches, in the same way (group 4, 32 requests; 8 heads at a time spill 440
// bytes with dim > 128, 100 with dim <= 64):
//     dim <= 64   2,1,5: 133.6, 2,1,6: 149.1, 2,1,4: 145.4 (64 requests)
//     dim <= 128  2,1,4: 141.6, 4,2,2: 192.3
//     dim > 128   2,1,3: 220.2, 4,2,2: 235.9, 2,2,2: 285.9 (one head 141.3, 156.4, 149.9;
//                 eight, where the spills weigh, 495, 540, 435)
template <int DC, int CW, int PW, int CTAS, int MODE>
cudaError_t launch_fma(const AttendArgs &a, int num_sms, cudaStream_t st) {
    if (a.group == 1) return launch_shape<FmaMath<DC, 1>, DC, CW, PW, CTAS, MODE>(a, num_sms, st);
    if (a.group == 2) return launch_shape<FmaMath<DC, 2>, DC, CW, PW, CTAS, MODE>(a, num_sms, st);
    if (a.group <= 4) return launch_shape<FmaMath<DC, 4>, DC, CW, PW, CTAS, MODE>(a, num_sms, st);
    return launch_shape<FmaMath<DC, 8>, DC, CW, PW, CTAS, MODE>(a, num_sms, st);
}
template <int MODE>
cudaError_t launch_attend_mode(const AttendArgs &a, int num_sms, cudaStream_t st) {
    if (a.kv.dtype == KV_BF16) return launch_mma<false, MODE>(a, num_sms, st);
    if (a.kv.dtype == KV_E4M3) return launch_mma<true, MODE>(a, num_sms, st);
    if (a.kv.dim <= 64) return launch_fma<64, 2, 1, 5, MODE>(a, num_sms, st);
    if (a.kv.dim <= 128) return launch_fma<128, 2, 1, 4, MODE>(a, num_sms, st);
    return launch_fma<256, 2, 1, 3, MODE>(a, num_sms, st);
}

}  // namespace

}  // namespace scute
