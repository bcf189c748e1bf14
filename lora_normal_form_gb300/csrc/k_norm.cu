// The end of a sub-block and the beginning of the next in one pass:
//     h = residual + scale * gate * post(y),   out = pre(h).
#include "internal.h"
#include "ptx.cuh"

namespace scute {

namespace {

__device__ __forceinline__ float ld(const float *p) { return *p; }
__device__ __forceinline__ float ld(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st(float *p, float x) { *p = x; }
__device__ __forceinline__ void st(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

__device__ __forceinline__ float cta_sum(float x, float *warp_sum) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = x;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) s += warp_sum[w];
    return s;
}

// (mean, 1 / deviation) of the row in shared memory; the squares are summed
// after the mean is taken off, so that they do not cancel.
__device__ __forceinline__ void row_stats(const float *row, int d, int layer, float eps, float *warp_sum, float *mean,
                                          float *rstd) {
    float m = 0.f;
    if (layer) {
        float s = 0.f;
        for (int i = threadIdx.x; i < d; i += blockDim.x) s += row[i];
        m = cta_sum(s, warp_sum) / d;
    }
    float q = 0.f;
    for (int i = threadIdx.x; i < d; i += blockDim.x) q += (row[i] - m) * (row[i] - m);
    *mean = m;
    *rstd = rsqrtf(cta_sum(q, warp_sum) / d + eps);
}

// Any d and alignment: one CTA per row, the row in shared memory in 32 bits.  What
// it costs: 8772 rows of 4096 take 180 us, with 16-byte vectors 47.
template <typename T>
__global__ void __launch_bounds__(256) residual_norm_kernel(const NormArgs a) {
    extern __shared__ float row[];
    __shared__ float warp_sum[8];
    const long long r = blockIdx.x;
    const int d = a.d;
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const T *y = reinterpret_cast<const T *>(a.y) + r * a.y_stride;
    for (int i = threadIdx.x; i < d; i += blockDim.x) row[i] = ld(y + i);
    float mean = 0.f, rstd = 1.f;
    if (a.post_w) row_stats(row, d, a.layer, a.eps, warp_sum, &mean, &rstd);
    for (int i = threadIdx.x; i < d; i += blockDim.x) {
        float x = row[i];
        if (a.post_w) x = (x - mean) * rstd * a.post_w[i] + (a.post_b ? a.post_b[i] : 0.f);
        if (a.gate_vec) x *= a.gate_vec[i];
        if (a.gate_rows) x *= ld(reinterpret_cast<const T *>(a.gate_rows) + r * a.gate_stride + i);
        x *= a.scale;
        if (a.residual) x += ld(reinterpret_cast<const T *>(a.residual) + r * a.residual_stride + i);
        row[i] = x;
        if (a.residual_out) st(reinterpret_cast<T *>(a.residual_out) + r * a.residual_out_stride + i, x);
    }
    if (!a.out) return;
    row_stats(row, d, a.layer, a.eps, warp_sum, &mean, &rstd);
    for (int i = threadIdx.x; i < d; i += blockDim.x) {
        float x = (row[i] - mean) * rstd;
        if (a.pre_w) x *= a.pre_w[i];
        if (a.pre_b) x += a.pre_b[i];
        st(reinterpret_cast<T *>(a.out) + r * a.out_stride + i, x);
    }
}

// Sixteen bytes of a row as 32-bit values, and back.
template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int N = 4;
    static __device__ __forceinline__ void open(const uint4 v, float *x) {
        x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y);
        x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ void load(const float *p, float *x) { open(*reinterpret_cast<const uint4 *>(p), x); }
    static __device__ __forceinline__ void store(float *p, const float *x) {
        *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void load(const __nv_bfloat16 *p, float *x) {
        open(*reinterpret_cast<const uint4 *>(p), x);
    }
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
};

// Four rows of d for each token (y, residual, h, out), so bound by memory: 8772 rows
// of 4096 with both norms, bf16, take 47.0 us, 6120 GB/s (90 % of the copy rate);
// 64 rows 2.8 us, of which a launch of nothing is 1.5.  The row stays in registers
// between the two norms, so that every element is read and written once.
//
// The row in registers: a row's threads hold NV 16-byte vectors each.  WARP: a
// warp for a row and shuffles alone; otherwise a CTA for a row.  The launch has
// as many CTAs as reside, and each fetches its next row or two before it is done
// with the one it has (rows that fill the registers: after).  FULL: with means taken
// off or biases.  HELD: a thread keeps its columns' factors from row to row, post_w,
// the gate and the scale as one; fetched anew for every row they are half of all
// that passes through L1.  Rows of more than 16384 elements do not fit the 64
// registers of 1024 threads (bf16, 4 vectors: 312 bytes of spills, 468 with means or
// biases; fp32, 8: 740 and 988): 1000 rows of 32768, bf16, reach 0.56 of the copy
// rate; nor do held factors and biases the 128 of 512 (64 bytes; 4000 layer norms of
// 8192 0.63).
template <typename T, int NV, bool WARP, bool FULL, bool HELD, int MOST>
__global__ void __launch_bounds__(MOST, MOST == 256 || (!HELD && MOST == 512) ? 2 : 1)
    residual_norm_vec_kernel(const NormArgs a) {
    constexpr int VE = Vec<T>::N;
    constexpr int AHEAD = HELD ? 2 : NV <= 2 ? 1 : 0;      // rows fetched ahead
    constexpr int BUF = AHEAD == 2 ? 2 : 1;
    __shared__ __align__(16) float red[2][32];
    const int d = a.d, nvec = d / VE;
    const int per_row = WARP ? 32 : blockDim.x, t = WARP ? threadIdx.x & 31 : threadIdx.x;
    const int step = WARP ? gridDim.x * 8 : gridDim.x;
    const float inv_d = 1.f / d;
    int turn = 0;
    if (HELD) {
        if (threadIdx.x < 64) red[threadIdx.x >> 5][threadIdx.x & 31] = 0.f;
        __syncthreads();
    }
    auto row_sum = [&](float x) -> float {
#pragma unroll
        for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (WARP) return x;
        // two buffers in turn: a warp can be one sum ahead of the slowest, not two
        if ((threadIdx.x & 31) == 0) red[turn][threadIdx.x >> 5] = x;
        __syncthreads();
        float s = 0.f;
        if (HELD) {           // the places of warps there are not stay zero
#pragma unroll
            for (int w = 0; w < MOST / 32; w += 4) {
                const float4 p = *reinterpret_cast<const float4 *>(red[turn] + w);
                s += (p.x + p.y) + (p.z + p.w);
            }
        } else {
            s = (threadIdx.x & 31) < (blockDim.x >> 5) ? red[turn][threadIdx.x & 31] : 0.f;
#pragma unroll
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        }
        turn ^= 1;
        return s;
    };
    // a vector's factors and terms: y's with the gate and the scale, and h's
    auto y_factors = [&](int at, float *cw, float *cb) {
        float f[4];
#pragma unroll
        for (int e = 0; e < VE; e += 4) {
#pragma unroll
            for (int k = 0; k < 4; ++k) f[k] = a.scale;
            if (a.gate_vec) {
                Vec<float>::load(a.gate_vec + at + e, f);
#pragma unroll
                for (int k = 0; k < 4; ++k) f[k] *= a.scale;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) cw[e + k] = f[k];
            if (FULL) {
                float g[4] = {0.f, 0.f, 0.f, 0.f};
                if (a.post_b) Vec<float>::load(a.post_b + at + e, g);
#pragma unroll
                for (int k = 0; k < 4; ++k) cb[e + k] = g[k] * f[k];
            }
            if (a.post_w) {
                Vec<float>::load(a.post_w + at + e, f);
#pragma unroll
                for (int k = 0; k < 4; ++k) cw[e + k] *= f[k];
            }
        }
    };
    auto h_factors = [&](int at, float *pw, float *pb) {
#pragma unroll
        for (int e = 0; e < VE; e += 4) {
#pragma unroll
            for (int k = 0; k < 4; ++k) pw[e + k] = 1.f;
            if (a.pre_w) Vec<float>::load(a.pre_w + at + e, pw + e);
            if (FULL) {
#pragma unroll
                for (int k = 0; k < 4; ++k) pb[e + k] = 0.f;
                if (a.pre_b) Vec<float>::load(a.pre_b + at + e, pb + e);
            }
        }
    };
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    constexpr int HV = HELD ? NV : 1, HF = HELD && FULL ? NV : 1;
    float cw[HV][VE], pw[HV][VE], cb[HF][VE], pb[HF][VE];
    if (HELD)
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (v * per_row + t < nvec) {
                y_factors((v * per_row + t) * VE, cw[v], cb[FULL ? v : 0]);
                h_factors((v * per_row + t) * VE, pw[v], pb[FULL ? v : 0]);
            }

    uint4 y_in[BUF][NV], r_in[BUF][NV];          // rows as stored
    auto fetch = [&](int b, long long r) {
        const T *y = reinterpret_cast<const T *>(a.y) + r * a.y_stride;
        const T *rs = reinterpret_cast<const T *>(a.residual) + r * a.residual_stride;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = v * per_row + t;
            y_in[b][v] = r_in[b][v] = make_uint4(0, 0, 0, 0);
            if (i < nvec) {
                y_in[b][v] = *reinterpret_cast<const uint4 *>(y + i * VE);
                if (a.residual) r_in[b][v] = *reinterpret_cast<const uint4 *>(rs + i * VE);
            }
        }
    };
    long long r = WARP ? (long long)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
    auto one_row = [&](int b) {
        float x[NV][VE];
        uint4 res[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            Vec<T>::open(y_in[b][v], x[v]);
            res[v] = r_in[b][v];
        }
        if (AHEAD && r + AHEAD * step < a.n) fetch(b, r + AHEAD * step);
        // (mean, 1 / deviation); the squares are summed after the mean is taken off
        auto stats = [&](float *mean, float *rstd) {
            float m = 0.f, q = 0.f;
            if (FULL && a.layer) {
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int e = 0; e < VE; ++e) m += x[v][e];
                m = row_sum(m) * inv_d;
            }
#pragma unroll
            for (int v = 0; v < NV; ++v)
                if (!FULL || v * per_row + t < nvec)
#pragma unroll
                    for (int e = 0; e < VE; ++e) {
                        const float z = FULL ? x[v][e] - m : x[v][e];
                        q = fmaf(z, z, q);
                    }
            *mean = m;
            *rstd = rsqrtf(row_sum(q) * inv_d + a.eps);
        };
        float mean = 0.f, rstd = 1.f;
        if (a.post_w) stats(&mean, &rstd);
        float mw[VE], mb[VE];                      // where they are not held
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int i = v * per_row + t;
            if (i >= nvec) continue;
            if (!HELD) y_factors(i * VE, mw, mb);
            const float *fw = HELD ? cw[HELD ? v : 0] : mw, *fb = HELD ? cb[HF > 1 ? v : 0] : mb;
            float old[VE], gate[VE];
            Vec<T>::open(res[v], old);
            if (a.gate_rows) {
                Vec<T>::load(reinterpret_cast<const T *>(a.gate_rows) + r * a.gate_stride + i * VE, gate);
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    float z = (FULL ? x[v][e] - mean : x[v][e]) * rstd * fw[e];
                    if (FULL) z += fb[e];
                    x[v][e] = fmaf(z, gate[e], old[e]);
                }
            } else {
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float z = (FULL ? x[v][e] - mean : x[v][e]) * rstd;
                    x[v][e] = fmaf(z, fw[e], FULL ? fb[e] + old[e] : old[e]);
                }
            }
            if (a.residual_out)
                Vec<T>::store(reinterpret_cast<T *>(a.residual_out) + r * a.residual_out_stride + i * VE, x[v]);
        }
        if (a.out) {
            stats(&mean, &rstd);
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const int i = v * per_row + t;
                if (i >= nvec) continue;
                if (!HELD) h_factors(i * VE, mw, mb);
                const float *fw = HELD ? pw[HELD ? v : 0] : mw, *fb = HELD ? pb[HF > 1 ? v : 0] : mb;
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    const float z = (FULL ? x[v][e] - mean : x[v][e]) * rstd;
                    x[v][e] = FULL ? fmaf(z, fw[e], fb[e]) : z * fw[e];
                }
                Vec<T>::store(reinterpret_cast<T *>(a.out) + r * a.out_stride + i * VE, x[v]);
            }
        }
        if (!AHEAD && r + step < a.n) fetch(b, r + step);
    };
    if (r < a.n) fetch(0, r);
    if (BUF == 2 && r + step < a.n) fetch(BUF - 1, r + step);
    while (r < a.n) {
        one_row(0);
        r += step;
        if (BUF == 2 && r < a.n) {
            one_row(BUF - 1);
            r += step;
        }
    }
}

// Whether every row of every operand can be read 16 bytes at a time.
template <typename T>
bool by_vectors(const NormArgs &a) {
    constexpr int VE = Vec<T>::N;
    if (a.d % VE) return false;
    uintptr_t p = 0;
    long long s = 0;
    const struct { const void *p; long long s; } rows[] = {{a.y, a.y_stride}, {a.residual, a.residual_stride},
        {a.residual_out, a.residual_out_stride}, {a.out, a.out_stride}, {a.gate_rows, a.gate_stride}};
    for (const auto &x : rows)
        if (x.p) p |= reinterpret_cast<uintptr_t>(x.p), s |= x.s % VE;
    for (const void *v : {a.post_w, a.post_b, a.pre_w, a.pre_b, a.gate_vec}) p |= reinterpret_cast<uintptr_t>(v);
    return (p & 15) == 0 && s == 0;
}

template <typename T, int NV, bool WARP, bool FULL, bool HELD, int MOST>
cudaError_t launch_one(const NormArgs &a, int threads, int num_sms, cudaStream_t s) {
    const auto kernel = residual_norm_vec_kernel<T, NV, WARP, FULL, HELD, MOST>;
    // CTAs that reside on an SM at once, by its registers (looked up once) and threads
    static const int regs = [&] {
        cudaFuncAttributes f;
        return cudaFuncGetAttributes(&f, kernel) == cudaSuccess ? (f.numRegs + 7) / 8 * 8 : 64;
    }();
    const int by_regs = 65536 / (regs * threads), by_threads = 2048 / threads;
    const int per_sm = by_regs < 1 ? 1 : by_regs < by_threads ? by_regs : by_threads;
    const long long rows = WARP ? (a.n + 7) / 8 : a.n, room = (long long)num_sms * per_sm;
    return launch_chained(kernel, (int)(rows < room ? rows : room), threads, 0, s, a);
}
template <typename T, int NV, bool WARP, bool HELD, int MOST>
cudaError_t launch_vec(const NormArgs &a, int threads, int num_sms, cudaStream_t s) {
    if (a.layer || a.post_b || a.pre_b) return launch_one<T, NV, WARP, true, HELD, MOST>(a, threads, num_sms, s);
    return launch_one<T, NV, WARP, false, HELD, MOST>(a, threads, num_sms, s);
}

template <typename T>
cudaError_t launch(const NormArgs &a, int num_sms, cudaStream_t s) {
    constexpr int VE = Vec<T>::N;
    if (by_vectors<T>(a)) {
        const int nvec = a.d / VE;
        auto threads = [&](int nv) { return ((nvec + nv - 1) / nv + 31) / 32 * 32; };
        // Short rows: a warp for each (16384 rows of 256, bf16: 5.5 us, a CTA each 6.3;
        // of 512 the other way, 13.8 and 12.9).  A thread's factors are worth holding
        // where it has a few rows (600 rows of 4096 with both norms 4.3 us, not held 4.5;
        // 8772 rows 47.2 and 48.7), with more threads, so fewer CTAs, where it has many
        // (4000 rows of 8192 with biases 61.4 and 76.4, but 600 fp32 rows of 4096 6.7 and
        // 6.3).  Few rows: one vector to a thread (64 rows of 4096 2.8 us, two 3.1), up to
        // 512 threads (64 rows of 8192: 3.7 with two, 4.0 with one and 1024).  Longer
        // rows: two vectors and 1024 threads before four and 512 (2400 rows of 14336 53.1
        // and 70.8 us).
        const bool few = a.n <= num_sms, some = a.n >= 2 * num_sms, many = a.n >= 8 * num_sms;
        if (nvec <= 32) return launch_vec<T, 1, true, false, 256>(a, 256, num_sms, s);
        if (some && threads(1) <= 256) return launch_vec<T, 1, false, true, 256>(a, threads(1), num_sms, s);
        if (some && threads(2) <= 256) return launch_vec<T, 2, false, true, 256>(a, threads(2), num_sms, s);
        if (many && threads(2) <= 512) return launch_vec<T, 2, false, true, 512>(a, threads(2), num_sms, s);
        if (threads(1) <= (few ? 512 : 256)) return launch_vec<T, 1, false, false, 512>(a, threads(1), num_sms, s);
        if (threads(2) <= 512) return launch_vec<T, 2, false, false, 512>(a, threads(2), num_sms, s);
        if (threads(2) <= 1024) return launch_vec<T, 2, false, false, 1024>(a, threads(2), num_sms, s);
        if (threads(4) <= 1024) return launch_vec<T, 4, false, false, 1024>(a, threads(4), num_sms, s);
        if constexpr (VE == 4) return launch_vec<T, 8, false, false, 1024>(a, threads(8), num_sms, s);
    }
    static std::atomic<unsigned long long> done{0};
    const size_t smem = sizeof(float) * a.d;
    if (smem > 40 * 1024) {
        const cudaError_t e = allow_max_dynamic_smem(residual_norm_kernel<T>, done);
        if (e != cudaSuccess) return e;
    }
    return launch_chained(residual_norm_kernel<T>, a.n, 256, smem, s, a);
}

}  // namespace

cudaError_t launch_residual_norm(bool f32, const NormArgs &a, int num_sms, cudaStream_t st) {
    return f32 ? launch<float>(a, num_sms, st) : launch<__nv_bfloat16>(a, num_sms, st);
}

}  // namespace scute
