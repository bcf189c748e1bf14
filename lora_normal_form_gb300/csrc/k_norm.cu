// The end of a sub-block and the beginning of the next in one pass:
//     h = residual + scale * gate * post(y),   out = pre(h).
#include "internal.h"

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

// Any d and alignment: one CTA per row, the row in shared memory in 32 bits.
template <typename T>
__global__ void __launch_bounds__(256) residual_norm_kernel(const NormArgs a) {
    extern __shared__ float row[];
    __shared__ float warp_sum[8];
    const long long r = blockIdx.x;
    const int d = a.d;
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

// The row in registers: a row's threads hold NV 16-byte vectors each.  WARP: a
// warp for a row and shuffles alone; otherwise a CTA for a row.
template <typename T, int NV, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : 1024) residual_norm_vec_kernel(const NormArgs a) {
    constexpr int VE = Vec<T>::N;
    __shared__ float red[2][32];
    const int d = a.d, nvec = d / VE;
    const int per_row = WARP ? 32 : blockDim.x, t = WARP ? threadIdx.x & 31 : threadIdx.x;
    const long long r = WARP ? (long long)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
    if (WARP && r >= a.n) return;
    int turn = 0;
    auto row_sum = [&](float x) -> float {
#pragma unroll
        for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (WARP) return x;
        // two buffers in turn: a warp can be one sum ahead of the slowest, not two
        if ((threadIdx.x & 31) == 0) red[turn][threadIdx.x >> 5] = x;
        __syncthreads();
        const int warps = blockDim.x >> 5;
        float s = (threadIdx.x & 31) < warps ? red[turn][threadIdx.x & 31] : 0.f;
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        turn ^= 1;
        return s;
    };
    float x[NV][VE];
    uint4 res[NV];             // as stored, until it is added
    const T *y = reinterpret_cast<const T *>(a.y) + r * a.y_stride;
    const T *rs = reinterpret_cast<const T *>(a.residual) + r * a.residual_stride;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int i = v * per_row + t;
        uint4 in = make_uint4(0, 0, 0, 0);
        res[v] = in;
        if (i < nvec) {
            in = *reinterpret_cast<const uint4 *>(y + i * VE);
            if (a.residual) res[v] = *reinterpret_cast<const uint4 *>(rs + i * VE);
        }
        Vec<T>::open(in, x[v]);
    }
    // (mean, 1 / deviation); the squares are summed after the mean is taken off
    auto stats = [&](float *mean, float *rstd) {
        float m = 0.f, q = 0.f;
        if (a.layer) {
#pragma unroll
            for (int v = 0; v < NV; ++v)
#pragma unroll
                for (int e = 0; e < VE; ++e) m += x[v][e];
            m = row_sum(m) / d;
        }
#pragma unroll
        for (int v = 0; v < NV; ++v)
            if (v * per_row + t < nvec)
#pragma unroll
                for (int e = 0; e < VE; ++e) q += (x[v][e] - m) * (x[v][e] - m);
        *mean = m;
        *rstd = rsqrtf(row_sum(q) / d + a.eps);
    };
    auto affine = [&](float *z, const float *w, const float *b, int at, float mean, float rstd) {
        float f[4];
#pragma unroll
        for (int e = 0; e < VE; e += 4) {
            if (w) Vec<float>::load(w + at + e, f);
            else f[0] = f[1] = f[2] = f[3] = 1.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) z[e + i] = (z[e + i] - mean) * rstd * f[i];
            if (b) {
                Vec<float>::load(b + at + e, f);
#pragma unroll
                for (int i = 0; i < 4; ++i) z[e + i] += f[i];
            }
        }
    };
    float mean = 0.f, rstd = 1.f;
    if (a.post_w) stats(&mean, &rstd);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int i = v * per_row + t;
        if (i >= nvec) continue;
        if (a.post_w) affine(x[v], a.post_w, a.post_b, i * VE, mean, rstd);
        if (a.gate_vec) {
            float f[4];
#pragma unroll
            for (int e = 0; e < VE; e += 4) {
                Vec<float>::load(a.gate_vec + i * VE + e, f);
#pragma unroll
                for (int k = 0; k < 4; ++k) x[v][e + k] *= f[k];
            }
        } else if (a.gate_rows) {
            float f[VE];
            Vec<T>::load(reinterpret_cast<const T *>(a.gate_rows) + r * a.gate_stride + i * VE, f);
#pragma unroll
            for (int e = 0; e < VE; ++e) x[v][e] *= f[e];
        }
        float old[VE];
        Vec<T>::open(res[v], old);
#pragma unroll
        for (int e = 0; e < VE; ++e) x[v][e] = fmaf(a.scale, x[v][e], old[e]);
        if (a.residual_out)
            Vec<T>::store(reinterpret_cast<T *>(a.residual_out) + r * a.residual_out_stride + i * VE, x[v]);
    }
    if (!a.out) return;
    stats(&mean, &rstd);
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int i = v * per_row + t;
        if (i >= nvec) continue;
        affine(x[v], a.pre_w, a.pre_b, i * VE, mean, rstd);
        Vec<T>::store(reinterpret_cast<T *>(a.out) + r * a.out_stride + i * VE, x[v]);
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

template <typename T>
cudaError_t launch(const NormArgs &a, int num_sms, cudaStream_t s) {
    constexpr int VE = Vec<T>::N;
    if (by_vectors<T>(a)) {
        const int nvec = a.d / VE;
        if (nvec <= 32) residual_norm_vec_kernel<T, 1, true><<<(a.n + 7) / 8, 256, 0, s>>>(a);
        else if (nvec <= 64) residual_norm_vec_kernel<T, 2, true><<<(a.n + 7) / 8, 256, 0, s>>>(a);
        else {
            auto threads = [&](int nv) { return ((nvec + nv - 1) / nv + 31) / 32 * 32; };
            const bool few = a.n <= num_sms;
            if (threads(1) <= (few ? 1024 : 256)) residual_norm_vec_kernel<T, 1, false><<<a.n, threads(1), 0, s>>>(a);
            else if (threads(2) <= (few ? 1024 : 512)) residual_norm_vec_kernel<T, 2, false><<<a.n, threads(2), 0, s>>>(a);
            else if (threads(4) <= 1024) residual_norm_vec_kernel<T, 4, false><<<a.n, threads(4), 0, s>>>(a);
            else if constexpr (VE == 4) residual_norm_vec_kernel<T, 8, false><<<a.n, threads(8), 0, s>>>(a);
        }
        return cudaGetLastError();
    }
    static std::atomic<unsigned long long> done{0};
    const size_t smem = sizeof(float) * a.d;
    if (smem > 40 * 1024) {
        const cudaError_t e = allow_max_dynamic_smem(residual_norm_kernel<T>, done);
        if (e != cudaSuccess) return e;
    }
    residual_norm_kernel<T><<<a.n, 256, smem, s>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_residual_norm(bool f32, const NormArgs &a, int num_sms, cudaStream_t st) {
    return f32 ? launch<float>(a, num_sms, st) : launch<__nv_bfloat16>(a, num_sms, st);
}

}  // namespace scute
