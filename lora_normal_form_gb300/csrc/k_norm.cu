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

// One CTA per row, the row in shared memory in 32 bits.
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

template <typename T>
cudaError_t launch(const NormArgs &a, cudaStream_t s) {
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
    (void)num_sms;
    return f32 ? launch<float>(a, st) : launch<__nv_bfloat16>(a, st);
}

}  // namespace scute
