// Attention of one new token of each request over its paged cache.
#include <cuda_fp8.h>

#include "internal.h"

namespace scute {

namespace {

__device__ __forceinline__ float ld(const float *p) { return *p; }
__device__ __forceinline__ float ld(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ float ld(const __nv_fp8_e4m3 *p) { return (float)*p; }
__device__ __forceinline__ void st(float *p, float x) { *p = x; }
__device__ __forceinline__ void st(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

constexpr int AT_HEADS = 8, AT_TILE = 32;

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

}  // namespace

size_t attend_part_floats(int num_sms) { return (size_t)num_sms; }
int attend_ctrs(int num_sms) { return num_sms; }

cudaError_t launch_attend(const AttendArgs &a, int num_sms, cudaStream_t st) {
    (void)num_sms;
    const dim3 grid(a.n_req, a.kv.heads, (a.group + AT_HEADS - 1) / AT_HEADS);
    if (a.kv.dtype == KV_FP32) attend_kernel<float, float><<<grid, 128, 0, st>>>(a);
    else if (a.kv.dtype == KV_BF16) attend_kernel<__nv_bfloat16, __nv_bfloat16><<<grid, 128, 0, st>>>(a);
    else attend_kernel<__nv_bfloat16, __nv_fp8_e4m3><<<grid, 128, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace scute
