// decode_cache.cu -- attention of one new token a sequence over a paged, possibly quantised
// cache with grouped heads.
//
//   x_j = mod(scale * q . k_j),  p = softmax of x over max(0, len - window) <= j < len,
//   out = sum_j p_j v_j,  lse = log sum_j exp x_j        (no key: out 0, lse -inf)
//
// The lengths are device data, so a captured step serves every length the page table covers.
// One CTA a (sequence, query head): warps share the keys out, each lane holds D / 32 dims, and
// the warps' (m, l, O) are joined in shared memory.
#include "serving.h"
#include "sm100_ptx.cuh"

#include <cuda_fp16.h>

namespace fa {
namespace {

__device__ int32_t g_cache_decode_status;   // 2: a length or page out of range was met

constexpr int kCdThreads = 256, kCdWarps = kCdThreads / 32;
constexpr float kCdLn2 = 0.6931471805599453f, kCdLog2e = 1.4426950408889634f;

template <int DT>
__device__ __forceinline__ float cached_value(const void* base, int64_t i) {
    if constexpr (DT == FA_DTYPE_S8) return (float)static_cast<const int8_t*>(base)[i];
    if constexpr (DT == FA_DTYPE_E4M3) {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)static_cast<const uint8_t*>(base)[i]));
        return __half2float(__ushort_as_half((unsigned short)(h & 0xFFFFu)));
    }
    const uint16_t r = static_cast<const uint16_t*>(base)[i];
    return DT == FA_DTYPE_BF16 ? __uint_as_float((uint32_t)r << 16) : __half2float(__ushort_as_half(r));
}

template <int DT, int D>
__global__ void __launch_bounds__(kCdThreads) cache_decode_simple(const __grid_constant__ CacheDecodeParams p, bool q_bf16) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.x / p.HQ, hq = blockIdx.x % p.HQ, h = hq / p.group;
    int64_t len = __ldg(p.kv_lens + b);
    const int64_t cap = (int64_t)p.c.table_width << p.c.page_shift;
    if (len < 0 || len > cap) {
        if (threadIdx.x == 0) atomicExch(&g_cache_decode_status, 2);
        len = len < 0 ? 0 : cap;
    }
    const int64_t lo = p.window > 0 && len > p.window ? len - p.window : 0;
    float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const uint16_t r = p.q[b * p.q_stride[0] + hq * p.q_stride[1] + lane * E + e];
        q[e] = q_bf16 ? __uint_as_float((uint32_t)r << 16) : __half2float(__ushort_as_half(r));
        o[e] = 0.f;
    }
    float slope = 0.f;
    if (p.score_kind & FA_SCORE_ALIBI)
        slope = kCdLog2e * (p.alibi_slopes ? p.alibi_slopes[hq] : exp2f(-8.f * (hq + 1) / p.HQ));
    for (int64_t j = lo + warp; j < len; j += kCdWarps) {
        const int page = cache_page(p.c, b, j >> p.c.page_shift);
        if (page < 0) {
            if (lane == 0) atomicExch(&g_cache_decode_status, 2);
            continue;
        }
        const int64_t row = j & ((1 << p.c.page_shift) - 1);
        const int64_t at = page * p.c.stride[0] + h * p.c.stride[1] + row * p.c.stride[2] + lane * E;
        const int64_t sat = page * p.c.scale_stride[0] + h * p.c.scale_stride[1] + row * p.c.scale_stride[2];
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) s = fmaf(q[e], cached_value<DT>(p.c.k, at + e), s);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(kFullMask, s, off);
        if constexpr (CacheType<DT>::k8) s *= p.c.k_scale[sat];
        float x = s * p.scale_log2;
        // cap tanh(y) = cap (1 - 2 / (e^2y + 1)); softcap_k takes s to 2 y log2 e.
        if (p.score_kind & FA_SCORE_SOFTCAP) x = p.softcap_log2 * (1.f - 2.f / (exp2f(s * p.softcap_k) + 1.f));
        if (p.score_kind & FA_SCORE_ALIBI) x = fmaf(slope, (float)(j - (len - 1)), x);
        const float mn = fmaxf(m, x);
        const float a = m == mn ? 1.f : exp2f(m - mn), pr = mn == -INFINITY ? 0.f : exp2f(x - mn);
        m = mn;
        l = l * a + pr;
        const float w = CacheType<DT>::k8 ? pr * p.c.v_scale[sat] : pr;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * a + w * cached_value<DT>(p.c.v, at + e);
    }
    __shared__ float sm[kCdWarps], sl[kCdWarps], so[kCdWarps][D];
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = o[e];
    if (lane == 0) sm[warp] = m, sl[warp] = l;
    __syncthreads();
    float M = -INFINITY, L = 0.f;
    for (int w = 0; w < kCdWarps; ++w) M = fmaxf(M, sm[w]);
    for (int w = 0; w < kCdWarps; ++w) L += sm[w] == -INFINITY ? 0.f : sl[w] * exp2f(sm[w] - M);
    for (int d = threadIdx.x; d < D; d += kCdThreads) {
        float O = 0.f;
        for (int w = 0; w < kCdWarps; ++w) O += sm[w] == -INFINITY ? 0.f : so[w][d] * exp2f(sm[w] - M);
        const float v = L == 0.f ? 0.f : O / L;
        p.out[b * p.out_stride[0] + hq * p.out_stride[1] + d] =
            (uint16_t)((q_bf16 ? pack2<true>(v, 0.f) : pack2<false>(v, 0.f)) & 0xFFFFu);
    }
    if (threadIdx.x == 0 && p.lse) p.lse[(int64_t)b * p.HQ + hq] = L == 0.f ? -INFINITY : (M + log2f(L)) * kCdLn2;
}

}  // namespace

int64_t cache_decode_workspace_bytes(int B, int HQ, int HK, int D, int nsm) { return 16; }

cudaError_t launch_cache_decode(const CacheDecodeParams& p, int dtype, int D, bool q_bf16, int nsm, cudaStream_t st) {
#define FA_CD(T, DD)                                                                         \
    if (dtype == T && D == DD) {                                                             \
        cache_decode_simple<T, DD><<<(unsigned)(p.B * p.HQ), kCdThreads, 0, st>>>(p, q_bf16); \
        return cudaGetLastError();                                                           \
    }
    FA_CD(FA_DTYPE_F16, 64) FA_CD(FA_DTYPE_F16, 128) FA_CD(FA_DTYPE_BF16, 64) FA_CD(FA_DTYPE_BF16, 128)
    FA_CD(FA_DTYPE_E4M3, 64) FA_CD(FA_DTYPE_E4M3, 128) FA_CD(FA_DTYPE_S8, 64) FA_CD(FA_DTYPE_S8, 128)
#undef FA_CD
    return cudaErrorInvalidValue;
}

cudaError_t cache_decode_status(cudaStream_t st, int32_t* out) {
    void* addr = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&addr, g_cache_decode_status);
    if (e != cudaSuccess) return e;
    e = cudaMemcpyAsync(out, addr, 4, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    if (e == cudaSuccess && *out != 0) {
        e = cudaMemsetAsync(addr, 0, 4, st);
        if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    }
    return e;
}

}  // namespace fa
