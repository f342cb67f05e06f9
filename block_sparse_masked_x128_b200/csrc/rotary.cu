// rotary.cu -- rotary positions of q and k, and their gradient.
//
// A pair (x1, x2) of the token at position t turns by a = t * f_i: y1 = c (x1 cos a - x2 sin a),
// y2 = c (x2 cos a + x1 sin a), rounded once; the gradient is the same with -a.  The angle is
// held in turns as a 64-bit fraction: F = f_i / 2 pi * 2^64 (from the frequency in 64-bit
// floating point) times the integer position, modulo 2^64, is the angle modulo one turn with no
// rounding but F's, so a position of a million is as exact as position one; cos and sin are then
// taken of a 32-bit fraction in [-1/2, 1/2) turns.
//
// Bound by HBM (2 bytes read and 2 written an element).  A CTA takes a few tokens of every
// head: their cos and sin are computed once into shared memory and serve all heads of q and k;
// a thread keeps one 16-byte column (half layout: the two columns of its pairs) and walks rows.
#include "serving.h"
#include "sm100_ptx.cuh"

#include <cuda_fp16.h>

namespace fa {
namespace {

constexpr int kRotThreads = 256;
constexpr int kRotTable = 2048;   // (token, pair) entries of cos and sin a CTA: 16 KiB

__device__ __forceinline__ float2 rotary_cos_sin(double freq, int64_t pos, float factor, bool inverse) {
    double turns = freq * 0.15915494309189533577;      // radians to turns
    turns -= floor(turns);
    const uint64_t fixed = (uint64_t)(turns * 18446744073709551616.0) * (uint64_t)pos;
    const float x = (float)(int32_t)(fixed >> 32) * 4.656612873077393e-10f;   // half turns, [-1, 1)
    float s, c;
    sincospif(x, &s, &c);
    return make_float2(c * factor, (inverse ? -s : s) * factor);
}

template <bool BF16>
__device__ __forceinline__ float2 rot_unpack(uint32_t w) {
    if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return make_float2(__half2float(__ushort_as_half((unsigned short)(w & 0xFFFFu))),
                       __half2float(__ushort_as_half((unsigned short)(w >> 16))));
}

template <bool BF16>
__device__ __forceinline__ uint16_t rot_round(float v) {
    return (uint16_t)(pack2<BF16>(v, 0.f) & 0xFFFFu);
}

// One pair of scalars: any number of pairs, any layout.
template <bool BF16, bool INTER>
__device__ __forceinline__ void rotate_pair(const uint16_t* x, uint16_t* y, int half, int i, float2 cs) {
    const int i1 = INTER ? 2 * i : i, i2 = INTER ? 2 * i + 1 : i + half;
    const float x1 = rot_unpack<BF16>(x[i1]).x, x2 = rot_unpack<BF16>(x[i2]).x;
    y[i1] = rot_round<BF16>(x1 * cs.x - x2 * cs.y);
    y[i2] = rot_round<BF16>(x2 * cs.x + x1 * cs.y);
}

template <bool BF16, bool INTER>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
    __shared__ float2 cs[kRotTable];
    const int64_t tokens = (int64_t)p.B * p.S;
    const int64_t t0 = (int64_t)blockIdx.x * p.tokens_per_cta;
    const int nt = (int)min((int64_t)p.tokens_per_cta, tokens - t0);
    const int heads = p.H[0] + p.H[1];
    // Heads of this CTA.
    const int h0 = (int)((int64_t)heads * blockIdx.y / gridDim.y), h1 = (int)((int64_t)heads * (blockIdx.y + 1) / gridDim.y);
    const int rot = 2 * p.half;
    for (int pair0 = 0; pair0 < p.half; pair0 += kRotTable) {      // one pass unless half > kRotTable
        const int np = min(kRotTable, p.half - pair0);
        for (int i = threadIdx.x; i < nt * np; i += kRotThreads) {
            const int t = i / np, j = i - t * np;
            const int64_t tok = t0 + t;
            const int64_t b = tok / p.S, s = tok - b * p.S;
            const int64_t pos = p.pos ? (int64_t)__ldg(p.pos + b * p.pos_stride + s) : p.pos0 + s;
            cs[i] = rotary_cos_sin(__ldg(p.freq + pair0 + j), pos, p.factor, p.inverse != 0);
        }
        __syncthreads();
        for (int64_t it = threadIdx.x; it < (int64_t)nt * (h1 - h0) * np; it += kRotThreads) {
            const int j = (int)(it % np);
            const int64_t row = it / np;
            const int h = h0 + (int)(row % (h1 - h0)), t = (int)(row / (h1 - h0));
            const int64_t tok = t0 + t, b = tok / p.S, s = tok - b * p.S;
            const int w = h >= p.H[0];
            const int hh = w ? h - p.H[0] : h;
            rotate_pair<BF16, INTER>(p.x[w] + b * p.xs[w][0] + hh * p.xs[w][1] + s * p.xs[w][2],
                                     p.y[w] + b * p.ys[w][0] + hh * p.ys[w][1] + s * p.ys[w][2], p.half, pair0 + j,
                                     cs[t * np + j]);
        }
        __syncthreads();
    }
    // The rest of each row is copied.
    if (!p.in_place && rot < p.D) {
        const int n = p.D - rot;
        for (int64_t it = threadIdx.x; it < (int64_t)nt * (h1 - h0) * n; it += kRotThreads) {
            const int j = (int)(it % n);
            const int64_t row = it / n;
            const int h = h0 + (int)(row % (h1 - h0)), t = (int)(row / (h1 - h0));
            const int64_t tok = t0 + t, b = tok / p.S, s = tok - b * p.S;
            const int w = h >= p.H[0];
            const int hh = w ? h - p.H[0] : h;
            p.y[w][b * p.ys[w][0] + hh * p.ys[w][1] + s * p.ys[w][2] + rot + j] =
                p.x[w][b * p.xs[w][0] + hh * p.xs[w][1] + s * p.xs[w][2] + rot + j];
        }
    }
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p0, bool bf16, bool interleaved, int nsm, cudaStream_t st) {
    RotaryParams p = p0;
    const int64_t tokens = (int64_t)p.B * p.S;
    int tt = p.half > 0 ? kRotTable / p.half : 16;
    tt = tt < 1 ? 1 : (tt > 16 ? 16 : tt);
    while (tt > 1 && (tokens + tt - 1) / tt < 4 * nsm) tt /= 2;
    p.tokens_per_cta = tt;
    const int64_t gx = (tokens + tt - 1) / tt;
    if (gx > 0x7fffffffLL) return cudaErrorInvalidValue;
    const int heads = p.H[0] + p.H[1];
    int gy = gx < nsm ? (int)((2 * nsm + gx - 1) / gx) : 1;
    gy = gy > heads ? heads : gy;
    const dim3 grid((unsigned)gx, (unsigned)gy);
    if (bf16 && interleaved) rotary_kernel<true, true><<<grid, kRotThreads, 0, st>>>(p);
    else if (bf16) rotary_kernel<true, false><<<grid, kRotThreads, 0, st>>>(p);
    else if (interleaved) rotary_kernel<false, true><<<grid, kRotThreads, 0, st>>>(p);
    else rotary_kernel<false, false><<<grid, kRotThreads, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace fa
