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
// head: their cos and sin are computed once into shared memory and serve all heads of q and k.
// Work goes in columns of 16 bytes (half layout: the two columns of eight pairs): a thread keeps
// its column and walks the rows (token, head), with the loads of kAhead rows in flight.  Pairs that
// do not fill such columns (half layout with rot_dim no multiple of 16) go one by one.
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

template <bool BF16>
__device__ __forceinline__ void rot_unpack8(const uint4& r, float (&f)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = rot_unpack<BF16>(w[i]);
        f[2 * i] = v.x;
        f[2 * i + 1] = v.y;
    }
}

// A token's offset in the inputs and outputs, and the row of one of its heads (q's, then k's).
struct RotToken {
    int64_t x[2], y[2];
};
struct RotRow {
    const uint16_t* x;
    uint16_t* y;
};
__device__ __forceinline__ RotToken rot_token(const RotaryParams& p, int64_t tok) {
    const int b = (int)tok / p.S, s = (int)tok - b * p.S;       // fewer than 2^31 tokens
    return {{b * p.xs[0][0] + s * p.xs[0][2], b * p.xs[1][0] + s * p.xs[1][2]},
            {b * p.ys[0][0] + s * p.ys[0][2], b * p.ys[1][0] + s * p.ys[1][2]}};
}
__device__ __forceinline__ RotRow rot_row(const RotaryParams& p, const RotToken& t, int head) {
    if (head < p.H[0]) return {p.x[0] + t.x[0] + head * p.xs[0][1], p.y[0] + t.y[0] + head * p.ys[0][1]};
    const int h = head - p.H[0];
    return {p.x[1] + t.x[1] + h * p.xs[1][1], p.y[1] + t.y[1] + h * p.ys[1][1]};
}

// cos and sin (times the factor) of pairs pair0 .. pair0 + np - 1 of tokens t0 .. t0 + nt - 1.
__device__ __forceinline__ void rot_table(const RotaryParams& p, float2* cs, int64_t t0, int nt, int pair0, int np) {
    for (int i = threadIdx.x; i < nt * np; i += kRotThreads) {
        const int t = i / np, j = i - t * np;
        const int tok = (int)(t0 + t), b = tok / p.S, s = tok - b * p.S;
        const int64_t pos = p.pos ? (int64_t)__ldg(p.pos + b * p.pos_stride + s) : p.pos0 + s;
        cs[i] = rotary_cos_sin(__ldg(p.freq + pair0 + j), pos, p.factor, p.inverse != 0);
    }
}

// By columns: half layout with rot_dim a multiple of 16, or interleaved with any rot_dim.
template <bool BF16, bool INTER>
__global__ void __launch_bounds__(kRotThreads) rotary_columns_kernel(const __grid_constant__ RotaryParams p) {
    __shared__ float2 cs[kRotTable];
    constexpr int kAhead = INTER ? 4 : 2;          // rows whose 16-byte loads are in flight at once
    grid_dependency_wait();
    const int64_t t0 = (int64_t)blockIdx.x * p.tokens_per_cta;
    const int nt = (int)min((int64_t)p.tokens_per_cta, (int64_t)p.B * p.S - t0);
    const int heads = p.H[0] + p.H[1];
    const int h0 = (int)((int64_t)heads * blockIdx.y / gridDim.y), h1 = (int)((int64_t)heads * (blockIdx.y + 1) / gridDim.y);
    // The columns of a row: rotated ones (half layout: pairs of columns), then copied ones.
    const int rot_cols = INTER ? (p.half + 3) / 4 : p.half / 8;
    const int copied0 = INTER ? rot_cols * 8 : 2 * p.half;
    const int cols = rot_cols + (p.in_place ? 0 : (p.D - copied0) / 8);
    const int col = threadIdx.x % cols, first = threadIdx.x / cols, stride = kRotThreads / cols;   // D <= 1024: cols <= 128
    rot_table(p, cs, t0, nt, 0, p.half);
    __syncthreads();
    if (first >= stride) return;
    const bool turns = col < rot_cols;
    const int at = turns ? col * 8 : copied0 + (col - rot_cols) * 8;
    for (int t = 0; t < nt; ++t) {
        const RotToken tok = rot_token(p, t0 + t);
        float c[8], s[8];                       // of this column's pairs (interleaved: four)
        if (turns) {
#pragma unroll
            for (int i = 0; i < (INTER ? 4 : 8); ++i) {
                const int pair = INTER ? col * 4 + i : col * 8 + i;
                const float2 v = pair < p.half ? cs[t * p.half + pair] : make_float2(1.f, 0.f);
                c[i] = v.x;
                s[i] = v.y;
            }
        }
        for (int hb = h0 + first; hb < h1; hb += stride * kAhead) {
            uint4 a[kAhead], b[kAhead];
            RotRow row[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int h = hb + k * stride;
                if (h >= h1) continue;
                row[k] = rot_row(p, tok, h);
                a[k] = *reinterpret_cast<const uint4*>(row[k].x + at);
                if (!INTER && turns) b[k] = *reinterpret_cast<const uint4*>(row[k].x + p.half + at);
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (hb + k * stride >= h1) continue;
                if (!turns) {
                    *reinterpret_cast<uint4*>(row[k].y + at) = a[k];
                } else if constexpr (INTER) {
                    uint32_t w[4] = {a[k].x, a[k].y, a[k].z, a[k].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float2 v = rot_unpack<BF16>(w[i]);
                        if (col * 4 + i < p.half) w[i] = pack2<BF16>(v.x * c[i] - v.y * s[i], v.y * c[i] + v.x * s[i]);
                    }
                    *reinterpret_cast<uint4*>(row[k].y + at) = make_uint4(w[0], w[1], w[2], w[3]);
                } else {
                    float x1[8], x2[8];
                    rot_unpack8<BF16>(a[k], x1);
                    rot_unpack8<BF16>(b[k], x2);
                    uint32_t w1[4], w2[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        w1[i] = pack2<BF16>(x1[2 * i] * c[2 * i] - x2[2 * i] * s[2 * i], x1[2 * i + 1] * c[2 * i + 1] - x2[2 * i + 1] * s[2 * i + 1]);
                        w2[i] = pack2<BF16>(x2[2 * i] * c[2 * i] + x1[2 * i] * s[2 * i], x2[2 * i + 1] * c[2 * i + 1] + x1[2 * i + 1] * s[2 * i + 1]);
                    }
                    *reinterpret_cast<uint4*>(row[k].y + at) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
                    *reinterpret_cast<uint4*>(row[k].y + p.half + at) = make_uint4(w2[0], w2[1], w2[2], w2[3]);
                }
            }
        }
    }
}

// Pair by pair: half layout with any even rot_dim.
template <bool BF16>
__global__ void __launch_bounds__(kRotThreads) rotary_pairs_kernel(const __grid_constant__ RotaryParams p) {
    __shared__ float2 cs[kRotTable];
    grid_dependency_wait();
    const int64_t t0 = (int64_t)blockIdx.x * p.tokens_per_cta;
    const int nt = (int)min((int64_t)p.tokens_per_cta, (int64_t)p.B * p.S - t0);
    const int heads = p.H[0] + p.H[1];
    const int h0 = (int)((int64_t)heads * blockIdx.y / gridDim.y), h1 = (int)((int64_t)heads * (blockIdx.y + 1) / gridDim.y);
    rot_table(p, cs, t0, nt, 0, p.half);
    __syncthreads();
    const int items = p.half + (p.in_place ? 0 : p.D - 2 * p.half);     // of a row: pairs, then copied elements
    for (int64_t it = threadIdx.x; it < (int64_t)nt * (h1 - h0) * items; it += kRotThreads) {
        const int j = (int)(it % items), rw = (int)(it / items);
        const int t = rw / (h1 - h0);
        const RotRow row = rot_row(p, rot_token(p, t0 + t), h0 + rw - t * (h1 - h0));
        if (j < p.half) {
            const float2 v = cs[t * p.half + j];
            const float x1 = rot_unpack<BF16>(row.x[j]).x, x2 = rot_unpack<BF16>(row.x[j + p.half]).x;
            const uint32_t w = pack2<BF16>(x1 * v.x - x2 * v.y, x2 * v.x + x1 * v.y);
            row.y[j] = (uint16_t)(w & 0xFFFFu);
            row.y[j + p.half] = (uint16_t)(w >> 16);
        } else {
            row.y[j + p.half] = row.x[j + p.half];
        }
    }
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p0, bool bf16, bool interleaved, int nsm, cudaStream_t st) {
    RotaryParams p = p0;
    const int64_t tokens = (int64_t)p.B * p.S;
    // Tokens a CTA: as the table holds them, up to 16, fewer while that leaves SMs without CTAs.
    int tt = kRotTable / p.half;
    tt = tt > 16 ? 16 : tt;
    while (tt > 1 && (tokens + tt - 1) / tt < 4 * nsm) tt /= 2;
    p.tokens_per_cta = tt;
    const int64_t gx = (tokens + tt - 1) / tt;
    const int heads = p.H[0] + p.H[1];
    int gy = gx < nsm ? (int)((2 * nsm + gx - 1) / gx) : 1;
    gy = gy > heads ? heads : gy;
    const dim3 grid((unsigned)gx, (unsigned)gy), block(kRotThreads);
    if (!interleaved && p.half % 8 != 0)
        return bf16 ? launch_early(rotary_pairs_kernel<true>, grid, block, 0, st, p) : launch_early(rotary_pairs_kernel<false>, grid, block, 0, st, p);
    if (interleaved)
        return bf16 ? launch_early(rotary_columns_kernel<true, true>, grid, block, 0, st, p)
                    : launch_early(rotary_columns_kernel<false, true>, grid, block, 0, st, p);
    return bf16 ? launch_early(rotary_columns_kernel<true, false>, grid, block, 0, st, p)
                : launch_early(rotary_columns_kernel<false, false>, grid, block, 0, st, p);
}

}  // namespace fa
