// rotary.cu -- rotary positions of q and k, and their gradient.
//
// A pair (x1, x2) of the token at position t turns by a = t * f_i: y1 = c (x1 cos a - x2 sin a),
// y2 = c (x2 cos a + x1 sin a), rounded once; the gradient is the same with -a.  The angle is
// held in turns as a 64-bit fraction: F = f_i / 2 pi * 2^64 (from the frequency in 64-bit
// floating point) times the integer position, modulo 2^64, is the angle modulo one turn with no
// rounding but F's, so a position of a million is as exact as position one; cos and sin are then
// taken of a 32-bit fraction in [-1/2, 1/2) turns.
//
// Bound by HBM (2 bytes read and 2 written an element): 40 heads x 32768 tokens of D = 128, half of
// it turned, 115 us, 5.84 TB/s or 0.89 of the copy rate; 32 heads x 8192 tokens of D = 64, 13.2 us
// (both replayed in a graph; calls 117 and 14.3).  A CTA takes a few tokens of every head: their cos and sin are computed once into
// shared memory and serve all heads of q and k.  Work goes in columns of 16 bytes (half layout: the
// two columns of eight pairs; of 8 bytes where rot_dim is a multiple of 8 but not of 16, the copied
// rest in 16 all the same: 10 x 1833 tokens of 32 heads, 24 of 192 elements, 80 us, 107 before): a thread
// keeps its column and walks the rows (token, head) by fixed offsets, with the loads of kAhead rows
// in flight (twice as many: 20.5 us at 8192 tokens).  Pairs that do not fill such columns (half
// layout with rot_dim no multiple of 8) go one by one: 26 of 64 elements at 8192 tokens take 83 us.
// The table's arithmetic is shared by the heads, and where those are few it is what is waited for: 5
// heads x 16384 tokens of D = 128, 12.8 us, half the copy rate.
#include "serving.h"
#include "sm100_ptx.cuh"

#include <algorithm>

namespace fa {
namespace {

constexpr int kRotThreads = 256;
constexpr int kRotTable = 2048;   // (token, pair) entries of cos and sin a CTA: 16 KiB

__device__ __forceinline__ float2 rotary_cos_sin(double freq, int64_t pos, float factor, bool inverse) {
    double turns = freq * 0.15915494309189533577;      // radians to turns
    turns -= floor(turns);
    const uint64_t fixed = (uint64_t)(turns * 18446744073709551616.0) * (uint64_t)pos;
    float x = (float)(int32_t)(fixed >> 32) * 4.656612873077393e-10f;   // half turns, [-1, 1)
    if (!isfinite(freq)) x = __int_as_float(0x7fc00000);
    float s, c;
    sincospif(x, &s, &c);
    return make_float2(c * factor, (inverse ? -s : s) * factor);
}

// cos and sin (times the factor) of the first `half` pairs of tokens t0 .. t0 + nt - 1 of sequence
// b, pair j of token t at cs[t * pitch + place(j)].
template <class Place>
__device__ __forceinline__ void rot_table(const RotaryParams& p, float2* cs, int b, int t0, int nt, int pitch, Place&& place) {
    constexpr int kEntries = 4;                     // of a thread whose loads are in flight at once
    const int n = nt * p.half;
    for (int i0 = threadIdx.x; i0 < n; i0 += kEntries * kRotThreads) {
        double freq[kEntries];
        int64_t pos[kEntries];
#pragma unroll
        for (int k = 0; k < kEntries; ++k) {
            const int i = i0 + k * kRotThreads, t = i / p.half, s = t0 + t;
            if (i >= n) break;
            freq[k] = p.freq[i - t * p.half];
            pos[k] = p.pos ? (int64_t)p.pos[b * p.pos_stride + s * p.pos_token_stride] : p.pos0 + s * p.pos_token_stride;
        }
#pragma unroll
        for (int k = 0; k < kEntries; ++k) {
            const int i = i0 + k * kRotThreads, t = i / p.half;
            if (i >= n) break;
            cs[t * pitch + place(i - t * p.half)] = rotary_cos_sin(freq[k], pos[k], p.factor, p.inverse != 0);
        }
    }
}

// A CTA's tokens, of one sequence, and its heads, of all those of q and k.
struct RotTile {
    int b, t0, nt, h0, h1;
};
__device__ __forceinline__ RotTile rot_tile(const RotaryParams& p) {
    RotTile r;
    r.b = blockIdx.x / p.ctas_per_seq;
    r.t0 = (blockIdx.x - r.b * p.ctas_per_seq) * p.tokens_per_cta;
    r.nt = min(p.tokens_per_cta, p.S - r.t0);
    const int heads = p.H[0] + p.H[1];
    r.h0 = (int)((int64_t)heads * blockIdx.y / gridDim.y);
    r.h1 = (int)((int64_t)heads * (blockIdx.y + 1) / gridDim.y);
    return r;
}

// W words as one access.
template <int W>
__device__ __forceinline__ void load_words(const uint16_t* x, uint32_t* w) {
    if constexpr (W == 4) {
        const uint4 v = *reinterpret_cast<const uint4*>(x);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(x);
        w[0] = v.x, w[1] = v.y;
    }
}
template <int W>
__device__ __forceinline__ void store_words(uint16_t* y, const uint32_t* w) {
    if constexpr (W == 4) *reinterpret_cast<uint4*>(y) = make_uint4(w[0], w[1], w[2], w[3]);
    else *reinterpret_cast<uint2*>(y) = make_uint2(w[0], w[1]);
}

// By columns of 2 W elements: half layout with rot_dim a multiple of 4 W, or interleaved (W = 4) with
// any rot_dim.
template <bool BF16, bool INTER, int W>
__global__ void __launch_bounds__(kRotThreads, 4) rotary_columns_kernel(const __grid_constant__ RotaryParams p) {
    __shared__ __align__(16) float2 cs[kRotTable];
    constexpr int kAhead = INTER || W == 2 ? 4 : 2;     // rows whose loads are in flight at once
    constexpr int E = 2 * W, J = INTER ? W : E;         // elements and pairs a column
    grid_dependency_wait();
    const RotTile tile = rot_tile(p);
    // The columns of a row: rotated ones (half layout: pairs of columns), then copied ones.
    const int rot_cols = (p.half + J - 1) / J;
    const int copied0 = INTER ? rot_cols * E : 2 * p.half;
    const int cols = rot_cols + (p.in_place ? 0 : (p.D - copied0) / 8);        // copied ones are of 16 bytes
    const int col = threadIdx.x % cols, first = threadIdx.x / cols, stride = kRotThreads / cols;   // D <= 1024: cols <= 256
    // Two pairs of all columns stand together: neighbouring columns read neighbouring 16 bytes.
    const int pitch = rot_cols * J;
    rot_table(p, cs, tile.b, tile.t0, tile.nt, pitch, [&](int j) { return (j % J / 2) * rot_cols * 2 + j / J * 2 + (j & 1); });
    __syncthreads();
    if (first >= stride) return;
    const bool turns = col < rot_cols, full = !INTER || col * W + W <= p.half;
    const int at = turns ? col * E : copied0 + (col - rot_cols) * 8;
#pragma unroll 1
    for (int w = 0; w < 2; ++w) {                  // q, k
        const int hb = w ? p.H[0] : 0;
        const int h0 = max(tile.h0, hb) - hb, nh = min(tile.h1 - hb, p.H[w]) - h0;
        if (nh <= 0) continue;
        // Rows (token, head), the index whose rows lie closer together first; a step of `stride` rows
        // is a fixed offset, another when the first index wraps.
        const bool tok_in = p.xs[w][2] < p.xs[w][1];
        const int inner = tok_in ? tile.nt : nh, rows = tile.nt * nh;
        int in = first % inner, out = first / inner;
        const int in_step = stride % inner, out_step = stride / inner;
        const int64_t xi = tok_in ? p.xs[w][2] : p.xs[w][1], xo = tok_in ? p.xs[w][1] : p.xs[w][2];
        const int64_t yi = tok_in ? p.ys[w][2] : p.ys[w][1], yo = tok_in ? p.ys[w][1] : p.ys[w][2];
        const uint16_t* x = p.x[w] + tile.b * p.xs[w][0] + tile.t0 * p.xs[w][2] + h0 * p.xs[w][1] + in * xi + out * xo + at;
        uint16_t* y = p.y[w] + tile.b * p.ys[w][0] + tile.t0 * p.ys[w][2] + h0 * p.ys[w][1] + in * yi + out * yo + at;
        const int64_t x_step = in_step * xi + out_step * xo, x_wrap = xo - inner * xi;
        const int64_t y_step = in_step * yi + out_step * yo, y_wrap = yo - inner * yi;
        for (int rw = first; rw < rows; rw += stride * kAhead) {
            uint32_t v[kAhead][2 * W];      // a column and, in half layout, its pairs' other halves
            int token[kAhead];
            uint16_t* to[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (rw + k * stride < rows) {
                    if (turns || W == 4) load_words<W>(x, v[k]);
                    else load_words<4>(x, v[k]);
                    if (!INTER && turns) load_words<W>(x + p.half, v[k] + W);
                }
                token[k] = tok_in ? in : out;
                to[k] = y;
                in += in_step;
                out += out_step;
                x += x_step;
                y += y_step;
                if (in >= inner) {
                    in -= inner;
                    ++out;
                    x += x_wrap;
                    y += y_wrap;
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (rw + k * stride >= rows) break;
                const float2* turn = cs + token[k] * pitch + col * 2;
                if (turns && INTER) {
#pragma unroll
                    for (int i = 0; i < W / 2; ++i) {
                        const float4 q = *reinterpret_cast<const float4*>(turn + i * rot_cols * 2);
                        const float2 e = unpack2<BF16>(v[k][2 * i]), f = unpack2<BF16>(v[k][2 * i + 1]);
                        if (full || col * W + 2 * i < p.half) v[k][2 * i] = pack2<BF16>(e.x * q.x - e.y * q.y, e.y * q.x + e.x * q.y);
                        if (full || col * W + 2 * i + 1 < p.half) v[k][2 * i + 1] = pack2<BF16>(f.x * q.z - f.y * q.w, f.y * q.z + f.x * q.w);
                    }
                } else if (turns) {
#pragma unroll
                    for (int i = 0; i < W; ++i) {
                        const float4 q = *reinterpret_cast<const float4*>(turn + i * rot_cols * 2);
                        const float2 x1 = unpack2<BF16>(v[k][i]), x2 = unpack2<BF16>(v[k][W + i]);
                        v[k][i] = pack2<BF16>(x1.x * q.x - x2.x * q.y, x1.y * q.z - x2.y * q.w);
                        v[k][W + i] = pack2<BF16>(x2.x * q.x + x1.x * q.y, x2.y * q.z + x1.y * q.w);
                    }
                    store_words<W>(to[k] + p.half, v[k] + W);
                }
                if (turns || W == 4) store_words<W>(to[k], v[k]);
                else store_words<4>(to[k], v[k]);
            }
        }
    }
}

// Pair by pair: half layout with any even rot_dim.
template <bool BF16>
__global__ void __launch_bounds__(kRotThreads) rotary_pairs_kernel(const __grid_constant__ RotaryParams p) {
    __shared__ float2 cs[kRotTable];
    grid_dependency_wait();
    const RotTile tile = rot_tile(p);
    rot_table(p, cs, tile.b, tile.t0, tile.nt, p.half, [](int j) { return j; });
    __syncthreads();
    const int items = p.half + (p.in_place ? 0 : p.D - 2 * p.half);     // of a row: pairs, then copied elements
    const int wide = min(items, kRotThreads), first = threadIdx.x / wide, step = kRotThreads / wide;
    const int nh = tile.h1 - tile.h0, rows = first < step ? tile.nt * nh : 0;
    for (int j = threadIdx.x - first * wide; j < items; j += kRotThreads)
        for (int rw = first; rw < rows; rw += step) {
            const int t = rw / nh, head = tile.h0 + rw - t * nh;
            const int w = head >= p.H[0], h = w ? head - p.H[0] : head, s = tile.t0 + t;
            const uint16_t* x = p.x[w] + tile.b * p.xs[w][0] + h * p.xs[w][1] + s * p.xs[w][2];
            uint16_t* y = p.y[w] + tile.b * p.ys[w][0] + h * p.ys[w][1] + s * p.ys[w][2];
            if (j < p.half) {
                const float2 v = cs[t * p.half + j];
                const float x1 = unpack2<BF16>(x[j]).x, x2 = unpack2<BF16>(x[j + p.half]).x;
                const uint32_t u = pack2<BF16>(x1 * v.x - x2 * v.y, x2 * v.x + x1 * v.y);
                y[j] = (uint16_t)(u & 0xFFFFu);
                y[j + p.half] = (uint16_t)(u >> 16);
            } else {
                y[j + p.half] = x[j + p.half];
            }
        }
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams& p0, bool bf16, bool interleaved, int nsm, cudaStream_t st) {
    RotaryParams p = p0;
    p.pos_token_stride = 1;
    if (p.S == 1) {
        // One token a sequence: the sequences take the tokens' place.
        p.S = p.B;
        p.B = 1;
        for (int w = 0; w < 2; ++w) {
            p.xs[w][2] = p.xs[w][0];
            p.ys[w][2] = p.ys[w][0];
        }
        p.pos_token_stride = p.pos ? p.pos_stride : 0;
    }
    // Tokens a CTA.  A CTA's latencies need work beside them, so few CTAs an SM (2048 tokens of 32
    // heads, D = 64: 5.0 us with two an SM, 6.4 with four, 8.4 with eight), four where two would take
    // more tokens than 16 or, with few heads, some 512 rows (8192 tokens: 13.1 us, with two 14.2; 65536
    // tokens of two heads: 18 us, with 16 tokens 33), and no more than that or the table holds.
    const int heads = p.H[0] + p.H[1];
    const int64_t tokens = (int64_t)p.B * p.S;
    const int most = std::min(kRotTable / ((p.half + 7) / 8 * 8), std::max(16, 512 / heads));
    int64_t tt = (tokens + 2 * nsm - 1) / (2 * nsm);
    if (tt > most) tt = std::min<int64_t>(most, (tokens + 4 * nsm - 1) / (4 * nsm));
    p.tokens_per_cta = (int)tt;
    p.ctas_per_seq = (int)((p.S + tt - 1) / tt);
    const int64_t gx = (int64_t)p.B * p.ctas_per_seq;       // at most the tokens: fewer than 2^31
    int gy = gx < nsm ? (int)((2 * nsm + gx - 1) / gx) : 1;
    gy = gy > heads ? heads : gy;
    const dim3 grid((unsigned)gx, (unsigned)gy), block(kRotThreads);
    if (!interleaved && p.half % 4 != 0)
        return bf16 ? launch_early(rotary_pairs_kernel<true>, grid, block, 0, st, p) : launch_early(rotary_pairs_kernel<false>, grid, block, 0, st, p);
    if (interleaved)
        return bf16 ? launch_early(rotary_columns_kernel<true, true, 4>, grid, block, 0, st, p)
                    : launch_early(rotary_columns_kernel<false, true, 4>, grid, block, 0, st, p);
    if (p.half % 8 != 0)
        return bf16 ? launch_early(rotary_columns_kernel<true, false, 2>, grid, block, 0, st, p)
                    : launch_early(rotary_columns_kernel<false, false, 2>, grid, block, 0, st, p);
    return bf16 ? launch_early(rotary_columns_kernel<true, false, 4>, grid, block, 0, st, p)
                : launch_early(rotary_columns_kernel<false, false, 4>, grid, block, 0, st, p);
}

}  // namespace fa
