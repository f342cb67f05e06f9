// kv_cache.cu -- writing new keys and values into a paged cache, quantised, and reading
// sequences back.
//
// A row is one token's D values of one head.  8-bit caches hold a code per value and one fp32
// scale per row:
//   s8     scale = max(rn(amax / 127), 2^-126), code = x / scale to the nearest even integer
//   e4m3   scale = the smallest power of two >= 2^-126 with amax / scale <= 448, code = x / scale
//          to the nearest even e4m3 value (the division is exact, so the code does not depend on
//          the precision it is done in)
// and a row that holds a NaN or an infinity gets scale = NaN, codes 0, and reads back as NaN.
// 16-bit caches hold the rows as they are.  Reading gives code * scale in fp32 (exact for the scales that
// e4m3 rows are written with, rounded for s8), rounded to 16 bits.
//
// Reading moves its bytes once and is bound by HBM (16 sequences of 1k-8k tokens, 16 heads, s8 to
// bf16: 201 us in a graph for 1.31 GB, 0.99 of the copy rate).  Appending is bound by its instructions as
// much (15k tokens of 8 heads to e4m3: 16.4 us in a graph for 95 MB; 16-bit magnitudes compared two at a
// time, 32-bit positions and eight lanes a row took two thirds of them away; to s8, with its test for
// quotients near a half, 22.9 us).  A row belongs to eight or D / 8
// lanes, so its maximum is a few shuffles and nothing is staged; rows of k and v at the same place go
// together.  The read has two rows of each in flight (four: 52.7 us against 49.6 for a prompt's write
// and read).
#include "serving.h"
#include "sm100_ptx.cuh"

#include <algorithm>

namespace fa {
namespace {

__device__ int32_t g_cache_rows_status;   // 2: a page or position out of range was met

constexpr int kRowThreads = 128;
constexpr int kReadAhead = 2;         // rows of k and of v that a lane group of the read has in flight

template <bool BF16>
__device__ __forceinline__ void row_unpack(const uint4& r, float (&f)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 two = unpack2<BF16>(w[i]);
        f[2 * i] = two.x;
        f[2 * i + 1] = two.y;
    }
}

// x / scale to the nearest integer, ties to even, exactly (|x / scale| <= 127 (1 + 2^-23)).  x times
// `inv`, which is within 2^-22 of 1 / scale, is within 2^-15 + 2^-18 of x / scale, so rounding the
// product is right unless it falls that near a half; the rows where one does within 10^-4 decide by
// the exact sign of x - (r +- 1/2) scale, one fma.
__device__ __forceinline__ int quantise_s8_exactly(float x, float scale, float inv) {
    float r = rintf(x * inv);
    const float up = fmaf(-(r + 0.5f), scale, x), down = fmaf(-(r - 0.5f), scale, x);
    const bool odd = ((int)r & 1) != 0;
    if (up > 0.f || (up == 0.f && odd)) r += 1.f;
    else if (down < 0.f || (down == 0.f && odd)) r -= 1.f;
    return (int)r;
}

__device__ __forceinline__ uint2 quantise_s8x8(const float (&x)[8], float scale, float inv) {
    constexpr float kMagic = 12582912.f;        // 1.5 * 2^23: its unit is 1, so adding it rounds to an integer
    uint32_t c[8];
    float near = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float m = fmaf(x[i], inv, kMagic);
        c[i] = __float_as_uint(m);              // the low byte is the code
        near = fmaxf(near, fabsf(fmaf(x[i], inv, kMagic - m)));
    }
    if (near > 0.4999f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = (uint32_t)quantise_s8_exactly(x[i], scale, inv);
    }
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = __byte_perm(__byte_perm(c[4 * i], c[4 * i + 1], 0x0040), __byte_perm(c[4 * i + 2], c[4 * i + 3], 0x0040), 0x5410);
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint32_t quantise_e4m3x2(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

// Two e4m3 codes as floats (exact).
__device__ __forceinline__ float2 value_e4m3x2(uint32_t codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    return unpack2<false>(h);
}

// The scale of a row from the bits of its largest magnitude.
template <int DT>
__device__ __forceinline__ float row_scale(uint32_t amax_bits) {
    if (amax_bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
    if constexpr (DT == FA_DTYPE_S8) return fmaxf(__fdiv_rn(__uint_as_float(amax_bits), 127.f), 1.17549435e-38f);
    // 448 = 1.75 * 2^8: the exponent of amax, one more where its mantissa exceeds 1.75, less 8.
    const int e = (int)((amax_bits + 0x1FFFFFu) >> 23) - 8;
    return __uint_as_float((uint32_t)max(e, 1) << 23);
}

// The bits, as fp32, of the largest magnitude of a row whose 16-bit values are spread over LPR
// lanes: magnitudes order as their bits, two at a time.
template <bool BF16, int P, int LPR>
__device__ __forceinline__ uint32_t row_amax(const uint4 (&r)[P]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < P; ++i)
        m = __vmaxu2(m, __vmaxu2(__vmaxu2(r[i].x & 0x7FFF7FFFu, r[i].y & 0x7FFF7FFFu), __vmaxu2(r[i].z & 0x7FFF7FFFu, r[i].w & 0x7FFF7FFFu)));
#pragma unroll
    for (int off = LPR / 2; off > 0; off >>= 1) m = __vmaxu2(m, __shfl_xor_sync(kFullMask, m, off));
    const uint32_t top = max(m & 0xFFFFu, m >> 16);
    return BF16 ? top << 16 : __float_as_uint(__half2float(__ushort_as_half((unsigned short)top)));
}

// What multiplies a row's values: the inverse of its scale, exactly for e4m3 (a power of two),
// within 2^-22 for s8.
template <int DT>
__device__ __forceinline__ float row_inverse(float scale) {
    if constexpr (DT == FA_DTYPE_E4M3) return __uint_as_float(0x7f000000u - __float_as_uint(scale));
    return __fdividef(1.f, scale);
}

// The code bytes of eight of a row's values.
template <int DT>
__device__ __forceinline__ uint2 quantise_8(const float (&x)[8], float scale, float inv) {
    if constexpr (DT == FA_DTYPE_S8) return quantise_s8x8(x, scale, inv);
    return make_uint2(quantise_e4m3x2(x[0] * inv, x[1] * inv) | quantise_e4m3x2(x[2] * inv, x[3] * inv) << 16,
                      quantise_e4m3x2(x[4] * inv, x[5] * inv) | quantise_e4m3x2(x[6] * inv, x[7] * inv) << 16);
}

// Grid (ceil(S / groups), H, B): LPR lanes take a row of k and of v, D / 8 / LPR pieces of 16 bytes a
// lane.  Eight lanes a row share its maximum and scale over most values (a prompt's write and read 45.9 us
// with eight, 49.3 with sixteen); for single rows D / 8 lanes are a little sooner done.
template <int DT, int D, bool BF16, int LPR>
__global__ void __launch_bounds__(kRowThreads) cache_append_kernel(const __grid_constant__ CacheRowsParams p) {
    constexpr int P = D / 8 / LPR;
    const int RPC = blockDim.x / LPR;
    grid_dependency_wait();
    const int sub = threadIdx.x % LPR;
    const int s = blockIdx.x * RPC + threadIdx.x / LPR;
    const int h = blockIdx.y, b = blockIdx.z;
    const int count = p.limit ? min(p.limit[b], p.S) : p.S;
    if ((int)(blockIdx.x * RPC) >= count) return;
    // A position start + s, as 32 bits without sign: past the capacity where it is negative.
    const uint32_t pos = (uint32_t)p.start[b] + s;
    uint4 raw[2][P];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const uint16_t* in = p.in[w] + b * p.rs[w][0] + h * p.rs[w][1] + (int64_t)s * p.rs[w][2] + sub * 8;
#pragma unroll
        for (int k = 0; k < P; ++k) raw[w][k] = s < count ? *reinterpret_cast<const uint4*>(in + 8 * LPR * k) : make_uint4(0, 0, 0, 0);
    }
    int page = -1;
    if (s < count) {
        page = cache_page(p.c, p.c.table + (int64_t)b * p.c.table_stride, pos);
        if (page < 0) g_cache_rows_status = 2;
    }
    const int row = pos & ((1 << p.c.page_shift) - 1);
    const int64_t at = (int64_t)page * p.c.stride[0] + h * p.c.stride[1] + (int64_t)row * p.c.stride[2] + sub * 8;
    const int64_t sat = (int64_t)page * p.c.scale_stride[0] + h * p.c.scale_stride[1] + (int64_t)row * p.c.scale_stride[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        void* pool = w ? p.c.v : p.c.k;
        if constexpr (!CacheType<DT>::k8) {
#pragma unroll
            for (int k = 0; k < P; ++k)
                if (page >= 0) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(pool) + at + 8 * LPR * k) = raw[w][k];
        } else {
            const uint32_t amax = row_amax<BF16, P, LPR>(raw[w]);
            const float scale = row_scale<DT>(amax), inv = row_inverse<DT>(scale);
            if (page >= 0 && sub == 0) (w ? p.c.v_scale : p.c.k_scale)[sat] = scale;
#pragma unroll
            for (int k = 0; k < P; ++k) {
                float x[8];
                row_unpack<BF16>(raw[w][k], x);
                uint2 c = quantise_8<DT>(x, scale, inv);
                if (amax >= 0x7f800000u) c = make_uint2(0u, 0u);
                if (page >= 0) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + at + 8 * LPR * k) = c;
            }
        }
    }
}

// Rows start .. start + S - 1 of each sequence; those past its length, or before position 0, are zero.
template <int DT, int D, bool BF16>
__global__ void __launch_bounds__(kRowThreads) cache_read_kernel(const __grid_constant__ CacheRowsParams p) {
    constexpr int LPR = D / 8;
    const int RPC = blockDim.x / LPR;
    grid_dependency_wait();
    const int sub = threadIdx.x % LPR;
    const int s0 = blockIdx.x * RPC * kReadAhead + threadIdx.x / LPR;
    const int h = blockIdx.y, b = blockIdx.z;
    const uint32_t start = p.start ? p.start[b] : 0;
    const int len = p.limit[b];
    const int32_t* table = p.c.table + (int64_t)b * p.c.table_stride;
    uint4 raw[kReadAhead][2];
    float scale[kReadAhead][2];
#pragma unroll
    for (int i = 0; i < kReadAhead; ++i) {
        const uint32_t pos = start + s0 + i * RPC;      // as in the append
        int page = -1;
        if (s0 + i * RPC < p.S && (int)pos >= 0 && (int)pos < len) {
            page = cache_page(p.c, table, pos);
            if (page < 0) g_cache_rows_status = 2;
        }
        const int row = pos & ((1 << p.c.page_shift) - 1);
        const int64_t at = (int64_t)page * p.c.stride[0] + h * p.c.stride[1] + (int64_t)row * p.c.stride[2] + sub * 8;
        const int64_t sat = (int64_t)page * p.c.scale_stride[0] + h * p.c.scale_stride[1] + (int64_t)row * p.c.scale_stride[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            raw[i][w] = make_uint4(0, 0, 0, 0);
            scale[i][w] = 0.f;
            if (page < 0) continue;
            const void* pool = w ? p.c.v : p.c.k;
            if constexpr (!CacheType<DT>::k8) {
                raw[i][w] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(pool) + at);
            } else {
                const uint2 c = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(pool) + at);
                raw[i][w].x = c.x;
                raw[i][w].y = c.y;
                scale[i][w] = (w ? p.c.v_scale : p.c.k_scale)[sat];
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kReadAhead; ++i) {
        const int s = s0 + i * RPC;
        if (s >= p.S) continue;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            uint4 r = raw[i][w];
            if constexpr (CacheType<DT>::k8) {
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t two = ((e < 2 ? raw[i][w].x : raw[i][w].y) >> (16 * (e % 2))) & 0xFFFFu;
                    float2 f;
                    if constexpr (DT == FA_DTYPE_S8) f = make_float2((float)(int8_t)(two & 0xFF), (float)(int8_t)(two >> 8));
                    else f = value_e4m3x2(two);
                    o[e] = pack2<BF16>(f.x * scale[i][w], f.y * scale[i][w]);
                }
                r = make_uint4(o[0], o[1], o[2], o[3]);
            }
            *reinterpret_cast<uint4*>(p.out[w] + b * p.rs[w][0] + h * p.rs[w][1] + (int64_t)s * p.rs[w][2] + sub * 8) = r;
        }
    }
    // A length or start that no page could hold is recorded even where it touches no page.
    if (blockIdx.x == 0 && blockIdx.y == 0 && ((unsigned)len > (unsigned)p.c.capacity || (int)start < 0)) g_cache_rows_status = 2;
}

template <int DT, int D, bool BF16>
cudaError_t launch_rows(const CacheRowsParams& p, bool append, cudaStream_t st) {
    const bool few = !append || p.S < 16;
    const int lanes = few ? D / 8 : 8;
    // A warp is enough for a step's single rows; a block's other warps would only be in the way.
    const int warps = (int)std::min<int64_t>(kRowThreads / 32, ((int64_t)p.S * lanes + 31) / 32);
    const int rows = warps * 32 / lanes * (append ? 1 : kReadAhead);
    const dim3 grid((unsigned)((p.S + rows - 1) / rows), (unsigned)p.c.H, (unsigned)p.B), block(warps * 32);
    if (!append) return launch_early(cache_read_kernel<DT, D, BF16>, grid, block, 0, st, p);
    return few ? launch_early(cache_append_kernel<DT, D, BF16, D / 8>, grid, block, 0, st, p)
               : launch_early(cache_append_kernel<DT, D, BF16, 8>, grid, block, 0, st, p);
}

cudaError_t launch_any(const CacheRowsParams& p, int dtype, int D, bool bf16, bool append, cudaStream_t st) {
#define FA_ROWS(T, DD, BB) \
    if (dtype == T && D == DD && bf16 == BB) return launch_rows<T, DD, BB>(p, append, st);
#define FA_ROWS_D(T, BB) FA_ROWS(T, 64, BB) FA_ROWS(T, 128, BB)
    FA_ROWS_D(FA_DTYPE_F16, false)
    FA_ROWS_D(FA_DTYPE_BF16, true)
    FA_ROWS_D(FA_DTYPE_E4M3, false)
    FA_ROWS_D(FA_DTYPE_E4M3, true)
    FA_ROWS_D(FA_DTYPE_S8, false)
    FA_ROWS_D(FA_DTYPE_S8, true)
#undef FA_ROWS_D
#undef FA_ROWS
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_cache_append(const CacheRowsParams& p, int dtype, int D, bool bf16, cudaStream_t st) {
    return launch_any(p, dtype, D, bf16, true, st);
}
cudaError_t launch_cache_read(const CacheRowsParams& p, int dtype, int D, bool bf16, cudaStream_t st) {
    return launch_any(p, dtype, D, bf16, false, st);
}

cudaError_t cache_rows_status_word(int32_t** word) { return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_cache_rows_status); }

}  // namespace fa
