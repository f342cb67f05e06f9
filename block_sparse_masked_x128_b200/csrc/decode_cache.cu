// decode_cache.cu -- attention of one new token a sequence over a paged, possibly quantised
// cache with grouped heads.
//
//   x_j = mod(scale * q . k_j),  p = softmax of x over max(0, len - window) <= j < len,
//   out = sum_j p_j v_j,  lse = log sum_j exp x_j        (no key: out 0, lse -inf)
//
// The work is reading K and V once, so HBM bounds it as long as nothing else is in the way:
//
//   Split      the keys of all (sequence, kv head)s form one list of units of kUnit keys, and the
//              CTAs of one wave take equal shares of it, so ragged lengths and single long
//              sequences load every SM alike.  The lengths are device data: each CTA finds its
//              share by a scan over the sequences.  A share that holds all of a head's keys writes
//              the result itself; otherwise its (m, l, O) goes to the workspace and the merge
//              kernel joins the pieces in key order (no atomics: the same bits every time).
//   Heads      the query heads of a kv head are the columns of the products (8 or 16 at a time):
//              S^T = K q^T and O^T = V^T P^T, with 16 keys or 16 dims as rows.  The matrix
//              pipe is needed only because one cache byte meets up to 16 heads; at 8 columns
//              mma.sync keeps up with HBM several times over, and its operands come straight
//              from the loaded bytes.
//   Loads      each lane copies with cp.async exactly the bytes that its own fragments are made
//              of, into slots that only it reads (the products' contraction index may run through
//              the dims in any order, so a lane's 16 contiguous bytes serve as four steps of it).
//              So shared memory is a queue a lane: no barrier, no layout, no bank conflict.
//   8 bits     codes become fp16 exactly, in registers.  The key's scale multiplies its score, the
//              value's scale the weight p, both in fp32.  q is brought into fp16's range by a
//              power of two a head, the weights by a running power of two R >= every v scale so
//              far, so neither rounds out of range: q keeps all its bits, p is rounded to 11.
//   Softmax    the reference m of a head's exponents is raised only when a score exceeds it by 8
//              (in log2): weights stay below 2^8 and most tiles need no reduction over the lanes.
#include "serving.h"
#include "sm100_ptx.cuh"

#include <cfloat>

#include <cuda_fp16.h>

namespace fa {
namespace {

__device__ int32_t g_cache_decode_status;   // 2: a length or page out of range was met

constexpr int kCdWarps = 4, kCdThreads = 32 * kCdWarps;
constexpr int kTileKeys = 16;               // keys a warp takes at a time
constexpr float kCdLn2 = 0.6931471805599453f, kCdLog2e = 1.4426950408889634f;
constexpr float kRaise = 8.f;               // how far (log2) a score may exceed the reference

template <int DT, int D, int NT>
struct CdConfig {
    static constexpr bool k8 = CacheType<DT>::k8;
    static constexpr int bytes = CacheType<DT>::bytes;
    static constexpr int kch = D * bytes / 64;            // 16-byte K chunks a lane and row
    static constexpr int vb = D / 8 * bytes < 16 ? 8 : 16;  // bytes of a V chunk
    static constexpr int vch = D / 8 * bytes / vb;        // V chunks a lane and row
    static constexpr int kbytes = 2 * kch * 512;          // 2 rows a lane
    static constexpr int vbytes = 4 * vch * 32 * vb;      // 4 rows a lane
    static constexpr int stage = kbytes + vbytes + (k8 ? 128 : 0);
    static constexpr int occ = D * bytes == 256 ? 2 : (NT == 1 ? 4 : 3);
    static constexpr int stages = D * bytes == 64 ? 6 : 3;
    static constexpr int ring = kCdWarps * stages * stage;
    // Join of the warps: O rows of D floats, 4 more after each 8 or 16 (bank conflicts).
    static constexpr int seg = k8 && D == 128 ? 16 : 8;
    static constexpr int orow = D + D / seg * 4;
    static constexpr int join = kCdWarps * 8 * NT * (orow + 2) * 4 + 8 * NT * (kCdWarps + 2) * 4;
    static constexpr int smem = ring > join ? ring : join;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src, int n) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src, int n) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float lds_f32(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

// D (16 x 8) += A (16 x 16) B (16 x 8), fp32 accumulation.  With r = lane / 4, c = lane % 4: A's
// registers hold (row r, k 2c 2c+1), (r + 8, same), (r, k 2c+8 2c+9), (r + 8, same); B's (k 2c 2c+1,
// column r), (k 2c+8 2c+9, column r); D's (row r, columns 2c 2c+1), (row r + 8, same).
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 matrix of 16-bit values, lane (r, c) holding (row r, columns 2c 2c+1).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// Bytes 2 HI and 2 HI + 1 of four codes as two fp16 values, exactly.  s8: the code plus 128 in the
// low byte of 1024 = 0x6400, whose unit is 1, less 1152.
template <int DT, int HI>
__device__ __forceinline__ uint32_t codes_to_half2(uint32_t w) {
    uint32_t h;
    if constexpr (DT == FA_DTYPE_S8) {
        const uint32_t u = __byte_perm(w ^ 0x80808080u, 0x64646464u, HI ? 0x4342 : 0x4140);
        asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(h) : "r"(u), "r"(0x64806480u));
    } else {
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(HI ? w >> 16 : w & 0xFFFFu)));
    }
    return h;
}

// The keys of sequence b that are attended to, [lo, len), and their number of units.
struct SeqRange {
    int32_t lo, len, tile0, tile1;
    int32_t units;
};
__device__ __forceinline__ SeqRange seq_range(const CacheDecodeParams& p, int b) {
    SeqRange r;
    const int64_t cap = min((int64_t)p.c.table_width << p.c.page_shift, (int64_t)0x7fffffc0);
    const int n = __ldg(p.kv_lens + b);
    if (n < 0 || n > cap) g_cache_decode_status = 2;
    r.len = (int32_t)max((int64_t)0, min((int64_t)n, cap));
    r.lo = p.window > 0 ? max(0, r.len - p.window) : 0;
    r.tile0 = r.lo / kTileKeys;
    r.tile1 = (r.len + kTileKeys - 1) / kTileKeys;
    r.units = r.len > r.lo ? (r.tile1 - r.tile0 + kCdWarps - 1) / kCdWarps : 0;
    return r;
}

// Scan over the sequences: the units of all of them, and those before thread t's own share
// [t n, (t + 1) n) of the sequences.
struct SeqScan {
    int64_t total, before;
    int32_t first, last;
};
template <int THREADS>
__device__ __forceinline__ SeqScan scan_sequences(const CacheDecodeParams& p) {
    __shared__ int64_t sums[THREADS / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = (p.B + THREADS - 1) / THREADS;
    SeqScan s;
    s.first = min(p.B, (int)threadIdx.x * n);
    s.last = min(p.B, s.first + n);
    int64_t mine = 0;
    for (int b = s.first; b < s.last; ++b) mine += seq_range(p, b).units;
    int64_t inc = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t v = __shfl_up_sync(kFullMask, inc, off);
        if (lane >= off) inc += v;
    }
    if (lane == 31) sums[warp] = inc;
    __syncthreads();
    int64_t below = 0, all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) below += sums[w];
        all += sums[w];
    }
    s.total = all;
    s.before = below + inc - mine;
    return s;
}

// The head groups of a kv head: columns of the products, `rows` of them at a time.
__host__ __device__ constexpr int col_blocks(int group, int cols) { return (group + cols - 1) / cols; }

template <int DT, int D, int NT>
__global__ void __launch_bounds__(kCdThreads, CdConfig<DT, D, NT>::occ)
cache_decode_kernel(const __grid_constant__ CacheDecodeParams p, bool q_bf16) {
    using C = CdConfig<DT, D, NT>;
    constexpr bool BF16 = DT == FA_DTYPE_BF16;      // type of the products (8-bit: fp16)
    constexpr int KS = D / 16;                      // contraction steps of K q^T, and row tiles of O^T
    constexpr int COLS = 8 * NT;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t s_before;
    __shared__ int32_t s_seq;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, c = lane & 3;

    // This CTA's share of the units, and where it begins.
    const int CB = col_blocks(p.group, COLS), HR = p.c.H * CB;
    const SeqScan scan = scan_sequences<kCdThreads>(p);
    const int64_t total = scan.total * HR;
    const int64_t share = (total + gridDim.x - 1) / gridDim.x;
    const int64_t u_begin = share * blockIdx.x, u_end = min(total, u_begin + share);
    if (u_begin >= u_end) return;
    {
        const int64_t q0 = u_begin / HR;
        int64_t before = scan.before;
        for (int b = scan.first; b < scan.last; ++b) {
            const int n = seq_range(p, b).units;
            if (q0 >= before && q0 < before + n) {
                s_seq = b;
                s_before = before;
            }
            before += n;
        }
    }
    __syncthreads();
    int b = s_seq;
    SeqRange sr = seq_range(p, b);
    int64_t u = u_begin;
    int hr, unit0;      // head group and first unit of the segment at hand
    {
        const int64_t rem = u_begin - s_before * HR;
        hr = (int)(rem / sr.units);
        unit0 = (int)(rem % sr.units);
    }
    const uint32_t ring = smem_u32(smem) + warp * C::stages * C::stage;
    const int64_t kv_row = p.c.stride[2] * C::bytes;
    // Offsets of this lane's bytes within a tile: K rows r and r + 8, V rows 2c, 2c+1, 2c+8, 2c+9.
    const int64_t k_off = r * kv_row + c * 16;
    const int64_t v_off = 2 * c * kv_row + r * C::vb;

    while (u < u_end) {
        const int seg_units = (int)min((int64_t)(sr.units - unit0), u_end - u);
        const int h = hr / CB, col0 = (hr - h * CB) * COLS;
        const int cols = min(COLS, p.group - col0);
        const int hq0 = h * p.group + col0;

        // q as the second operand: lane (r, c) holds column r's dims of step s at
        // (16-byte chunk of 64 bytes of a K row) + 4 (step within the chunk) + 0..3.
        uint32_t qf[NT][KS][2];
        float cs[NT][2], slope[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int col = nt * 8 + r;
            const uint16_t* q = p.q + b * p.q_stride[0] + (int64_t)(hq0 + col) * p.q_stride[1];
            uint2 raw[KS];
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                constexpr int SPC = 4 / C::bytes;   // steps a chunk
                const int dim = (s / SPC) * (64 / C::bytes) + c * (16 / C::bytes) + (s % SPC) * 4;
                raw[s] = col < cols ? *reinterpret_cast<const uint2*>(q + dim) : make_uint2(0, 0);
            }
            float unit = 1.f;                       // q = unit * (what goes into the product)
            if constexpr (!C::k8) {
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    qf[nt][s][0] = raw[s].x;
                    qf[nt][s][1] = raw[s].y;
                }
            } else {
                float f[KS][4];
                uint32_t top = 0;
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    const uint32_t w[2] = {raw[s].x, raw[s].y};
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        f[s][2 * i] = q_bf16 ? __uint_as_float(w[i] << 16) : __half2float(__ushort_as_half((unsigned short)(w[i] & 0xFFFFu)));
                        f[s][2 * i + 1] = q_bf16 ? __uint_as_float(w[i] & 0xFFFF0000u) : __half2float(__ushort_as_half((unsigned short)(w[i] >> 16)));
                        top = max(top, max(__float_as_uint(f[s][2 * i]) & 0x7fffffffu, __float_as_uint(f[s][2 * i + 1]) & 0x7fffffffu));
                    }
                }
                top = max(top, __shfl_xor_sync(kFullMask, top, 1));
                top = max(top, __shfl_xor_sync(kFullMask, top, 2));
                // 2^n takes the largest magnitude into [2^14, 2^15) (n at most 126).
                const int n = top == 0 ? 0 : min(126, 14 + 127 - (int)(top >> 23));
                const float up = __uint_as_float((uint32_t)(n + 127) << 23);
                unit = __uint_as_float((uint32_t)(127 - n) << 23);
#pragma unroll
                for (int s = 0; s < KS; ++s) {
                    qf[nt][s][0] = pack2<false>(f[s][0] * up, f[s][1] * up);
                    qf[nt][s][1] = pack2<false>(f[s][2] * up, f[s][3] * up);
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {           // columns 2c and 2c + 1
                cs[nt][j] = p.scale_log2 * __shfl_sync(kFullMask, unit, (2 * c + j) * 4);
                slope[nt][j] = 0.f;
                if ((p.score_kind & FA_SCORE_ALIBI) && nt * 8 + 2 * c + j < cols) {
                    const int hq = hq0 + nt * 8 + 2 * c + j;
                    slope[nt][j] = kCdLog2e * (p.alibi_slopes ? __ldg(p.alibi_slopes + hq) : exp2f(-8.f * (float)(hq + 1) / (float)p.HQ));
                }
            }
        }
        float m[NT][2], l[NT][2], o[NT][KS][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -FLT_MAX;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int t = 0; t < KS; ++t) o[nt][t][0] = o[nt][t][1] = o[nt][t][2] = o[nt][t][3] = 0.f;
        }
        float R = C::k8 ? 1.17549435e-38f : 1.f, inv_R = 8.50705917e37f;    // 2^-126 and 2^126; unused for 16 bits

        const int t_end = min(sr.tile1, sr.tile0 + (unit0 + seg_units) * kCdWarps);
        int t = sr.tile0 + unit0 * kCdWarps + warp;           // tile at hand
        int ti = t;                                           // next tile to load
        uint32_t bad = 0;                                     // ring slots whose page is out of range
        auto page_of = [&](int tile) { return tile < t_end ? cache_page(p.c, b, ((int64_t)tile * kTileKeys) >> p.c.page_shift) : -1; };
        int page = page_of(ti);
        auto issue = [&](int slot) {
            const int key0 = ti * kTileKeys;
            if (page < 0) {
                bad |= 1u << slot;
                if (lane == 0) g_cache_decode_status = 2;
            } else {
                bad &= ~(1u << slot);
            }
            const bool whole = page >= 0 && key0 >= sr.lo && key0 + kTileKeys <= sr.len;
            // Rows outside [lo, len) are filled with zeros, not read.
            auto live = [&](int row) { return whole || (page >= 0 && key0 + row >= sr.lo && key0 + row < sr.len); };
            const int row0 = key0 & ((1 << p.c.page_shift) - 1);
            const int64_t at = page < 0 ? 0 : ((int64_t)page * p.c.stride[0] + h * p.c.stride[1]) * C::bytes + row0 * kv_row;
            const uint8_t* kp = static_cast<const uint8_t*>(p.c.k) + at + k_off;
            const uint8_t* vp = static_cast<const uint8_t*>(p.c.v) + at + v_off;
            const uint32_t ks = ring + slot * C::stage + lane * 16;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const bool ok = live(r + 8 * i);
                const uint8_t* src = ok ? kp + 8 * i * kv_row : static_cast<const uint8_t*>(p.c.k);
#pragma unroll
                for (int e = 0; e < C::kch; ++e) cp_async16(ks + (i * C::kch + e) * 512, ok ? src + 64 * e : src, ok ? 16 : 0);
            }
            const uint32_t vs = ring + slot * C::stage + C::kbytes + lane * C::vb;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = (i & 1) + 8 * (i >> 1);
                const bool ok = live(2 * c + row);
                const uint8_t* src = ok ? vp + row * kv_row : static_cast<const uint8_t*>(p.c.v);
#pragma unroll
                for (int e = 0; e < C::vch; ++e) {
                    const uint32_t dst = vs + (i * C::vch + e) * 32 * C::vb;
                    if constexpr (C::vb == 16) cp_async16(dst, ok ? src + 128 * e : src, ok ? 16 : 0);
                    else cp_async8(dst, src, ok ? 8 : 0);
                }
            }
            if constexpr (C::k8) {
                // Lanes 0-15 the K scales, 16-31 the V scales.
                const bool ok = live(lane & 15);
                const float* sp = lane < 16 ? p.c.k_scale : p.c.v_scale;
                if (ok) sp += (int64_t)page * p.c.scale_stride[0] + h * p.c.scale_stride[1] + (int64_t)(row0 + (lane & 15)) * p.c.scale_stride[2];
                cp_async4(ring + slot * C::stage + C::kbytes + C::vbytes + lane * 4, sp, ok ? 4 : 0);
            }
            ti += kCdWarps;
            page = page_of(ti);
        };
#pragma unroll
        for (int s = 0; s < C::stages - 1; ++s) {
            if (ti < t_end) issue(s);
            cp_async_commit();
        }
        int slot = 0;
        for (; t < t_end; t += kCdWarps) {
            cp_async_wait<C::stages - 2>();
            __syncwarp();       // the scales come from other lanes; and all lanes are done with the last slot
            if (ti < t_end) issue(slot == 0 ? C::stages - 1 : slot - 1);
            cp_async_commit();
            const uint32_t st = ring + slot * C::stage;

            // S^T: 16 keys x columns, in two halves of the contraction.
            float acc[NT][2][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[nt][0][i] = acc[nt][1][i] = 0.f;
#pragma unroll
            for (int e = 0; e < C::kch; ++e) {
                const uint4 x = lds128(st + e * 512 + lane * 16), y = lds128(st + (C::kch + e) * 512 + lane * 16);
                const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
                if constexpr (C::k8) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t a0 = codes_to_half2<DT, 0>(xw[i]), a1 = codes_to_half2<DT, 0>(yw[i]);
                        const uint32_t a2 = codes_to_half2<DT, 1>(xw[i]), a3 = codes_to_half2<DT, 1>(yw[i]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma16816<false>(acc[nt][i & 1], a0, a1, a2, a3, qf[nt][4 * e + i][0], qf[nt][4 * e + i][1]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma16816<BF16>(acc[nt][i], xw[2 * i], yw[2 * i], xw[2 * i + 1], yw[2 * i + 1], qf[nt][2 * e + i][0], qf[nt][2 * e + i][1]);
                }
            }
            float kscale[2] = {1.f, 1.f}, vscale[2] = {1.f, 1.f};
            if constexpr (C::k8) {
                const uint32_t ss = st + C::kbytes + C::vbytes + r * 4;
                kscale[0] = lds_f32(ss);
                kscale[1] = lds_f32(ss + 32);
                vscale[0] = lds_f32(ss + 64);
                vscale[1] = lds_f32(ss + 96);
            }
            // Scores in log2 units; x[nt][2 i + j]: key r + 8 i, column 2c + j.
            float x[NT][4];
            const int key = t * kTileKeys + r;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float s = acc[nt][0][i] + acc[nt][1][i];
                    if constexpr (C::k8) s *= kscale[i >> 1];
                    x[nt][i] = s * cs[nt][i & 1];
                }
            if (p.score_kind != 0) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        // cap tanh(y) = cap (1 - 2 / (e^2y + 1)); softcap_k takes x to 2 y log2 e.
                        if (p.score_kind & FA_SCORE_SOFTCAP) {
                            const float y = x[nt][i] * p.softcap_k;
                            x[nt][i] = p.softcap_log2 * (1.f - __fdividef(2.f, ex2_approx(y > 120.f ? 120.f : y) + 1.f));
                        }
                        if (p.score_kind & FA_SCORE_ALIBI)
                            x[nt][i] = fmaf(slope[nt][i & 1], (float)(key + 8 * (i >> 1) - (sr.len - 1)), x[nt][i]);
                    }
            }
            if (((bad >> slot) & 1u) || t * kTileKeys < sr.lo || (t + 1) * kTileKeys > sr.len) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int k = key + 8 * i;
                    if (((bad >> slot) & 1u) || k < sr.lo || k >= sr.len)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) x[nt][2 * i] = x[nt][2 * i + 1] = -INFINITY;
                }
            }
            bool raise = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) raise = raise || fmaxf(x[nt][j], x[nt][2 + j]) > m[nt][j] + kRaise;
            float vtop = 0.f;
            if constexpr (C::k8) {
                vtop = fmaxf(fabsf(vscale[0]), fabsf(vscale[1]));
                raise = raise || vtop > R;
            }
            if (__any_sync(kFullMask, raise)) {
                float beta = 1.f;
                if constexpr (C::k8) {
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) vtop = fmaxf(vtop, __shfl_xor_sync(kFullMask, vtop, off));
                    const uint32_t up = min((__float_as_uint(vtop) + 0x7fffffu) & 0x7f800000u, 0x7e800000u);   // at most 2^126
                    const float Rn = fmaxf(R, __uint_as_float(up));
                    const float inv = __uint_as_float(0x7f000000u - __float_as_uint(Rn));
                    beta = R * inv;
                    R = Rn;
                    inv_R = inv;
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float top = fmaxf(x[nt][j], x[nt][2 + j]);
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, off));
                        const float mn = fmaxf(m[nt][j], top);
                        const float alpha = ex2_approx(m[nt][j] - mn);
                        m[nt][j] = mn;
                        l[nt][j] *= alpha;
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            o[nt][k][j] *= alpha * beta;
                            o[nt][k][2 + j] *= alpha * beta;
                        }
                    }
            }
            // Weights, and their transpose as the second operand.
            uint32_t pb[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float w0 = ex2_approx(x[nt][2 * i] - m[nt][0]), w1 = ex2_approx(x[nt][2 * i + 1] - m[nt][1]);
                    l[nt][0] += w0;
                    l[nt][1] += w1;
                    if constexpr (C::k8) {
                        const float f = vscale[i] * inv_R;
                        w0 *= f;
                        w1 *= f;
                    }
                    pb[nt][i] = transpose8x8(pack2<BF16>(w0, w1));
                }
            // O^T += V^T P^T: rows are dims, lane (r, c) holds D / 8 of them for its four keys.
            const uint32_t vst = st + C::kbytes + lane * C::vb;
            if constexpr (C::k8) {
                uint32_t w[4][C::vb / 4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (C::vb == 16) {
                        const uint4 v = lds128(vst + i * 512);
                        w[i][0] = v.x, w[i][1] = v.y, w[i][2] = v.z, w[i][3] = v.w;
                    } else {
                        const uint2 v = lds64(vst + i * 256);
                        w[i][0] = v.x, w[i][1] = v.y;
                    }
                }
#pragma unroll
                for (int q = 0; q < C::vb / 4; ++q)
#pragma unroll
                    for (int hi = 0; hi < 2; ++hi) {
                        const uint32_t pa = __byte_perm(w[0][q], w[1][q], hi ? 0x7362 : 0x5140);   // keys 2c, 2c + 1
                        const uint32_t pc = __byte_perm(w[2][q], w[3][q], hi ? 0x7362 : 0x5140);   // keys 2c + 8, 2c + 9
                        const uint32_t a0 = codes_to_half2<DT, 0>(pa), a1 = codes_to_half2<DT, 1>(pa);
                        const uint32_t a2 = codes_to_half2<DT, 0>(pc), a3 = codes_to_half2<DT, 1>(pc);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma16816<false>(o[nt][2 * q + hi], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                    }
            } else {
#pragma unroll
                for (int e = 0; e < C::vch; ++e) {
                    uint32_t w[4][4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint4 v = lds128(vst + (i * C::vch + e) * 512);
                        w[i][0] = v.x, w[i][1] = v.y, w[i][2] = v.z, w[i][3] = v.w;
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t a0 = __byte_perm(w[0][q], w[1][q], 0x5410), a1 = __byte_perm(w[0][q], w[1][q], 0x7632);
                        const uint32_t a2 = __byte_perm(w[2][q], w[3][q], 0x5410), a3 = __byte_perm(w[2][q], w[3][q], 0x7632);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) mma16816<BF16>(o[nt][4 * e + q], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                    }
                }
            }
            slot = slot + 1 == C::stages ? 0 : slot + 1;
        }
        cp_async_wait<0>();
        __syncthreads();        // every warp is done with its ring: it now holds the join

        // Join of the warps: O rows, then m, l per (warp, column), then the factors.
        float* so = reinterpret_cast<float*>(smem);
        float* sm = so + kCdWarps * COLS * C::orow;
        float* sl = sm + kCdWarps * COLS;
        float* sf = sl + kCdWarps * COLS;           // [warp][column] factor of O, then [column] M, L
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int col = nt * 8 + 2 * c + j;
                float sum = l[nt][j];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(kFullMask, sum, off);
                if (r == 0) {
                    sm[warp * COLS + col] = m[nt][j];
                    sl[warp * COLS + col] = sum;
                    sf[warp * COLS + col] = R;
                }
                float* row = so + (warp * COLS + col) * C::orow;
#pragma unroll
                for (int k = 0; k < KS; k += 2) {
                    // dims 2k .. 2k + 3 of this lane's: contiguous within a segment of C::seg
                    const int d = 2 * k, dim = (d / C::seg) * 64 + r * C::seg + d % C::seg;
                    *reinterpret_cast<float4*>(row + dim + dim / C::seg * 4) = make_float4(o[nt][k][j], o[nt][k][2 + j], o[nt][k + 1][j], o[nt][k + 1][2 + j]);
                }
            }
        __syncthreads();
        float* sM = sf + kCdWarps * COLS;
        float* sL = sM + COLS;
        if (threadIdx.x < COLS) {
            const int col = threadIdx.x;
            float M = -FLT_MAX, L = 0.f;
#pragma unroll
            for (int w = 0; w < kCdWarps; ++w) M = fmaxf(M, sm[w * COLS + col]);
#pragma unroll
            for (int w = 0; w < kCdWarps; ++w) {
                const float f = ex2_approx(sm[w * COLS + col] - M);
                L = fmaf(sl[w * COLS + col], f, L);
                sf[w * COLS + col] *= f;
            }
            sM[col] = M;
            sL[col] = L;
        }
        __syncthreads();
        const bool complete = unit0 == 0 && seg_units == sr.units;
        // Pieces: a CTA's first segment in slot 2 cta, another in slot 2 cta + 1.
        const int64_t piece = 2 * (int64_t)blockIdx.x + (u == u_begin ? 0 : 1);
        float* po = p.partials + piece * COLS * (D + 2);
        for (int i = threadIdx.x; i < cols * (D / 4); i += kCdThreads) {
            const int col = i / (D / 4), dim = (i % (D / 4)) * 4;
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kCdWarps; ++w) {
                const float f = sf[w * COLS + col];
                const float4 v = *reinterpret_cast<const float4*>(so + (w * COLS + col) * C::orow + dim + dim / C::seg * 4);
                s.x = fmaf(v.x, f, s.x);
                s.y = fmaf(v.y, f, s.y);
                s.z = fmaf(v.z, f, s.z);
                s.w = fmaf(v.w, f, s.w);
            }
            if (complete) {
                const float L = sL[col], inv = L == 0.f ? 0.f : 1.f / L;
                uint2 w;
                if (q_bf16) w = make_uint2(pack2<true>(s.x * inv, s.y * inv), pack2<true>(s.z * inv, s.w * inv));
                else w = make_uint2(pack2<false>(s.x * inv, s.y * inv), pack2<false>(s.z * inv, s.w * inv));
                if (L == 0.f) w = make_uint2(0, 0);
                *reinterpret_cast<uint2*>(p.out + b * p.out_stride[0] + (int64_t)(hq0 + col) * p.out_stride[1] + dim) = w;
            } else {
                *reinterpret_cast<float4*>(po + col * D + dim) = s;
            }
        }
        if (threadIdx.x < cols) {
            const int col = threadIdx.x;
            const float M = sM[col], L = sL[col];
            if (!complete) {
                po[COLS * D + 2 * col] = M;
                po[COLS * D + 2 * col + 1] = L;
            } else if (p.lse) {
                p.lse[(int64_t)b * p.HQ + hq0 + col] = L == 0.f ? -INFINITY : (M + log2f(L)) * kCdLn2;
            }
        }
        // The next segment.
        u += seg_units;
        unit0 = 0;
        if (u < u_end && ++hr == HR) {
            hr = 0;
            do sr = seq_range(p, ++b); while (sr.units == 0);
        }
        __syncthreads();        // the join is read: the ring may be filled again
    }
}

// One CTA a (sequence, query head): joins the pieces of a head whose keys several CTAs shared, in
// key order; and writes the result of a sequence without keys.
template <int D>
__global__ void __launch_bounds__(kCdThreads) cache_decode_merge_kernel(const __grid_constant__ CacheDecodeParams p, bool q_bf16, int cols_pow, int ctas) {
    constexpr int LPR = D / 4, GROUPS = kCdThreads / LPR;
    __shared__ int64_t s_before;
    __shared__ __align__(16) float s_o[GROUPS][D];      // written as float4
    __shared__ float s_l[GROUPS], s_m[GROUPS];
    const int b = blockIdx.x / p.HQ, hq = blockIdx.x - b * p.HQ;
    const int CB = col_blocks(p.group, cols_pow), HR = p.c.H * CB;
    const int h = hq / p.group, g = hq - h * p.group;
    const int hr = h * CB + g / cols_pow, col = g % cols_pow;
    const SeqScan scan = scan_sequences<kCdThreads>(p);
    if (b >= scan.first && b < scan.last) {
        int64_t before = scan.before;
        for (int i = scan.first; i < b; ++i) before += seq_range(p, i).units;
        s_before = before;
    }
    __syncthreads();
    const int n = seq_range(p, b).units;
    const int64_t total = scan.total * HR, share = (total + ctas - 1) / ctas;
    const int64_t begin = s_before * HR + (int64_t)hr * n, end = begin + n;
    const int grp = threadIdx.x / LPR, d = (threadIdx.x % LPR) * 4;
    int64_t c0 = 0, c1 = -1;
    if (n > 0) {
        c0 = begin / share;
        c1 = (end - 1) / share;
        if (c0 == c1) return;   // one CTA had all its keys and wrote the result
    }
    // Each group of lanes joins every GROUPS-th piece.
    float M = -FLT_MAX, L = 0.f;
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int64_t k = c0 + grp; k <= c1; k += GROUPS) {
        const int64_t piece = 2 * k + (max(begin, k * share) == k * share ? 0 : 1);
        const float* po = p.partials + piece * cols_pow * (D + 2);
        const float m = po[cols_pow * D + 2 * col], l = po[cols_pow * D + 2 * col + 1];
        const float4 v = *reinterpret_cast<const float4*>(po + col * D + d);
        const float Mn = fmaxf(M, m), a = ex2_approx(M - Mn), f = ex2_approx(m - Mn);
        M = Mn;
        L = L * a + l * f;
        O = make_float4(O.x * a + v.x * f, O.y * a + v.y * f, O.z * a + v.z * f, O.w * a + v.w * f);
    }
    *reinterpret_cast<float4*>(&s_o[grp][d]) = O;
    if (d == 0) {
        s_m[grp] = M;
        s_l[grp] = L;
    }
    __syncthreads();
    float MM = -FLT_MAX, LL = 0.f;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) MM = fmaxf(MM, s_m[i]);
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) LL = fmaf(s_l[i], ex2_approx(s_m[i] - MM), LL);
    if (threadIdx.x < D) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) v = fmaf(s_o[i][threadIdx.x], ex2_approx(s_m[i] - MM), v);
        v = LL == 0.f ? 0.f : v / LL;
        p.out[b * p.out_stride[0] + (int64_t)hq * p.out_stride[1] + threadIdx.x] =
            (uint16_t)((q_bf16 ? pack2<true>(v, 0.f) : pack2<false>(v, 0.f)) & 0xFFFFu);
    }
    if (threadIdx.x == 0 && p.lse) p.lse[(int64_t)b * p.HQ + hq] = LL == 0.f ? -INFINITY : (MM + log2f(LL)) * kCdLn2;
}

constexpr int kMaxOcc = 4;
int columns(int group) { return group > 8 ? 16 : 8; }

template <int DT, int D, int NT>
cudaError_t launch_split(const CacheDecodeParams& p, bool q_bf16, int nsm, cudaStream_t st) {
    using C = CdConfig<DT, D, NT>;
    static_assert(C::occ <= kMaxOcc, "the workspace counts kMaxOcc CTAs an SM");
    auto kern = cache_decode_kernel<DT, D, NT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem);
    if (e != cudaSuccess) return e;
    const int grid = nsm * C::occ;
    kern<<<grid, kCdThreads, C::smem, st>>>(p, q_bf16);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    cache_decode_merge_kernel<D><<<(unsigned)(p.B * p.HQ), kCdThreads, 0, st>>>(p, q_bf16, 8 * NT, grid);
    return cudaGetLastError();
}

}  // namespace

int64_t cache_decode_workspace_bytes(int B, int HQ, int HK, int D, int nsm) {
    return (int64_t)2 * kMaxOcc * nsm * columns(HQ / HK) * (D + 2) * 4;
}

cudaError_t launch_cache_decode(const CacheDecodeParams& p, int dtype, int D, bool q_bf16, int nsm, cudaStream_t st) {
#define FA_CD(T, DD)              \
    if (dtype == T && D == DD)    \
        return columns(p.group) == 8 ? launch_split<T, DD, 1>(p, q_bf16, nsm, st) : launch_split<T, DD, 2>(p, q_bf16, nsm, st);
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
