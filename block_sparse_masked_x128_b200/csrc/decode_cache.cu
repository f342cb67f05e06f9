// decode_cache.cu -- attention of one new token a sequence over a paged, possibly quantised
// cache with grouped heads.
//
//   x_j = mod(scale * q . k_j),  p = softmax of x over max(0, len - window) <= j < len,
//   out = sum_j p_j v_j,  lse = log sum_j exp x_j        (no key: out 0, lse -inf)
//
// The work is reading K and V once, so HBM bounds it as long as nothing else is in the way:
//
//   Split      the keys of every (sequence, kv head) are cut into steps of 16 or 32, and the warps of
//              one wave of CTAs take equal runs of the list of all steps, so ragged lengths and
//              single long sequences load every SM alike.  The lengths are device data: each warp
//              finds its run by a scan over the sequences.  A run may go through several heads; the
//              loads run ahead across the border, so a warp's stream of copies never stops.  A head
//              whose steps are all one warp's is finished by it; otherwise the (m, l, O / l) of its
//              part goes to the workspace and the merge kernel joins the parts in key order (no
//              atomics: the same bits every time).  Warps share nothing and never wait.  Where
//              the tables map few tokens, a CTA takes a head alone instead and joins its warps' parts
//              in shared memory: one launch.
//   Heads      the query heads of a kv head are the columns of the products (8 or 16 at a time):
//              S^T = K q^T and O^T = V^T P^T, with 16 keys or 16 dims as rows.  The matrix
//              pipe is needed only because one cache byte meets up to 16 heads; at 8 columns
//              mma.sync keeps up with HBM several times over, and its operands come straight
//              from the loaded bytes.
//   Loads      each warp has a ring of its own in shared memory, filled with cp.async and read back
//              as fragments: the products' contraction index may run through the dims in any order,
//              so 16 contiguous bytes of a row serve a lane for four steps of it, and nothing but
//              the slots' order (below) is arranged.  No barrier between the warps.
//   8 bits     codes become fp16 exactly, in registers.  The key's scale multiplies its score, the
//              value's scale the weight, both in fp32.  q is brought into fp16's range by a power of
//              two a head: its elements keep all their bits down to 2^-28 of the head's largest, and
//              are off by 2^-39 of that below.
//   Softmax    l sums 2^(x_j - m) in fp32, and O sums w_j v_j with w_j = 2^(x_j - m); over 8-bit
//              caches w_j code_j with w_j = 2^(x_j - m) (vscale_j u), u a power of two that takes
//              the largest weight near 1, so neither sum depends on the size of the other's terms.
//              For the product a weight becomes two 16-bit numbers.  m is raised to the largest x_j
//              so far, and u set by the largest x_j + log2 vscale_j, only when a weight exceeds 2^8
//              (bf16 caches: m to 8 above the largest x_j, when one exceeds 1): most tiles need no
//              reduction over the lanes, and a weight is held to 2^-16 (bf16) or 2^-22 of itself or,
//              in fp16, 2^-25 of the largest, however the v scales differ.
//
// Measured (calls replayed in a graph, B200, copy rate 6.57 TB/s): 16 sequences x 16 heads of 1k-8k
// tokens, bf16, D = 128: 75 us, 6.1 TB/s; 96 sequences to 16384 tokens, 32 over 8 heads, bf16: 235 us,
// 6.35 TB/s; one of 131072 tokens, 32 over 8 heads, e4m3: 52 us, 5.3 TB/s, of them 4 us the merge; 16 of
// 1k-8k tokens, 64 over 8 heads, s8: 31 us; one of 257 tokens, by a CTA a head: 4.5 us.  Calls from
// Python take 1 to 4 us more.  Without its arithmetic the kernel takes some 3 us less at 8 bits, nothing
// less at 16.
#include "serving.h"
#include "sm100_ptx.cuh"

#include <algorithm>
#include <atomic>
#include <cfloat>

namespace fa {
namespace {

__device__ int32_t g_cache_decode_status;   // 2: a length or page out of range was met

constexpr int kCdWarps = 4, kCdThreads = 32 * kCdWarps;
constexpr int kTileKeys = 16;               // keys a warp takes at a time
constexpr float kCdLn2 = 0.6931471805599453f, kCdLog2e = 1.4426950408889634f;
// A weight above 2^8 raises the reference to the largest score; over a bf16 cache, whose values reach
// the end of fp32's range, one above 1 raises it to 8 above, so that a weight times a value fits.
template <int DT>
constexpr float kTopWeight = DT == FA_DTYPE_BF16 ? 1.f : 256.f;
template <int DT>
constexpr float kHeadroom = DT == FA_DTYPE_BF16 ? 8.f : 0.f;
// Value scales count as 2^-126 to 2^126 in the unit u of O, which is 2^126 to 2^-126 then: every scale
// that a written row can have, and zeros as fresh pools hold them.
constexpr float kMaxScaleLog2 = 126.f;

template <int DT, int D, int NT>
struct CdConfig {
    static constexpr bool k8 = CacheType<DT>::k8;
    static constexpr int bytes = CacheType<DT>::bytes;
    static constexpr int kch = D * bytes / 64;            // 16-byte K chunks a lane and row
    static constexpr int vb = D / 8 * bytes < 16 ? 8 : 16;  // bytes of a V chunk
    static constexpr int vch = D / 8 * bytes / vb;        // V chunks a lane and row
    static constexpr int lpr = D * bytes >= 128 ? 8 : 4;  // lanes that copy a row's line
    // Copy j brings rows krow + k_row(j), and of a two-line row the line k_line(j).
    static constexpr int lines = D * bytes == 256 ? 2 : 1;
    static __device__ constexpr int k_row(int j) { return j / lines * (32 / lpr); }
    static __device__ constexpr int k_line(int j) { return j % lines; }
    static __device__ constexpr int k_dst(int j) { return (k_row(j) >> 3) * kch * 512 + (k_row(j) & 7) * 64 + k_line(j) * 1024; }
    static __device__ constexpr int v_odd(int j) { return vb == 16 ? (j / lines) & 1 : 0; }
    static __device__ constexpr int v_dst(int j) { return vb == 16 ? (j / lines >> 1) * 2 * vch * 512 + k_line(j) * 512 : j * 512; }
    static constexpr int copies = 2 * kch;                // of 512 bytes, a tile's K or V
    static constexpr int kbytes = 2 * kch * 512;          // 2 rows a lane
    static constexpr int vbytes = 4 * vch * 32 * vb;      // 4 rows a lane
    static constexpr int tile = kbytes + vbytes + (k8 ? 128 : 0);
    // Tiles a warp works on at once: two independent chains of products and half the loop's
    // overhead, where the ring has room for it (131072 tokens of e4m3 in a graph, when it took 52 us
    // too: with one tile 53.3 at three CTAs an SM and 55.3 at four; with two CTAs and deeper rings 53.3).
    static constexpr int sub = D * bytes == 256 ? 1 : 2;
    static constexpr int stage = sub * tile;
    static constexpr int occ = NT == 1 ? 3 : 2;
    static constexpr int stages = (D * bytes == 64 ? 4 : 2) + (NT == 1 ? 0 : 1);
    static constexpr int smem = kCdWarps * stages * stage;
    static constexpr int seg = k8 && D == 128 ? 16 : 8;   // a lane's dims come in runs of this
    static constexpr int orow = D + D / seg * 4;
    static_assert(8 * NT * (kCdWarps * (orow + 2) + 1) * 4 <= smem, "join_and_write uses the rings' memory");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int n) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
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

// 2^k and k of 2^k, for integers -126 <= k <= 126.
__device__ __forceinline__ float power_of_two(float k) { return __uint_as_float((uint32_t)((int)k + 127) << 23); }
__device__ __forceinline__ float exponent_of(float u) { return (float)((int)(__float_as_uint(u) >> 23) - 127); }

// a with its magnitude at most that of the largest finite number; NaN stays NaN.
__device__ __forceinline__ float finite(float a) {
    float d;
    asm("min.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(FLT_MAX));
    return d;
}

// Two 16-bit values with infinities as the largest finite ones.
template <bool BF16>
__device__ __forceinline__ uint32_t finite2(uint32_t v) {
    uint32_t d;
    if constexpr (BF16) asm("min.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(0x7F7F7F7Fu));
    else asm("min.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(d) : "r"(v), "r"(0x7BFF7BFFu));
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

// The keys of sequence b that are attended to, [lo, len), from tile `tile` (of 16 keys) in `steps`
// steps of `sub` tiles.
struct SeqRange {
    int32_t lo, len, tile, steps;
};
__device__ __forceinline__ SeqRange seq_range(const CacheDecodeParams& p, int b, int sub) {
    SeqRange r;
    const int n = p.kv_lens[b];
    if ((unsigned)n > (unsigned)p.c.capacity) g_cache_decode_status = 2;
    r.len = max(0, min(n, p.c.capacity));
    r.lo = p.window > 0 ? max(0, r.len - p.window) : 0;
    r.tile = r.lo / kTileKeys;
    r.steps = r.len > r.lo ? ((r.len + kTileKeys - 1) / kTileKeys - r.tile + sub - 1) / sub : 0;
    return r;
}

// Division of counts of steps: 32 bits wherever they fit, which they do unless terabytes are read.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
    return (uint64_t)(a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// A warp's run of steps.  The list of steps goes by (sequence, kv head, step); `runs` warps take
// `share` steps each.
struct Run {
    int32_t seq, head, step;    // where the run begins
    int64_t first, last;        // its steps, [first, last)
    int64_t share;
};
__device__ __forceinline__ Run find_run(const CacheDecodeParams& p, int sub, int64_t which, int64_t runs) {
    const int lane = threadIdx.x & 31;
    const int n = (p.B + 31) / 32;
    const int b0 = min(p.B, lane * n), b1 = min(p.B, b0 + n);
    int64_t mine = 0;
#pragma unroll 4
    for (int b = b0; b < b1; ++b) mine += seq_range(p, b, sub).steps;
    mine *= p.c.H;
    int64_t before = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t v = __shfl_up_sync(kFullMask, before, off);
        if (lane >= off) before += v;
    }
    const int64_t total = __shfl_sync(kFullMask, before, 31);
    before -= mine;
    Run r;
    r.share = divide(total + runs - 1, runs);
    r.first = r.share * which;
    r.last = min(total, r.first + r.share);
    r.seq = -1;
    r.head = r.step = 0;
    if (r.first < r.last && r.first >= before && r.first < before + mine) {
        for (int b = b0; b < b1; ++b) {
            const int steps = seq_range(p, b, sub).steps;
            const int64_t k = (int64_t)steps * p.c.H;
            if (r.first < before + k) {
                r.seq = b;
                r.head = (int)divide(r.first - before, steps);
                r.step = (int)(r.first - before - (int64_t)r.head * steps);
                break;
            }
            before += k;
        }
    }
    const unsigned owner = __ballot_sync(kFullMask, r.seq >= 0);
    const int from = owner ? __ffs(owner) - 1 : 0;
    r.seq = __shfl_sync(kFullMask, r.seq, from);
    r.head = __shfl_sync(kFullMask, r.head, from);
    r.step = __shfl_sync(kFullMask, r.step, from);
    return r;
}

// cap tanh(y) of x = cap y, both in log2 units; k = 2 / cap takes x to 2 y log2 e.  From |y| = 1/4 on it
// is cap (1 - 2 / (e^2y + 1)), which is off by some 2^-23 of cap; below, x times the series of
// tanh(y) / y (its next term: 2^-26), so that scores far below a large cap keep their bits.
__device__ __forceinline__ float soft_cap(float x, float k, float cap_log2) {
    const float z = x * k, u = z * z * 0.12011325347955035f;       // u = y^2
    const float series = fmaf(fmaf(fmaf(0.021869488f, u, -0.053968254f), u, 0.13333333f), u, -0.33333333f);
    const float far = cap_log2 * (1.f - __fdividef(2.f, ex2_approx(z > 120.f ? 120.f : z) + 1.f));
    return fabsf(z) < 0.72f ? fmaf(x * u, series, x) : far;
}

// The head groups of a kv head: columns of the products, `rows` of them at a time.
__host__ __device__ constexpr int col_blocks(int group, int cols) { return (group + cols - 1) / cols; }

// Dims 2k .. 2k + 3 of lane (r, c)'s: contiguous within a run of `seg`.
template <int SEG>
__device__ __forceinline__ int lane_dim(int r, int k) {
    return 2 * k / SEG * 64 + r * SEG + 2 * k % SEG;
}

// What takes a column's O to its average over the keys: 1 / l and 1 / u, apart because either may be
// as small as fp32 goes (no key: 0).
struct Average {
    float inv, unit;
    __device__ __forceinline__ float operator()(float o) const { return o * inv * unit; }
};
__device__ __forceinline__ Average average(float l, float u) {
    return {l == 0.f ? 0.f : __fdividef(1.f, l), power_of_two(-exponent_of(u))};
}

// Joins the parts (m, l, average) of the CTA's warps in shared memory (over the rings, which are done
// with) and writes the result.
template <int DT, int D, int NT, bool QBF>
__device__ __forceinline__ void join_and_write(const CacheDecodeParams& p, uint8_t* smem, const float (&o)[NT][D / 16][4], const float (&m)[NT][2],
                                               const float (&unit)[NT][2], const float (&l)[NT][2], int b, int hq0, int cols) {
    using C = CdConfig<DT, D, NT>;
    constexpr int COLS = 8 * NT;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, c = lane & 3;
    float* so = reinterpret_cast<float*>(smem);     // [warp][column] rows of D floats, 4 more after each run (bank conflicts)
    float* sm = so + kCdWarps * COLS * C::orow;     // [warp][column] m, then the average's share
    float* sl = sm + kCdWarps * COLS;               // [warp][column] l
    float* sL = sl + kCdWarps * COLS;               // [column] L
    cp_async_wait<0>();
    __syncthreads();
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
            }
            const Average av = average(sum, unit[nt][j]);
            float* row = so + (warp * COLS + col) * C::orow;
#pragma unroll
            for (int k = 0; k < D / 16; k += 2) {
                const int dim = lane_dim<C::seg>(r, k);
                *reinterpret_cast<float4*>(row + dim + dim / C::seg * 4) =
                    make_float4(av(o[nt][k][j]), av(o[nt][k][2 + j]), av(o[nt][k + 1][j]), av(o[nt][k + 1][2 + j]));
            }
        }
    __syncthreads();
    if (threadIdx.x < COLS) {
        const int col = threadIdx.x;
        float M = -FLT_MAX, L = 0.f;
#pragma unroll
        for (int w = 0; w < kCdWarps; ++w) M = fmaxf(M, sm[w * COLS + col]);
#pragma unroll
        for (int w = 0; w < kCdWarps; ++w) {
            const float f = sl[w * COLS + col] * ex2_approx(sm[w * COLS + col] - M);
            L += f;
            sm[w * COLS + col] = f;
        }
        const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
        for (int w = 0; w < kCdWarps; ++w) sm[w * COLS + col] *= inv;
        sL[col] = L;
        if (col < cols && p.lse) p.lse[(int64_t)b * p.HQ + hq0 + col] = L == 0.f ? -INFINITY : (M + log2f(L)) * kCdLn2;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < cols * (D / 4); i += kCdThreads) {
        const int col = i / (D / 4), dim = (i % (D / 4)) * 4;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kCdWarps; ++w) {
            const float f = sm[w * COLS + col];
            const float4 v = *reinterpret_cast<const float4*>(so + (w * COLS + col) * C::orow + dim + dim / C::seg * 4);
            s = make_float4(fmaf(v.x, f, s.x), fmaf(v.y, f, s.y), fmaf(v.z, f, s.z), fmaf(v.w, f, s.w));
        }
        uint2 w = make_uint2(pack2<QBF>(s.x, s.y), pack2<QBF>(s.z, s.w));
        if (sL[col] == 0.f) w = make_uint2(0, 0);
        *reinterpret_cast<uint2*>(p.out + b * p.out_stride[0] + (int64_t)(hq0 + col) * p.out_stride[1] + dim) = w;
    }
}

// WHOLE: a CTA takes all the keys of a (sequence, kv head, block of columns), its warps every fourth
// step, and joins its warps' parts itself: one launch, for tables that map few tokens.  QBF: q and the
// result are bf16.
template <int DT, int D, int NT, bool WHOLE, bool QBF>
__global__ void __launch_bounds__(kCdThreads, CdConfig<DT, D, NT>::occ)
cache_decode_kernel(const __grid_constant__ CacheDecodeParams p) {
    using C = CdConfig<DT, D, NT>;
    constexpr bool BF16 = DT == FA_DTYPE_BF16;      // type of the products (8-bit: fp16)
    constexpr int KS = D / 16;                      // contraction steps of K q^T, and row tiles of O^T
    constexpr int COLS = 8 * NT;
    extern __shared__ __align__(128) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, c = lane & 3;

    grid_dependency_wait();
    const int CB = col_blocks(p.group, COLS);
    int worker = 0, mine = 0, cb;
    Run run;
    if constexpr (WHOLE) {
        const int kv = blockIdx.x / CB;
        cb = blockIdx.x - kv * CB;
        run.seq = kv / p.c.H;
        run.head = kv - run.seq * p.c.H;
        run.step = warp;
        run.first = 0;
        run.last = max(0, (seq_range(p, run.seq, C::sub).steps - warp + kCdWarps - 1) / kCdWarps);
    } else {
        // With more query heads than columns, neighbouring warps take the same run for one block of
        // columns each, so the keys are read from HBM once.
        worker = blockIdx.x * kCdWarps + warp;
        mine = worker / CB;
        cb = worker - mine * CB;
        run = find_run(p, C::sub, mine, (int)(gridDim.x * kCdWarps) / CB);
        if (run.seq < 0) return;
    }
    constexpr int kTiles = WHOLE ? kCdWarps * C::sub : C::sub;      // from a warp's step to its next
    const int col0 = cb * COLS, cols = min(COLS, p.group - col0);

    const uint32_t ring = smem_u32(smem) + warp * C::stages * C::stage;
    const int64_t kv_row = p.c.stride[2] * C::bytes, page_bytes = p.c.stride[0] * C::bytes;
    const int page_mask = (1 << p.c.page_shift) - 1;
    // Copies go by whole 128-byte lines, eight consecutive lanes a line (a 64-byte row: four), into
    // the slots of the lanes whose fragments the bytes are.  The slots' order makes the writes and
    // the reads of each quarter warp hit all banks once; with lanes of a line apart, or slots in
    // plain lane order, the copies alone ran at 5.4 TB/s instead of 7.3.
    const int krow = lane / C::lpr, kpiece = lane % C::lpr;
    const int64_t lane_off = krow * kv_row + kpiece * 16;
    const uint8_t* k_lane = static_cast<const uint8_t*>(p.c.k) + lane_off;
    const uint8_t* v_lane = static_cast<const uint8_t*>(p.c.v) + lane_off;
    // K: chunk e of rows r, r + 8 at lane (r ^ (e & 1), c)'s place.
    const uint32_t k_slot = (kpiece >> 2) * 512 + ((krow ^ (kpiece >> 2)) * 4 + (kpiece & 3)) * 16;
    // V: 16 bytes of row 2c at place 8 c + (r ^ 2c), for even and odd copies; 8 bytes at 16-byte
    // place 4 (c ^ odd row) + (r / 2 ^ 2 (c / 2)).
    uint32_t v_slot[2], v_read[2];
    if constexpr (C::vb == 16) {
        const int cl = lane >> 4;
#pragma unroll
        for (int odd = 0; odd < 2; ++odd)
            v_slot[odd] = ((lane >> 3) & 1) * C::vch * 512 + (2 * odd + cl) * 128 + (kpiece ^ (2 * cl) ^ (4 * odd)) * 16;
        v_read[0] = v_read[1] = (c * 8 + (r ^ (2 * c))) * 16;
    } else {
        const int odd = (lane >> 2) & 1;
        v_slot[0] = odd * 256 + ((lane >> 3) ^ odd) * 64 + (kpiece ^ (2 * (lane >> 4))) * 16;
        v_slot[1] = v_slot[0];
#pragma unroll
        for (int i = 0; i < 2; ++i) v_read[i] = (c ^ i) * 64 + ((r >> 1) ^ (2 * (c >> 1))) * 16 + (r & 1) * 8;
    }
    const uint32_t s_slot_of_lane = (lane & 7) * 16 + (lane >> 3) * 4;     // of row r: K r, K r + 8, V r, V r + 8
    const float* s_lane = lane < 16 ? p.c.k_scale : p.c.v_scale;      // lanes 0-15 K scales, 16-31 V scales
    if constexpr (C::k8) s_lane += (lane & 15) * p.c.scale_stride[2];

    // The loads' place: the next step to bring, which may be of a later head than the one at hand.
    struct {
        int b, h, tile, left;           // steps left of its head
        SeqRange sr;
        int32_t todo;                   // steps left of the run
        int64_t head_off, scale_off;    // the head's offset in a page
        const int32_t* table;
    } ld;
    ld.b = run.seq;
    ld.h = run.head;
    ld.sr = seq_range(p, ld.b, C::sub);
    ld.tile = ld.sr.tile + run.step * C::sub;
    ld.left = WHOLE ? (int)run.last : ld.sr.steps - run.step;
    ld.todo = (int)(run.last - run.first);
    int page[C::sub];                   // looked up one step ahead of their use
    auto look_up = [&]() {
#pragma unroll
        for (int u = 0; u < C::sub; ++u) {
            const int key0 = (ld.tile + u) * kTileKeys;
            page[u] = key0 < ld.sr.len ? ld.table[key0 >> p.c.page_shift] : 0;
        }
    };
    auto enter_head = [&]() {
        ld.head_off = ld.h * p.c.stride[1] * C::bytes;
        if constexpr (C::k8) ld.scale_off = ld.h * p.c.scale_stride[1];
        ld.table = p.c.table + (int64_t)ld.b * p.c.table_stride;
        look_up();
    };
    enter_head();
    uint32_t bad = 0;                   // tiles of the ring whose page is out of range
    auto issue_tile = [&](uint32_t st, int tile, int pg, uint32_t bit) {
        const int key0 = tile * kTileKeys, row0 = key0 & page_mask;
        const uint32_t ks = st + k_slot, vs = st + C::kbytes, ss = st + C::kbytes + C::vbytes + s_slot_of_lane;
        const bool good = (unsigned)pg < (unsigned)p.c.n_pages;
        const int64_t at = pg * page_bytes + row0 * kv_row + ld.head_off;
        const uint8_t *kp = k_lane + at, *vp = v_lane + at;
        const float* sp = s_lane;
        if constexpr (C::k8) sp += pg * p.c.scale_stride[0] + row0 * p.c.scale_stride[2] + ld.scale_off;
        if (good && key0 >= ld.sr.lo && key0 + kTileKeys <= ld.sr.len) {
            bad &= ~bit;
#pragma unroll
            for (int j = 0; j < C::copies; ++j) cp_async16(ks + C::k_dst(j), kp + C::k_row(j) * kv_row + C::k_line(j) * 128, 16);
#pragma unroll
            for (int j = 0; j < C::copies; ++j)
                cp_async16(vs + v_slot[C::v_odd(j)] + C::v_dst(j), vp + C::k_row(j) * kv_row + C::k_line(j) * 128, 16);
            if constexpr (C::k8) cp_async4(ss, sp, 4);
        } else {
            // Rows outside [lo, len), and a page outside the pool, are filled with zeros, not read.
            if (!good && lane == 0) g_cache_decode_status = 2;
            bad = good ? bad & ~bit : bad | bit;
            auto live = [&](int row) { return good && key0 + row >= ld.sr.lo && key0 + row < ld.sr.len; };
#pragma unroll
            for (int j = 0; j < C::copies; ++j) {
                const bool ok = live(krow + C::k_row(j));
                const int64_t off = C::k_row(j) * kv_row + C::k_line(j) * 128;
                cp_async16(ks + C::k_dst(j), ok ? kp + off : k_lane, ok ? 16 : 0);
                cp_async16(vs + v_slot[C::v_odd(j)] + C::v_dst(j), ok ? vp + off : v_lane, ok ? 16 : 0);
            }
            if constexpr (C::k8) {
                const bool ok = live(lane & 15);
                cp_async4(ss, ok ? sp : s_lane, ok ? 4 : 0);
            }
        }
    };
    auto issue = [&](int slot) {
        if (ld.todo > 0) {
#pragma unroll
            for (int u = 0; u < C::sub; ++u)
                issue_tile(ring + slot * C::stage + u * C::tile, ld.tile + u, page[u], 1u << (slot * C::sub + u));
            ld.tile += kTiles;
            if (--ld.todo > 0) {
                if (--ld.left > 0) {
                    look_up();
                } else {
                    if (++ld.h == p.c.H) {
                        ld.h = 0;
                        do ld.sr = seq_range(p, ++ld.b, C::sub); while (ld.sr.steps == 0);
                    }
                    ld.tile = ld.sr.tile;
                    ld.left = ld.sr.steps;
                    enter_head();
                }
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < C::stages - 1; ++s) issue(s);

    int b = run.seq, h = run.head, step0 = run.step, slot = 0;
    SeqRange sr = seq_range(p, b, C::sub);
    int64_t at = run.first;
    do {
        // This warp's part of the head: `steps` of its steps, from step0.
        const int steps = WHOLE ? (int)run.last : (int)min((int64_t)(sr.steps - step0), run.last - at);
        const int hq0 = h * p.group + col0;
        const bool complete = steps == sr.steps;

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
                        const float2 two = unpack2<QBF>(w[i]);
                        f[s][2 * i] = two.x;
                        f[s][2 * i + 1] = two.y;
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
                    slope[nt][j] = kCdLog2e * (p.alibi_slopes ? p.alibi_slopes[hq] : exp2f(-8.f * (float)(hq + 1) / (float)p.HQ));
                }
            }
        }
        float m[NT][2], ou[NT][2], l[NT][2], o[NT][KS][4];      // ou: the unit of O, 1 over 16-bit caches
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            m[nt][0] = m[nt][1] = -FLT_MAX;
            ou[nt][0] = ou[nt][1] = 1.f;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int t = 0; t < KS; ++t) o[nt][t][0] = o[nt][t][1] = o[nt][t][2] = o[nt][t][3] = 0.f;
        }
        int t = sr.tile + step0 * C::sub;       // first tile of the step at hand
        for (int i = 0; i < steps; ++i, t += kTiles) {
            cp_async_wait<C::stages - 2>();
            __syncwarp();       // other lanes' copies have landed too; and all lanes are done with the last slot
            issue(slot == 0 ? C::stages - 1 : slot - 1);
            const uint32_t st = ring + slot * C::stage;

            // S^T: 16 keys x columns a tile; with one tile in two halves of the contraction.
            constexpr int CHAINS = C::sub == 1 ? 2 : 1;
            float x[C::sub][NT][4], vscale[C::sub][2];
#pragma unroll
            for (int u = 0; u < C::sub; ++u) {
                const uint32_t su = st + u * C::tile;
                float acc[NT][CHAINS][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int k = 0; k < CHAINS; ++k) acc[nt][k][0] = acc[nt][k][1] = acc[nt][k][2] = acc[nt][k][3] = 0.f;
#pragma unroll
                for (int e = 0; e < C::kch; ++e) {
                    const uint32_t at = su + e * 512 + (lane * 16 ^ (e & 1) * 64);
                    const uint4 v0 = lds128(at), v1 = lds128(at + C::kch * 512);
                    const uint32_t xw[4] = {v0.x, v0.y, v0.z, v0.w}, yw[4] = {v1.x, v1.y, v1.z, v1.w};
                    if constexpr (C::k8) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t a0 = codes_to_half2<DT, 0>(xw[i]), a1 = codes_to_half2<DT, 0>(yw[i]);
                            const uint32_t a2 = codes_to_half2<DT, 1>(xw[i]), a3 = codes_to_half2<DT, 1>(yw[i]);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816<false>(acc[nt][i % CHAINS], a0, a1, a2, a3, qf[nt][4 * e + i][0], qf[nt][4 * e + i][1]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma16816<BF16>(acc[nt][i % CHAINS], xw[2 * i], yw[2 * i], xw[2 * i + 1], yw[2 * i + 1], qf[nt][2 * e + i][0], qf[nt][2 * e + i][1]);
                    }
                }
                // Scores in log2 units; x[2 i + j]: key r + 8 i, column 2c + j.  The key's scale meets
                // the column's factor first: the product of codes and scaled-up q alone may leave fp32.
                // (Where their own product leaves it, it counts as the largest number: a sum of 0 stays 0.)
                float kscale[2] = {1.f, 1.f};
                if constexpr (C::k8) {
                    const uint4 s4 = lds128(su + C::kbytes + C::vbytes + r * 16);
                    kscale[0] = __uint_as_float(s4.x), kscale[1] = __uint_as_float(s4.y);
                    vscale[u][0] = __uint_as_float(s4.z), vscale[u][1] = __uint_as_float(s4.w);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float s = acc[nt][0][i];
                        if constexpr (CHAINS == 2) s += acc[nt][1][i];
                        x[u][nt][i] = s * (C::k8 ? finite(kscale[i >> 1] * cs[nt][i & 1]) : cs[nt][i & 1]);
                    }
                const int key = (t + u) * kTileKeys + r;
                if (p.score_kind != 0) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (p.score_kind & FA_SCORE_SOFTCAP) x[u][nt][i] = soft_cap(x[u][nt][i], p.softcap_k, p.softcap_log2);
                            if (p.score_kind & FA_SCORE_ALIBI)
                                x[u][nt][i] = fmaf(slope[nt][i & 1], (float)(key + 8 * (i >> 1) - (sr.len - 1)), x[u][nt][i]);
                        }
                }
                const bool lost = (bad >> (slot * C::sub + u)) & 1u;
                if (lost || (t + u) * kTileKeys < sr.lo || (t + u + 1) * kTileKeys > sr.len) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int k = key + 8 * i;
                        if (lost || k < sr.lo || k >= sr.len)
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) x[u][nt][2 * i] = x[u][nt][2 * i + 1] = -INFINITY;
                    }
                }
            }
            // Weights against the present reference and unit; one that is too large changes them first.
            // (A scale times the unit that leaves fp32 belongs to a key below 2^-120 of the heaviest, or
            // to one that changes them.)
            float w[C::sub][NT][4], e2[C::sub][NT][4];
            auto weights = [&]() {
                bool high = false;
#pragma unroll
                for (int u = 0; u < C::sub; ++u)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float e = ex2_approx(x[u][nt][i] - m[nt][i & 1]);
                            e2[u][nt][i] = e;
                            w[u][nt][i] = C::k8 ? e * finite(vscale[u][i >> 1] * ou[nt][i & 1]) : e;
                            high = high || e > kTopWeight<DT> || (C::k8 && fabsf(w[u][nt][i]) > kTopWeight<DT>);
                        }
                return high;
            };
            if (__any_sync(kFullMask, weights())) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        // heavy: log2 of the heaviest weight with its scale, so far 1 / u at m.
                        float top = m[nt][j], heavy = m[nt][j] - exponent_of(ou[nt][j]);
#pragma unroll
                        for (int u = 0; u < C::sub; ++u)
#pragma unroll
                            for (int i = 0; i < 2; ++i) {
                                const float y = x[u][nt][2 * i + j];
                                top = fmaxf(top, y + kHeadroom<DT>);
                                if constexpr (C::k8) heavy = fmaxf(heavy, y + fminf(fmaxf(__log2f(fabsf(vscale[u][i])), -kMaxScaleLog2), kMaxScaleLog2));
                            }
#pragma unroll
                        for (int off = 4; off < 32; off <<= 1) {
                            top = fmaxf(top, __shfl_xor_sync(kFullMask, top, off));
                            if constexpr (C::k8) heavy = fmaxf(heavy, __shfl_xor_sync(kFullMask, heavy, off));
                        }
                        float shift = m[nt][j] - top;
                        l[nt][j] *= ex2_approx(shift);
                        m[nt][j] = top;
                        if constexpr (C::k8) {
                            const float k = fminf(fmaxf(floorf(top - heavy), -kMaxScaleLog2), kMaxScaleLog2);
                            shift += k - exponent_of(ou[nt][j]);
                            ou[nt][j] = power_of_two(k);
                        }
                        const float alpha = ex2_approx(shift);
#pragma unroll
                        for (int k = 0; k < KS; ++k) {
                            o[nt][k][j] *= alpha;
                            o[nt][k][2 + j] *= alpha;
                        }
                    }
                weights();
            }
#pragma unroll
            for (int u = 0; u < C::sub; ++u) {
                // The weights' transpose is the second operand.  A weight goes as two numbers, itself rounded
                // and the rest, so that the result's error is that of its own rounding: one bf16 number makes
                // it 1.3 times that, one fp16 number over 8-bit caches 1.5 times for fp16 results.  (The second
                // costs a grouped s8 decode 31.0 -> 32.0 us, 16-bit caches nothing.)  Over 16-bit caches a
                // positive weight's first number is positive (fp16's least, 2^-24, at least; the rest, which
                // may be negative, makes up for it) and alone meets infinite values, so that they stay infinite.
                uint32_t pb[2][NT][2];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        l[nt][0] += e2[u][nt][2 * i];
                        l[nt][1] += e2[u][nt][2 * i + 1];
                        auto first = [](float w) { return DT == FA_DTYPE_F16 && w > 0.f ? fmaxf(w, 0x1p-24f) : w; };
                        const uint32_t two = pack2<BF16>(first(w[u][nt][2 * i]), first(w[u][nt][2 * i + 1]));
                        pb[0][nt][i] = transpose8x8(two);
                        const float2 r2 = unpack2<BF16>(two);
                        pb[1][nt][i] = transpose8x8(pack2<BF16>(w[u][nt][2 * i] - r2.x, w[u][nt][2 * i + 1] - r2.y));
                    }
                // O^T += V^T P^T: rows are dims, lane (r, c) holds D / 8 of them for its four keys.
                const uint32_t vst = st + u * C::tile + C::kbytes;
                if constexpr (C::k8) {
                    uint32_t v[4][C::vb / 4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (C::vb == 16) {
                            const uint4 q4 = lds128(vst + v_read[0] + i * 512);
                            v[i][0] = q4.x, v[i][1] = q4.y, v[i][2] = q4.z, v[i][3] = q4.w;
                        } else {
                            const uint2 q2 = lds64(vst + v_read[i & 1] + i * 256);
                            v[i][0] = q2.x, v[i][1] = q2.y;
                        }
                    }
#pragma unroll
                    for (int q = 0; q < C::vb / 4; ++q)
#pragma unroll
                        for (int hi = 0; hi < 2; ++hi) {
                            const uint32_t pa = __byte_perm(v[0][q], v[1][q], hi ? 0x7362 : 0x5140);   // keys 2c, 2c + 1
                            const uint32_t pc = __byte_perm(v[2][q], v[3][q], hi ? 0x7362 : 0x5140);   // keys 2c + 8, 2c + 9
                            const uint32_t a0 = codes_to_half2<DT, 0>(pa), a1 = codes_to_half2<DT, 1>(pa);
                            const uint32_t a2 = codes_to_half2<DT, 0>(pc), a3 = codes_to_half2<DT, 1>(pc);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                for (int k = 0; k < 2; ++k) mma16816<false>(o[nt][2 * q + hi], a0, a1, a2, a3, pb[k][nt][0], pb[k][nt][1]);
                        }
                } else {
#pragma unroll
                    for (int e = 0; e < C::vch; ++e) {
                        uint32_t v[4][4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint4 q4 = lds128(vst + v_read[0] + (i * C::vch + e) * 512);
                            v[i][0] = q4.x, v[i][1] = q4.y, v[i][2] = q4.z, v[i][3] = q4.w;
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t a0 = __byte_perm(v[0][q], v[1][q], 0x5410), a1 = __byte_perm(v[0][q], v[1][q], 0x7632);
                            const uint32_t a2 = __byte_perm(v[2][q], v[3][q], 0x5410), a3 = __byte_perm(v[2][q], v[3][q], 0x7632);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma16816<BF16>(o[nt][4 * e + q], a0, a1, a2, a3, pb[0][nt][0], pb[0][nt][1]);
                            const uint32_t f0 = finite2<BF16>(a0), f1 = finite2<BF16>(a1), f2 = finite2<BF16>(a2), f3 = finite2<BF16>(a3);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt) mma16816<BF16>(o[nt][4 * e + q], f0, f1, f2, f3, pb[1][nt][0], pb[1][nt][1]);
                        }
                    }
                }
            }
            slot = slot + 1 == C::stages ? 0 : slot + 1;
        }
        if constexpr (WHOLE) {
            join_and_write<DT, D, NT, QBF>(p, smem, o, m, ou, l, b, hq0, cols);
            return;
        }
        // The part's (m, l, average), or the result.  A worker's first head has slot 2 worker, a later one
        // that it leaves unfinished slot 2 worker + 1.
        const int part = 2 * worker + (at == run.first ? 0 : 1);
        float* po = p.partials + (int64_t)part * COLS * (D + 2);
        if (step0 == 0 && lane == 0)        // for the merge: the head's parts and the first one's slot
            p.heads[((int64_t)b * p.c.H + h) * CB + cb] = make_int2(
                complete ? 1 : (int)divide(at + sr.steps - 1, run.share) - mine + 1, part);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int col = nt * 8 + 2 * c + j;
                float sum = l[nt][j];
#pragma unroll
                for (int off = 4; off < 32; off <<= 1) sum += __shfl_xor_sync(kFullMask, sum, off);
                if (col >= cols) continue;
                auto dim = [&](int k) { return lane_dim<C::seg>(r, k); };
                const Average av = average(sum, ou[nt][j]);
                auto four = [&](int k) { return make_float4(av(o[nt][k][j]), av(o[nt][k][2 + j]), av(o[nt][k + 1][j]), av(o[nt][k + 1][2 + j])); };
                if (!complete) {
#pragma unroll
                    for (int k = 0; k < KS; k += 2) *reinterpret_cast<float4*>(po + col * D + dim(k)) = four(k);
                    if (r == 0) *reinterpret_cast<float2*>(po + COLS * D + 2 * col) = make_float2(m[nt][j], sum);
                } else {
                    uint16_t* out = p.out + b * p.out_stride[0] + (int64_t)(hq0 + col) * p.out_stride[1];
#pragma unroll
                    for (int k = 0; k < KS; k += 2) {
                        const float4 v = four(k);
                        uint2 w = make_uint2(pack2<QBF>(v.x, v.y), pack2<QBF>(v.z, v.w));
                        if (sum == 0.f) w = make_uint2(0, 0);
                        *reinterpret_cast<uint2*>(out + dim(k)) = w;
                    }
                    if (r == 0 && p.lse) p.lse[(int64_t)b * p.HQ + hq0 + col] = sum == 0.f ? -INFINITY : (m[nt][j] + log2f(sum)) * kCdLn2;
                }
            }
        // The next head.
        at += steps;
        step0 = 0;
        if (at < run.last && ++h == p.c.H) {
            h = 0;
            do sr = seq_range(p, ++b, C::sub); while (sr.steps == 0);
        }
    } while (at < run.last);
    cp_async_wait<0>();
    grid_dependency_release();
}

// ---- the merge: joins the parts of a head whose keys several warps shared, in key order, and writes
// the result of a sequence without keys.  The parts are in L2, so latency is its cost: a group of
// D / 4 lanes takes every stride-th part, kAhead of them loaded at a time.

// O is the average of the keys so far, so that no sum of large values leaves fp32.
struct Joined {
    float M, L;
    float4 O;
};

// n of them, in the order of `get`: no step waits for another's exponential and quotient.
template <class Get>
__device__ __forceinline__ Joined join_all(int n, Get&& get) {
    Joined r = {-FLT_MAX, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int k = 0; k < n; ++k) r.M = fmaxf(r.M, get(k).M);
    for (int k = 0; k < n; ++k) r.L = fmaf(get(k).L, ex2_approx(get(k).M - r.M), r.L);
    const float inv = r.L == 0.f ? 0.f : __fdividef(1.f, r.L);
    for (int k = 0; k < n; ++k) {
        const Joined& a = get(k);
        const float f = a.L * ex2_approx(a.M - r.M) * inv;
        r.O = make_float4(fmaf(a.O.x, f, r.O.x), fmaf(a.O.y, f, r.O.y), fmaf(a.O.z, f, r.O.z), fmaf(a.O.w, f, r.O.w));
    }
    return r;
}

// A query head: its parts, the first one's slot (the others are the first slots of the following
// workers of its block of columns), and its column there.
struct MergeHead {
    int b, hq, col, parts, slot;
};
__device__ __forceinline__ MergeHead merge_head(const CacheDecodeParams& p, int i, int cols, int sub) {
    MergeHead m;
    m.b = i / p.HQ;
    m.hq = i - m.b * p.HQ;
    const int CB = col_blocks(p.group, cols), h = m.hq / p.group, g = m.hq - h * p.group, cb = g / cols;
    m.col = g - cb * cols;
    const int2 e = p.heads[((int64_t)m.b * p.c.H + h) * CB + cb];      // nobody's, where there are no keys
    const bool none = seq_range(p, m.b, sub).steps == 0;
    m.parts = none ? 0 : e.x;
    m.slot = e.y;
    return m;
}

template <int D, int kAhead>
__device__ __forceinline__ Joined join_parts(const CacheDecodeParams& p, const MergeHead& m, int cols, int first, int stride, int d) {
    const int64_t step = (int64_t)2 * col_blocks(p.group, cols);
    Joined r = {-FLT_MAX, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
    for (int k0 = first; k0 < m.parts; k0 += stride * kAhead) {
        float2 ml[kAhead];
        float4 v[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int k = k0 + i * stride;
            ml[i] = make_float2(-FLT_MAX, 0.f);
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (k < m.parts) {
                const float* po = p.partials + (k == 0 ? (int64_t)m.slot : (m.slot & ~1) + k * step) * cols * (D + 2);
                ml[i] = *reinterpret_cast<const float2*>(po + cols * D + 2 * m.col);
                v[i] = *reinterpret_cast<const float4*>(po + m.col * D + d);
            }
        }
        float M = r.M;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) M = fmaxf(M, ml[i].x);
        float a = r.L * ex2_approx(r.M - M), L = a;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            ml[i].y *= ex2_approx(ml[i].x - M);
            L += ml[i].y;
        }
        const float inv = L == 0.f ? 0.f : __fdividef(1.f, L);
        a *= inv;
        r = {M, L, make_float4(r.O.x * a, r.O.y * a, r.O.z * a, r.O.w * a)};
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const float f = ml[i].y * inv;
            r.O = make_float4(fmaf(v[i].x, f, r.O.x), fmaf(v[i].y, f, r.O.y), fmaf(v[i].z, f, r.O.z), fmaf(v[i].w, f, r.O.w));
        }
    }
    return r;
}

// The groups of LPR lanes of a warp together: every lane gets the whole of its dims.
template <int LPR>
__device__ __forceinline__ Joined join_warp(const Joined& r) {
    float M = r.M;
#pragma unroll
    for (int off = LPR; off < 32; off <<= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, off));
    const float l = r.L * ex2_approx(r.M - M);
    float L = l;
#pragma unroll
    for (int off = LPR; off < 32; off <<= 1) L += __shfl_xor_sync(kFullMask, L, off);
    const float f = L == 0.f ? 0.f : l * __fdividef(1.f, L);
    float4 O = make_float4(r.O.x * f, r.O.y * f, r.O.z * f, r.O.w * f);
#pragma unroll
    for (int off = LPR; off < 32; off <<= 1) {
        O.x += __shfl_xor_sync(kFullMask, O.x, off);
        O.y += __shfl_xor_sync(kFullMask, O.y, off);
        O.z += __shfl_xor_sync(kFullMask, O.z, off);
        O.w += __shfl_xor_sync(kFullMask, O.w, off);
    }
    return {M, L, O};
}

__device__ __forceinline__ void write_joined(const CacheDecodeParams& p, bool q_bf16, const MergeHead& m, const Joined& r, int d) {
    uint2 w = q_bf16 ? make_uint2(pack2<true>(r.O.x, r.O.y), pack2<true>(r.O.z, r.O.w)) : make_uint2(pack2<false>(r.O.x, r.O.y), pack2<false>(r.O.z, r.O.w));
    if (r.L == 0.f) w = make_uint2(0, 0);
    *reinterpret_cast<uint2*>(p.out + m.b * p.out_stride[0] + (int64_t)m.hq * p.out_stride[1] + d) = w;
    if (d == 0 && p.lse) p.lse[(int64_t)m.b * p.HQ + m.hq] = r.L == 0.f ? -INFINITY : (r.M + log2f(r.L)) * kCdLn2;
}

// SLICES CTAs of WARPS warps a head, D / SLICES dims each.
template <int D, int SLICES, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) cache_decode_merge_head_kernel(const __grid_constant__ CacheDecodeParams p, bool q_bf16, int cols, int sub) {
    constexpr int DS = D / SLICES, LPR = DS / 4;
    __shared__ Joined joined[WARPS][LPR];
    grid_dependency_wait();
    const MergeHead m = merge_head(p, blockIdx.x, cols, sub);
    if (m.parts == 1) return;       // its warp wrote the result
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, d = blockIdx.y * DS + (lane % LPR) * 4;
    Joined r = join_warp<LPR>(join_parts<D, 4>(p, m, cols, threadIdx.x / LPR, 32 * WARPS / LPR, d));
    if (lane < LPR) joined[warp][lane] = r;
    __syncthreads();
    if (threadIdx.x < LPR) write_joined(p, q_bf16, m, join_all(WARPS, [&](int w) -> const Joined& { return joined[w][threadIdx.x]; }), d);
}

// A CTA for all the query heads of a (sequence, kv head, block of columns): a thread joins four dims
// of one of them over every `groups`-th part.
constexpr int kBlockThreads = 256;
template <int D>
__global__ void __launch_bounds__(kBlockThreads) cache_decode_merge_block_kernel(const __grid_constant__ CacheDecodeParams p, bool q_bf16, int cols, int sub) {
    constexpr int LPR = D / 4;
    __shared__ Joined joined[kBlockThreads];
    grid_dependency_wait();
    const int CB = col_blocks(p.group, cols);
    const int2 e = p.heads[blockIdx.x];
    const int kv = blockIdx.x / CB, cb = blockIdx.x - kv * CB, b = kv / p.c.H, h = kv - b * p.c.H;
    const bool none = seq_range(p, b, sub).steps == 0;
    if (!none && e.x == 1) return;      // its warp wrote the result
    const int used = min(cols, p.group - cb * cols), items = used * LPR;
    const int groups = items < kBlockThreads ? kBlockThreads / items : 1;
    for (int i0 = 0; i0 < items; i0 += kBlockThreads) {
        const int i = i0 + (groups > 1 ? (int)threadIdx.x % items : (int)threadIdx.x), grp = groups > 1 ? threadIdx.x / items : 0;
        const int col = i / LPR, d = (i - col * LPR) * 4;
        const MergeHead m = {b, h * p.group + cb * cols + col, col, none ? 0 : e.x, e.y};
        Joined r = {-FLT_MAX, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
        if (i < items && grp < groups) r = join_parts<D, 4>(p, m, cols, grp, groups, d);
        if (groups > 1) {
            joined[threadIdx.x] = r;
            __syncthreads();
            if (grp == 0) r = join_all(groups, [&](int k) -> const Joined& { return joined[k * items + i]; });
        }
        if (i < items && grp == 0) write_joined(p, q_bf16, m, r, d);
    }
}

constexpr int kMaxOcc = 3;
int columns(int group) { return group > 8 ? 16 : 8; }

// The workspace: the table of heads, then the slots.
int64_t heads_bytes(int64_t B, int64_t HQ, int64_t HK) {
    const int group = (int)(HQ / HK);
    return (B * HK * col_blocks(group, columns(group)) * 8 + 15) / 16 * 16;
}

// The kernel, with its shared memory allowed once a device.
template <int DT, int D, int NT, bool WHOLE, bool QBF>
cudaError_t launch_kernel(const CacheDecodeParams& p, unsigned grid, cudaStream_t st) {
    using C = CdConfig<DT, D, NT>;
    auto kern = cache_decode_kernel<DT, D, NT, WHOLE, QBF>;
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !(ready.load(std::memory_order_relaxed) >> dev & 1)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem);
        if (e != cudaSuccess) return e;
        if (dev < 64) ready.fetch_or(1ull << dev, std::memory_order_relaxed);
    }
    return launch_early(kern, dim3(grid), dim3(kCdThreads), C::smem, st, p);
}

template <int DT, int D, int NT, bool QBF>
cudaError_t launch_split(CacheDecodeParams p, int nsm, cudaStream_t st) {
    using C = CdConfig<DT, D, NT>;
    static_assert(C::occ <= kMaxOcc, "the workspace counts kMaxOcc CTAs an SM");
    const int64_t blocks = (int64_t)p.B * p.c.H * col_blocks(p.group, 8 * NT);
    // Where the tables (or the window) leave few keys a head, a CTA each is faster than splitting and
    // merging: up to 512 keys (in a graph, 8 sequences of 100-200 tokens, 32 over 8 heads: 4.8 us
    // against 8.0; one of 500, 8 heads: 7.0 against 6.3, but outside a graph the split's second launch
    // takes 2.4 us more of the host), and up to 1024 where there is a head for every SM (32 of 500-1000:
    // 20 against 23; with 16 heads in all 14.8 against 11.5).
    const int keys = p.window > 0 ? std::min(p.window, p.c.capacity) : p.c.capacity;
    if (keys <= 512 || (keys <= 1024 && blocks >= nsm))
        return launch_kernel<DT, D, NT, true, QBF>(p, (unsigned)blocks, st);
    const int grid = nsm * C::occ;
    p.heads = static_cast<int2*>(p.workspace);
    p.partials = reinterpret_cast<float*>(static_cast<char*>(p.workspace) + heads_bytes(p.B, p.HQ, p.c.H));
    cudaError_t e = launch_kernel<DT, D, NT, false, QBF>(p, (unsigned)grid, st);
    if (e != cudaSuccess) return e;
    const int64_t heads = (int64_t)p.B * p.HQ;
    const int cols = 8 * NT, sub = C::sub;
    // The merge.  A head has workers / blocks parts on average, and what counts is how many loads
    // follow one another and how many CTAs start: few heads get four CTAs of 16 warps each, more get
    // four warps, and where heads are many, and their parts few, a CTA takes all the query heads of a
    // kv head (in a graph: 1024 heads of 14 parts 30 us with four warps a head, 33 with one; 5824
    // heads of one part 7.5 us by kv heads, 11.8 with four warps a query head).
    if (heads <= nsm)
        return launch_early(cache_decode_merge_head_kernel<D, 4, 16>, dim3((unsigned)heads, 4), dim3(512), 0, st, p, QBF, cols, sub);
    if (heads <= 12 * nsm)
        return launch_early(cache_decode_merge_head_kernel<D, 1, 4>, dim3((unsigned)heads), dim3(128), 0, st, p, QBF, cols, sub);
    return launch_early(cache_decode_merge_block_kernel<D>, dim3((unsigned)blocks), dim3(kBlockThreads), 0, st, p, QBF, cols, sub);
}

}  // namespace

int64_t cache_decode_workspace_bytes(int B, int HQ, int HK, int D, int nsm) {
    return heads_bytes(B, HQ, HK) + (int64_t)2 * kMaxOcc * kCdWarps * nsm * columns(HQ / HK) * (D + 2) * 4;
}

cudaError_t launch_cache_decode(const CacheDecodeParams& p, int dtype, int D, bool q_bf16, int nsm, cudaStream_t st) {
#define FA_CD(T, DD, BB)                        \
    if (dtype == T && D == DD && q_bf16 == BB)  \
        return columns(p.group) == 8 ? launch_split<T, DD, 1, BB>(p, nsm, st) : launch_split<T, DD, 2, BB>(p, nsm, st);
#define FA_CD_D(T, BB) FA_CD(T, 64, BB) FA_CD(T, 128, BB)
    FA_CD_D(FA_DTYPE_F16, false)
    FA_CD_D(FA_DTYPE_BF16, true)
    FA_CD_D(FA_DTYPE_E4M3, false)
    FA_CD_D(FA_DTYPE_E4M3, true)
    FA_CD_D(FA_DTYPE_S8, false)
    FA_CD_D(FA_DTYPE_S8, true)
#undef FA_CD_D
#undef FA_CD
    return cudaErrorInvalidValue;
}

cudaError_t cache_decode_status_word(int32_t** word) { return cudaGetSymbolAddress(reinterpret_cast<void**>(word), g_cache_decode_status); }

}  // namespace fa
