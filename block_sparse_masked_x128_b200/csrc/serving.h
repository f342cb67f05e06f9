// serving.h -- structures shared by the host side (serving_api.cu) and the kernels of the
// serving operators: rotary positions, the paged K/V cache, and one-token attention over it.
#pragma once

#include "fa_internal.h"

#ifdef __CUDACC__
#include <cuda_fp16.h>
#endif

namespace fa {

// Checks of api.cu that every entry point shares.
fa_status_t check_tensor_arg(const fa_tensor_t* t, const char* name);
int device_sm_count(int device);
fa_status_t check_device_memory(const void* ptr, int dev, const char* name);

// Codes of the cache's element types (the FA_DTYPE_* values of the header).
template <int DT>
struct CacheType {
    static constexpr bool k8 = DT == FA_DTYPE_E4M3 || DT == FA_DTYPE_S8;
    static constexpr int bytes = k8 ? 1 : 2;
};

struct RotaryParams {
    const uint16_t* x[2];         // q and k (k may be absent: H[1] = 0)
    uint16_t* y[2];
    int64_t xs[2][3], ys[2][3];   // B, H, S strides in elements
    int32_t H[2];
    int32_t B, S, D, half;        // half = rotated pairs a row
    const int32_t* pos;           // [B][pos_stride] or null (then pos0 + s)
    int64_t pos_stride, pos0;
    const double* freq;           // [half] radians a position
    float factor;
    int32_t inverse, in_place;
    // Set by launch_rotary.
    int64_t pos_token_stride;
    int32_t tokens_per_cta, ctas_per_seq;
};
cudaError_t launch_rotary(const RotaryParams& p, bool bf16, bool interleaved, int nsm, cudaStream_t st);

// A paged cache as the kernels see it.
struct CacheView {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    int64_t stride[3];            // page, head, row, in elements
    int64_t scale_stride[3];
    int32_t page_shift, n_pages, H;
    const int32_t* table;         // [B][table_stride] page of each block of the sequence
    int64_t table_stride;
    int32_t table_width;
    int32_t capacity;             // tokens that a row of the table maps, at most 2^31 - 64
};

struct CacheRowsParams {
    CacheView c;
    const uint16_t* in[2];        // append: new k and v rows
    uint16_t* out[2];             // read: the sequences' rows
    int64_t rs[2][3];             // strides of in / out: B, H, S
    int32_t B, S;
    const int32_t* start;         // [B] position of row 0, or null (0)
    const int32_t* limit;         // append: [B] number of new rows or null (S); read: [B] lengths
};
cudaError_t launch_cache_append(const CacheRowsParams& p, int dtype, int D, bool bf16, cudaStream_t st);
cudaError_t launch_cache_read(const CacheRowsParams& p, int dtype, int D, bool bf16, cudaStream_t st);
cudaError_t cache_rows_status_word(int32_t** word);      // on the current device

struct CacheDecodeParams {
    CacheView c;
    const uint16_t* q;
    uint16_t* out;
    int64_t q_stride[2], out_stride[2];   // B, H
    float* lse;                   // [B][HQ] or null
    int32_t B, HQ, group;         // group = query heads a kv head
    const int32_t* kv_lens;       // [B]
    int32_t window;               // 0: all keys
    float scale_log2, softcap_log2, softcap_k;   // softcap_k: 2 / softcap
    const float* alibi_slopes;
    int32_t score_kind;
    void* workspace;
    // Set by launch_cache_decode.
    int2* heads;                  // [B][H][column blocks] parts and the first one's slot
    float* partials;              // slots of averages [cols][D], then (m, l) [cols]
};
int64_t cache_decode_workspace_bytes(int B, int HQ, int HK, int D, int nsm);
cudaError_t launch_cache_decode(const CacheDecodeParams& p, int dtype, int D, bool q_bf16, int nsm, cudaStream_t st);
cudaError_t cache_decode_status_word(int32_t** word);

#ifdef __CUDACC__
// The kernels of these operators are short and follow one another: each is launched so that it may
// start before its predecessor on the stream ends, and its first act is to wait for that end
// (with all the predecessor's writes) before it reads or writes anything.  What overlaps is the
// launch.  The predecessor may write what they read (positions, lengths, tables, rows) while they
// are already on the SMs, so they load it as memory that changes, not by __ldg, whose data must stay
// the same for a kernel's whole life.  A kernel that comes to grid_dependency_release in all its
// blocks lets its successor start there rather than at its own end.
__device__ __forceinline__ void grid_dependency_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_dependency_release() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class... Params, class... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Two 16-bit values as fp32, the low half first.
template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return make_float2(__half2float(__ushort_as_half((unsigned short)(w & 0xFFFFu))), __half2float(__ushort_as_half((unsigned short)(w >> 16))));
}

// The page of position `pos` (32 bits without sign) by a sequence's row of the table, or -1 where
// the row does not reach it or names a page outside the pool.
__device__ __forceinline__ int cache_page(const CacheView& c, const int32_t* table, uint32_t pos) {
    if (pos >= (uint32_t)c.capacity) return -1;
    const int page = table[pos >> c.page_shift];
    return (unsigned)page < (unsigned)c.n_pages ? page : -1;
}
#endif

}  // namespace fa
