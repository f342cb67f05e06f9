// serving_api.cu -- the C ABI of the serving operators (include/fa_b200.h): rotary positions, the
// paged K/V cache and one-token attention over it.  Argument checks and launches; all checks come
// before any launch.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>

#include <nvtx3/nvToolsExt.h>

#include "serving.h"

namespace {

struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
};

fa_status_t fail(fa_status_t s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
fa_status_t fail(fa_status_t s, const char* fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    return fa::record_error(s, buf);
}

fa_status_t cuda_fail(cudaError_t e, const char* what) {
    return fail(FA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Query heads a kv head: a warp takes 16, and every block of them needs warps of its own.
constexpr int kMaxGroup = 1024;

// A pointer that the kernels read through, aligned to `align` bytes.
fa_status_t check_pointer(const void* ptr, size_t align, int dev, const char* name) {
    if ((reinterpret_cast<uintptr_t>(ptr) & (align - 1)) != 0)
        return fail(FA_ERR_INVALID_ARG, "%s is not %zu-byte aligned", name, align);
    return fa::check_device_memory(ptr, dev, name);
}

bool same_shape(const fa_tensor_t* a, const fa_tensor_t* b) {
    return a->B == b->B && a->H == b->H && a->S == b->S && a->D == b->D && a->dtype == b->dtype;
}

bool empty(const fa_tensor_t* t) { return t->B == 0 || t->H == 0 || t->S == 0; }

bool eight_bit(int32_t dtype) { return dtype == FA_DTYPE_E4M3 || dtype == FA_DTYPE_S8; }

// The checks of a cache and a page table that need no device; fills the kernels' view.
fa_status_t check_cache(const fa_kv_cache_t* c, const int32_t* table, int64_t table_stride, int64_t table_width,
                        int64_t B, fa::CacheView* view) {
    if (!c) return fail(FA_ERR_INVALID_ARG, "cache is NULL");
    if (c->dtype < FA_DTYPE_F16 || c->dtype > FA_DTYPE_S8)
        return fail(FA_ERR_INVALID_ARG, "cache.dtype %d is not a cache type", c->dtype);
    if (!c->k || !c->v) return fail(FA_ERR_INVALID_ARG, "cache.k and cache.v are required");
    if (((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v)) & 15u) != 0)
        return fail(FA_ERR_INVALID_ARG, "cache.k and cache.v must be 16-byte aligned");
    const bool e8 = eight_bit(c->dtype);
    if (e8 && (!c->k_scale || !c->v_scale))
        return fail(FA_ERR_INVALID_ARG, "an 8-bit cache needs k_scale and v_scale");
    if (c->page_size < 16 || c->page_size > 1024 || (c->page_size & (c->page_size - 1)) != 0)
        return fail(FA_ERR_UNSUPPORTED, "page_size %d: powers of two from 16 to 1024", c->page_size);
    if (c->n_pages <= 0 || c->n_pages > 0x7fffffffLL || c->H <= 0 || c->H > 65535)
        return fail(FA_ERR_INVALID_ARG, "cache extents (%lld pages, %lld heads) out of range", (long long)c->n_pages,
                    (long long)c->H);
    if (c->D != 64 && c->D != 128)
        return fail(FA_ERR_UNSUPPORTED, "head_dim %lld: only 64 and 128 are implemented", (long long)c->D);
    const int64_t vec = e8 ? 16 : 8;
    for (int i = 0; i < 3; ++i) {
        if (c->stride[i] <= 0 || c->stride[i] % vec != 0)
            return fail(FA_ERR_INVALID_ARG, "cache.stride[%d]=%lld must be a positive multiple of 16 bytes", i,
                        (long long)c->stride[i]);
        if (e8 && c->scale_stride[i] <= 0)
            return fail(FA_ERR_INVALID_ARG, "cache.scale_stride[%d] must be positive", i);
    }
    if (B > 65535) return fail(FA_ERR_UNSUPPORTED, "more than 65535 sequences");
    if (table_width < 0 || table_width > 0x7fffffffLL || table_stride < table_width)
        return fail(FA_ERR_INVALID_ARG, "page table of %lld columns with stride %lld", (long long)table_width,
                    (long long)table_stride);
    if (!table && table_width > 0 && B > 0) return fail(FA_ERR_INVALID_ARG, "page_table is NULL");
    view->k = c->k;
    view->v = c->v;
    view->k_scale = c->k_scale;
    view->v_scale = c->v_scale;
    for (int i = 0; i < 3; ++i) {
        view->stride[i] = c->stride[i];
        view->scale_stride[i] = c->scale_stride[i];
    }
    view->page_shift = 0;
    while ((1 << view->page_shift) < c->page_size) ++view->page_shift;
    view->n_pages = (int32_t)c->n_pages;
    view->H = (int32_t)c->H;
    view->table = table;
    view->table_stride = table_stride;
    view->table_width = (int32_t)table_width;
    // The kernels count tokens in 32 bits.
    const int64_t capacity = table_width << view->page_shift;
    view->capacity = (int32_t)(capacity < 0x7fffffc0 ? capacity : 0x7fffffc0);
    return FA_OK;
}

fa_status_t check_cache_memory(const fa_kv_cache_t* c, const fa::CacheView& v, int dev) {
    fa_status_t s;
    if ((s = fa::check_device_memory(c->k, dev, "cache.k")) != FA_OK) return s;
    if ((s = fa::check_device_memory(c->v, dev, "cache.v")) != FA_OK) return s;
    if (eight_bit(c->dtype)) {
        if ((s = check_pointer(c->k_scale, 4, dev, "cache.k_scale")) != FA_OK) return s;
        if ((s = check_pointer(c->v_scale, 4, dev, "cache.v_scale")) != FA_OK) return s;
    }
    if (v.table_width > 0 && (s = check_pointer(v.table, 4, dev, "page_table")) != FA_OK) return s;
    return FA_OK;
}

// Rows that go to or come from a cache: (B, H, S, D) pairs of one dtype that suits it.
fa_status_t check_rows(const fa_tensor_t* k, const fa_tensor_t* v, const char* kn, const char* vn) {
    fa_status_t s;
    if ((s = fa::check_tensor_arg(k, kn)) != FA_OK) return s;
    if ((s = fa::check_tensor_arg(v, vn)) != FA_OK) return s;
    if (!same_shape(k, v)) return fail(FA_ERR_INVALID_ARG, "%s and %s must share shape and dtype", kn, vn);
    return FA_OK;
}

fa_status_t rows_match_cache(const fa_tensor_t* k, const fa_kv_cache_t* c) {
    if (k->H != c->H || k->D != c->D) return fail(FA_ERR_INVALID_ARG, "rows and cache must share H and D");
    if (!eight_bit(c->dtype) && k->dtype != c->dtype)
        return fail(FA_ERR_INVALID_ARG, "a 16-bit cache takes and gives its own dtype");
    if (k->S > 0x7fffffffLL - 1024) return fail(FA_ERR_UNSUPPORTED, "more than 2^31 - 1024 rows a sequence");
    return FA_OK;
}

// Reads and clears the status words in one act each, so that what a kernel on another stream records
// meanwhile is either taken here or left for the next look.
__device__ int32_t g_status_taken;
__global__ void take_status_kernel(int32_t* rows, int32_t* decode) { g_status_taken = atomicExch(rows, 0) | atomicExch(decode, 0); }

cudaError_t take_status(cudaStream_t st, int32_t* out) {
    int32_t *rows = nullptr, *decode = nullptr;
    cudaError_t e = fa::cache_rows_status_word(&rows);
    if (e == cudaSuccess) e = fa::cache_decode_status_word(&decode);
    if (e != cudaSuccess) return e;
    static std::mutex mutex;        // one look at a time: g_status_taken is one word a device
    std::lock_guard<std::mutex> lock(mutex);
    take_status_kernel<<<1, 1, 0, st>>>(rows, decode);
    e = cudaGetLastError();
    if (e == cudaSuccess) e = cudaMemcpyFromSymbolAsync(out, g_status_taken, sizeof(*out), 0, cudaMemcpyDeviceToHost, st);
    return e == cudaSuccess ? cudaStreamSynchronize(st) : e;
}

fa_status_t current_device(int* dev) {
    const cudaError_t e = cudaGetDevice(dev);
    return e == cudaSuccess ? FA_OK : cuda_fail(e, "cudaGetDevice");
}

}  // namespace

extern "C" {

fa_status_t fa_rotary_frequencies(int32_t rot_dim, double base, const fa_rotary_scaling_t* sc, double* out) {
    if (rot_dim < 2 || rot_dim % 2 != 0) return fail(FA_ERR_INVALID_ARG, "rot_dim %d must be even and at least 2", rot_dim);
    if (!(base > 0) || !std::isfinite(base)) return fail(FA_ERR_INVALID_ARG, "base must be positive");
    if (!out) return fail(FA_ERR_INVALID_ARG, "frequencies is NULL");
    const int kind = sc ? sc->kind : FA_ROTARY_SCALE_NONE;
    if (kind < FA_ROTARY_SCALE_NONE || kind > FA_ROTARY_SCALE_BY_PARTS)
        return fail(FA_ERR_INVALID_ARG, "unknown scaling kind %d", kind);
    if (kind != FA_ROTARY_SCALE_NONE && (!(sc->factor > 0) || !std::isfinite(sc->factor)))
        return fail(FA_ERR_INVALID_ARG, "scaling needs a positive factor");
    if (kind == FA_ROTARY_SCALE_BASE) {
        if (rot_dim < 4) return fail(FA_ERR_INVALID_ARG, "a stretched base needs rot_dim >= 4");
        base *= std::pow(sc->factor, (double)rot_dim / (rot_dim - 2));
    }
    if (kind == FA_ROTARY_SCALE_BY_PARTS &&
        (!(sc->original_len > 0) || !(sc->low_turns >= 0) || !(sc->high_turns > sc->low_turns)))
        return fail(FA_ERR_INVALID_ARG, "scaling by parts needs original_len > 0 and 0 <= low_turns < high_turns");
    for (int i = 0; i < rot_dim / 2; ++i) {
        double f = std::pow(base, -2.0 * i / rot_dim);
        if (kind == FA_ROTARY_SCALE_LINEAR) f /= sc->factor;
        if (kind == FA_ROTARY_SCALE_BY_PARTS) {
            const double r = sc->original_len * f / 6.283185307179586477;
            const double g = std::fmin(1.0, std::fmax(0.0, (r - sc->low_turns) / (sc->high_turns - sc->low_turns)));
            f = f / sc->factor * (1.0 - g) + f * g;
        }
        out[i] = f;
    }
    return fa::record_ok();
}

fa_status_t fa_rotary(const fa_tensor_t* q, const fa_tensor_t* k, const int32_t* positions,
                      int64_t position_stride, int64_t position0, const double* frequencies,
                      int32_t rot_dim, int32_t layout, float factor, int32_t inverse,
                      fa_tensor_t* q_out, fa_tensor_t* k_out, void* stream) {
    NvtxRange nvtx_range("fa_rotary");
    fa_status_t s;
    if ((s = check_rows(q, q_out, "q", "q_out")) != FA_OK) return s;
    if ((k == nullptr) != (k_out == nullptr)) return fail(FA_ERR_INVALID_ARG, "k and k_out go together");
    if (k && (s = check_rows(k, k_out, "k", "k_out")) != FA_OK) return s;
    if (k && (k->B != q->B || k->S != q->S || k->D != q->D || k->dtype != q->dtype))
        return fail(FA_ERR_INVALID_ARG, "q and k must share B, S, D and dtype");
    if (q->D % 8 != 0 || q->D > 1024)
        return fail(FA_ERR_UNSUPPORTED, "head_dim %lld: multiples of 8 up to 1024", (long long)q->D);
    if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > q->D)
        return fail(FA_ERR_INVALID_ARG, "rot_dim %d must be even, from 2 to head_dim", rot_dim);
    if (layout != FA_ROTARY_HALF && layout != FA_ROTARY_INTERLEAVED)
        return fail(FA_ERR_INVALID_ARG, "unknown layout %d", layout);
    if (position_stride < 0) return fail(FA_ERR_INVALID_ARG, "position_stride must not be negative");
    const fa_tensor_t* in[2] = {q, k};
    const fa_tensor_t* out[2] = {q_out, k_out};
    for (int i = 0; i < (k ? 2 : 1); ++i)
        if (in[i]->data == out[i]->data && std::memcmp(in[i]->stride, out[i]->stride, sizeof(in[i]->stride)) != 0)
            return fail(FA_ERR_INVALID_ARG, "in-place rotation needs input and output to share strides");
    const int64_t heads = q->H + (k ? k->H : 0);
    if (q->B > 0x7fffffff || q->S > 0x7fffffff || heads > 0x7fffffff || q->B * q->S > 0x7fffffff)
        return fail(FA_ERR_UNSUPPORTED, "more than 2^31 - 1 tokens or heads");
    if (q->B == 0 || q->S == 0 || heads == 0) return fa::record_ok();
    if (!frequencies) return fail(FA_ERR_INVALID_ARG, "frequencies is NULL");
    int dev = 0;
    if ((s = current_device(&dev)) != FA_OK) return s;
    const char* names[2] = {"q", "k"};
    for (int i = 0; i < (k ? 2 : 1); ++i) {
        if (empty(in[i])) continue;
        if ((s = fa::check_device_memory(in[i]->data, dev, names[i])) != FA_OK) return s;
        if (out[i]->data != in[i]->data && (s = fa::check_device_memory(out[i]->data, dev, i ? "k_out" : "q_out")) != FA_OK)
            return s;
    }
    if ((s = check_pointer(frequencies, 8, dev, "frequencies")) != FA_OK) return s;
    if (positions && (s = check_pointer(positions, 4, dev, "positions")) != FA_OK) return s;
    const int nsm = fa::device_sm_count(dev);
    if (nsm <= 0) return fail(FA_ERR_CUDA, "could not read the SM count");
    fa::RotaryParams p;
    std::memset(&p, 0, sizeof(p));
    p.in_place = 1;
    for (int i = 0; i < (k ? 2 : 1); ++i) {
        p.x[i] = static_cast<const uint16_t*>(in[i]->data);
        p.y[i] = static_cast<uint16_t*>(out[i]->data);
        p.H[i] = (int32_t)in[i]->H;
        if (p.x[i] != p.y[i]) p.in_place = 0;
        for (int j = 0; j < 3; ++j) {
            p.xs[i][j] = in[i]->stride[j];
            p.ys[i][j] = out[i]->stride[j];
        }
    }
    p.B = (int32_t)q->B;
    p.S = (int32_t)q->S;
    p.D = (int32_t)q->D;
    p.half = rot_dim / 2;
    p.pos = positions;
    p.pos_stride = position_stride;
    p.pos0 = position0;
    p.freq = frequencies;
    p.factor = factor;
    p.inverse = inverse != 0;
    const cudaError_t e = fa::launch_rotary(p, q->dtype == FA_DTYPE_BF16, layout == FA_ROTARY_INTERLEAVED, nsm,
                                            static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? fa::record_ok() : cuda_fail(e, "rotary launch");
}

fa_status_t fa_cache_append(const fa_tensor_t* k, const fa_tensor_t* v, const fa_kv_cache_t* cache,
                            const int32_t* page_table, int64_t table_stride, int64_t table_width,
                            const int32_t* start, const int32_t* count, void* stream) {
    NvtxRange nvtx_range("fa_cache_append");
    fa_status_t s;
    fa::CacheRowsParams p;
    std::memset(&p, 0, sizeof(p));
    if ((s = check_rows(k, v, "k", "v")) != FA_OK) return s;
    if ((s = check_cache(cache, page_table, table_stride, table_width, k->B, &p.c)) != FA_OK) return s;
    if ((s = rows_match_cache(k, cache)) != FA_OK) return s;
    if (empty(k)) return fa::record_ok();
    if (!start) return fail(FA_ERR_INVALID_ARG, "start is NULL");
    int dev = 0;
    if ((s = current_device(&dev)) != FA_OK) return s;
    if ((s = fa::check_device_memory(k->data, dev, "k")) != FA_OK) return s;
    if ((s = fa::check_device_memory(v->data, dev, "v")) != FA_OK) return s;
    if ((s = check_cache_memory(cache, p.c, dev)) != FA_OK) return s;
    if ((s = check_pointer(start, 4, dev, "start")) != FA_OK) return s;
    if (count && (s = check_pointer(count, 4, dev, "count")) != FA_OK) return s;
    const fa_tensor_t* in[2] = {k, v};
    for (int i = 0; i < 2; ++i) {
        p.in[i] = static_cast<const uint16_t*>(in[i]->data);
        for (int j = 0; j < 3; ++j) p.rs[i][j] = in[i]->stride[j];
    }
    p.B = (int32_t)k->B;
    p.S = (int32_t)k->S;
    p.start = start;
    p.limit = count;
    const cudaError_t e = fa::launch_cache_append(p, cache->dtype, (int)cache->D, k->dtype == FA_DTYPE_BF16,
                                                  static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? fa::record_ok() : cuda_fail(e, "cache append launch");
}

fa_status_t fa_cache_read(const fa_kv_cache_t* cache, const int32_t* page_table, int64_t table_stride,
                          int64_t table_width, const int32_t* start, const int32_t* kv_lens,
                          fa_tensor_t* k_out, fa_tensor_t* v_out, void* stream) {
    NvtxRange nvtx_range("fa_cache_read");
    fa_status_t s;
    fa::CacheRowsParams p;
    std::memset(&p, 0, sizeof(p));
    if ((s = check_rows(k_out, v_out, "k_out", "v_out")) != FA_OK) return s;
    if ((s = check_cache(cache, page_table, table_stride, table_width, k_out->B, &p.c)) != FA_OK) return s;
    if ((s = rows_match_cache(k_out, cache)) != FA_OK) return s;
    if (empty(k_out)) return fa::record_ok();
    if (!kv_lens) return fail(FA_ERR_INVALID_ARG, "kv_lens is NULL");
    int dev = 0;
    if ((s = current_device(&dev)) != FA_OK) return s;
    if ((s = fa::check_device_memory(k_out->data, dev, "k_out")) != FA_OK) return s;
    if ((s = fa::check_device_memory(v_out->data, dev, "v_out")) != FA_OK) return s;
    if ((s = check_cache_memory(cache, p.c, dev)) != FA_OK) return s;
    if ((s = check_pointer(kv_lens, 4, dev, "kv_lens")) != FA_OK) return s;
    if (start && (s = check_pointer(start, 4, dev, "start")) != FA_OK) return s;
    const fa_tensor_t* out[2] = {k_out, v_out};
    for (int i = 0; i < 2; ++i) {
        p.out[i] = static_cast<uint16_t*>(out[i]->data);
        for (int j = 0; j < 3; ++j) p.rs[i][j] = out[i]->stride[j];
    }
    p.B = (int32_t)k_out->B;
    p.S = (int32_t)k_out->S;
    p.start = start;
    p.limit = kv_lens;
    const cudaError_t e = fa::launch_cache_read(p, cache->dtype, (int)cache->D, k_out->dtype == FA_DTYPE_BF16,
                                                static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? fa::record_ok() : cuda_fail(e, "cache read launch");
}

size_t fa_decode_workspace_bytes(int64_t B, int64_t HQ, int64_t H, int64_t D) {
    if (B <= 0 || HQ <= 0 || H <= 0 || HQ % H != 0 || B > 65535 || HQ > 65535 || HQ / H > kMaxGroup || (D != 64 && D != 128)) return 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return (size_t)fa::cache_decode_workspace_bytes((int)B, (int)HQ, (int)H, (int)D, fa::device_sm_count(dev));
}

fa_status_t fa_decode(const fa_tensor_t* q, const fa_kv_cache_t* cache, const int32_t* page_table,
                      int64_t table_stride, int64_t table_width, const int32_t* kv_lens, int32_t window,
                      uint32_t score_mod_kind, const fa_score_params_t* params, float scale,
                      fa_tensor_t* out, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
    NvtxRange nvtx_range("fa_decode");
    fa_status_t s;
    fa::CacheDecodeParams p;
    std::memset(&p, 0, sizeof(p));
    if ((s = check_rows(q, out, "q", "out")) != FA_OK) return s;
    if ((s = check_cache(cache, page_table, table_stride, table_width, q->B, &p.c)) != FA_OK) return s;
    if (q->S != 1) return fail(FA_ERR_INVALID_ARG, "q must hold one token a sequence (S = 1), got %lld", (long long)q->S);
    if (q->D != cache->D) return fail(FA_ERR_INVALID_ARG, "q and cache must share D");
    if (q->H % cache->H != 0 || q->H > 65535)
        return fail(FA_ERR_INVALID_ARG, "%lld query heads are no multiple of %lld kv heads", (long long)q->H, (long long)cache->H);
    if (q->H / cache->H > kMaxGroup || q->B * q->H > 0x7fffffffLL)
        return fail(FA_ERR_UNSUPPORTED, "more than %d query heads a kv head, or 2^31 - 1 heads in all", kMaxGroup);
    if (!eight_bit(cache->dtype) && q->dtype != cache->dtype)
        return fail(FA_ERR_INVALID_ARG, "a 16-bit cache takes queries of its own dtype");
    if (window < 0) return fail(FA_ERR_INVALID_ARG, "window must not be negative");
    const uint32_t known = FA_SCORE_SOFTCAP | FA_SCORE_ALIBI;
    if (score_mod_kind & ~known) return fail(FA_ERR_INVALID_ARG, "unknown score_mod_kind bits 0x%x", score_mod_kind);
    if ((score_mod_kind & FA_SCORE_SOFTCAP) && (!params || !(params->softcap > 0.f)))
        return fail(FA_ERR_INVALID_ARG, "soft-cap needs params->softcap > 0");
    if (empty(q)) return fa::record_ok();
    if (!kv_lens) return fail(FA_ERR_INVALID_ARG, "kv_lens is NULL");
    int dev = 0;
    if ((s = current_device(&dev)) != FA_OK) return s;
    const size_t need = fa_decode_workspace_bytes(q->B, q->H, cache->H, q->D);
    if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 15u))
        return fail(FA_ERR_INVALID_ARG, "workspace must be 16-byte aligned device memory of at least %zu bytes", need);
    if ((s = fa::check_device_memory(q->data, dev, "q")) != FA_OK) return s;
    if ((s = fa::check_device_memory(out->data, dev, "out")) != FA_OK) return s;
    if ((s = check_cache_memory(cache, p.c, dev)) != FA_OK) return s;
    if ((s = check_pointer(kv_lens, 4, dev, "kv_lens")) != FA_OK) return s;
    if (lse && (s = check_pointer(lse, 4, dev, "lse")) != FA_OK) return s;
    if ((s = fa::check_device_memory(workspace, dev, "workspace")) != FA_OK) return s;
    if (params && params->alibi_slopes && (s = check_pointer(params->alibi_slopes, 4, dev, "alibi_slopes")) != FA_OK) return s;
    const int nsm = fa::device_sm_count(dev);
    if (nsm <= 0) return fail(FA_ERR_CUDA, "could not read the SM count");
    const double log2e = 1.4426950408889634;
    const double sc = scale > 0.f ? (double)scale : 1.0 / std::sqrt((double)q->D);
    const double cap = (score_mod_kind & FA_SCORE_SOFTCAP) ? (double)params->softcap : 1.0;
    p.q = static_cast<const uint16_t*>(q->data);
    p.out = static_cast<uint16_t*>(out->data);
    for (int i = 0; i < 2; ++i) {
        p.q_stride[i] = q->stride[i];
        p.out_stride[i] = out->stride[i];
    }
    p.lse = lse;
    p.B = (int32_t)q->B;
    p.HQ = (int32_t)q->H;
    p.group = (int32_t)(q->H / cache->H);
    p.kv_lens = kv_lens;
    p.window = window;
    p.scale_log2 = (float)(sc * log2e);
    p.softcap_log2 = (float)(cap * log2e);
    p.softcap_k = (float)std::fmin(2.0 / cap, 3.4028234663852886e38);     // of a subnormal cap
    p.alibi_slopes = params ? params->alibi_slopes : nullptr;
    p.score_kind = (int32_t)score_mod_kind;
    p.workspace = workspace;
    const cudaError_t e = fa::launch_cache_decode(p, cache->dtype, (int)q->D, q->dtype == FA_DTYPE_BF16, nsm,
                                                  static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? fa::record_ok() : cuda_fail(e, "decode launch");
}

fa_status_t fa_cache_status(void* stream) {
    int32_t taken = 0;
    const cudaError_t e = take_status(static_cast<cudaStream_t>(stream), &taken);
    if (e != cudaSuccess) return cuda_fail(e, "reading the cache status words");
    if (taken != 0)
        return fail(FA_ERR_INVALID_ARG, "a page index, position or length was out of range");
    return fa::record_ok();
}

}  // extern "C"
