// kvcache.cuh -- the paged key/value cache as the kernels see it: slots,
// element types and the E4M3 quantiser, shared by cache.cu and attend.cu.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "dspark_common.cuh"

namespace dspark {

// An element of the E4M3 cache (the byte; its scale lies elsewhere).
struct e4m3 {
    unsigned char code;
};

// dspark_kv_cache by value, strides in elements.
struct KvView {
    unsigned char *k, *v;
    float *k_scale, *v_scale;
    const int32_t *table;
    long long page_stride, token_stride, head_stride;
    int n_pages, page_size, n_kv_heads, head_dim, n_requests, table_width;
};

// Where position p of request r lies: the page, or -1 when p, r or the table's
// entry is out of range.
__device__ __forceinline__ int kv_page(const KvView &c, int r, long long p, int *token) {
    if (r < 0 || r >= c.n_requests || p < 0) return -1;
    const long long col = div_nonneg(p, c.page_size);
    if (col >= c.table_width) return -1;
    *token = (int)(p - col * c.page_size);
    const int g = __ldg(c.table + (long long)r * c.table_width + col);
    return g >= 0 && g < c.n_pages ? g : -1;
}

__device__ __forceinline__ long long kv_offset(const KvView &c, int page, int token, int head) {
    return page * c.page_stride + token * c.token_stride + head * c.head_stride;
}

__device__ __forceinline__ long long kv_scale_offset(const KvView &c, int page, int token,
                                                     int head) {
    return ((long long)page * c.n_kv_heads + head) * c.page_size + token;
}

__device__ __forceinline__ float e4m3_value(unsigned char code) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(code, __NV_E4M3);
    return __half2float(__half(h));
}

__device__ __forceinline__ float elem_value(float x) { return x; }
__device__ __forceinline__ float elem_value(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float elem_value(e4m3 x) { return e4m3_value(x.code); }

__device__ __forceinline__ void elem_store(float *p, float x) { *p = x; }
__device__ __forceinline__ void elem_store(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }

// The scale of a head whose largest magnitude has the bits `amax` (unsigned
// order of |x|'s bits: NaN above infinity above the numbers, so either shows
// in the scale).  448 is the largest E4M3 value; the floor keeps the division
// below it in range for a head of zeros.
__device__ __forceinline__ float e4m3_scale(unsigned amax) {
    const float s = __fdiv_rn(__uint_as_float(amax), 448.0f);
    return s < 0x1p-100f ? 0x1p-100f : s;
}

// Two codes, x0 in the low byte: rounded to nearest even, saturated.
__device__ __forceinline__ unsigned e4m3_pair(float x0, float x1) {
    return __nv_cvt_float2_to_fp8x2(make_float2(x0, x1), __NV_SATFINITE, __NV_E4M3);
}

// The four E4M3 codes of a word as halves, the lower two and the upper: exact.
__device__ __forceinline__ void four_halves(unsigned codes, uint32_t *lower, uint32_t *upper) {
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n"
        " cvt.rn.f16x2.e4m3x2 %1, hi;\n}\n"
        : "=r"(*lower), "=r"(*upper)
        : "r"(codes));
}

__device__ __forceinline__ uint4 eight_halves(uint2 codes) {
    uint4 x;
    four_halves(codes.x, &x.x, &x.y);
    four_halves(codes.y, &x.z, &x.w);
    return x;
}

}  // namespace dspark

// ---------------------------------------------------------------- host side
namespace dspark {

inline int kv_elem_bytes(int dtype) {
    return dtype == DSPARK_DTYPE_BF16 ? 2 : (dtype == DSPARK_DTYPE_F32 ? 4 : 1);
}

// Host-side checks of a cache; DSPARK_OK or the call's error.
inline int kv_check(const dspark_kv_cache *c) {
    if (!c || !c->k || !c->v || !c->block_table) return DSPARK_ERR_INVALID_ARG;
    if (c->dtype != DSPARK_DTYPE_BF16 && c->dtype != DSPARK_DTYPE_F32 &&
        c->dtype != DSPARK_DTYPE_E4M3)
        return DSPARK_ERR_INVALID_ARG;
    if (c->dtype == DSPARK_DTYPE_E4M3 && (!c->k_scale || !c->v_scale))
        return DSPARK_ERR_INVALID_ARG;
    if (c->n_pages < 1 || c->page_size < 1 || c->n_kv_heads < 1 || c->n_requests < 1 ||
        c->table_width < 1 || c->page_stride < 0 || c->token_stride < 0 || c->head_stride < 0)
        return DSPARK_ERR_INVALID_ARG;
    if (c->head_dim < 2 || c->head_dim > DSPARK_MAX_HEAD_DIM || c->head_dim % 2)
        return DSPARK_ERR_UNSUPPORTED;
    return DSPARK_OK;
}

inline KvView kv_view(const dspark_kv_cache &c) {
    KvView w;
    w.k = static_cast<unsigned char *>(c.k);
    w.v = static_cast<unsigned char *>(c.v);
    w.k_scale = c.k_scale;
    w.v_scale = c.v_scale;
    w.table = c.block_table;
    w.page_stride = c.page_stride;
    w.token_stride = c.token_stride;
    w.head_stride = c.head_stride;
    w.n_pages = c.n_pages;
    w.page_size = c.page_size;
    w.n_kv_heads = c.n_kv_heads;
    w.head_dim = c.head_dim;
    w.n_requests = c.n_requests;
    w.table_width = c.table_width;
    return w;
}

}  // namespace dspark
