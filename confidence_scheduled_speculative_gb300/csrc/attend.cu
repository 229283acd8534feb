// attend.cu -- attention of a verify window's drafted tokens over the paged
// cache that holds their requests' prefixes and the tokens themselves.
//
// For packed row i (token t of request r's window, query head h, kv head
// h / G, G query heads a kv head) over the positions p it sees, the prefix
// and the window tokens of its ancestor bits:
//   s_p = scale q . k_p,  m = max s_p,  l = sum exp(s_p - m)
//   out = sum exp(s_p - m) v_p / l,     lse = m + ln l
//
// attend_any_kernel   any types, strides, head and page sizes, in 32 bits
//   throughout: a CTA a (row, query head), its four warps take every fourth
//   position, each with a running maximum and sum, joined at the end.

#include "kvcache.cuh"

namespace dspark {

constexpr int kAnyWarps = 4;
constexpr int kAnySteps = DSPARK_MAX_HEAD_DIM / 32;

struct AttendArgs {
    const void *q;
    long long ld_q;
    void *out;
    long long ld_out;
    float *lse;
    const int32_t *cu, *prefix;
    const uint32_t *ancestors;
    int B, n_q_heads, max_rows;
    float scale;
    KvView cache;
    int32_t *status;
};

// Request r's window: rows [*row0, *row0 + *len) and prefix *P.  False when it
// has none or one that cannot be used (flagged by the caller that asks for it).
__device__ __forceinline__ bool window_of(const AttendArgs &a, int r, int *row0, int *len, int *P,
                                          bool report) {
    const int lo = __ldg(a.cu + r), hi = __ldg(a.cu + r + 1);
    *row0 = lo;
    *len = hi - lo;
    *P = __ldg(a.prefix + r);
    if (hi == lo) return false;
    int bad = 0;
    if (lo < 0 || hi < lo || hi - lo > DSPARK_MAX_WINDOW || hi > a.max_rows)
        bad = DSPARK_STATUS_BAD_LEN;
    else if (*P < 0 || (long long)*P + *len > (long long)a.cache.table_width * a.cache.page_size)
        bad = DSPARK_STATUS_BAD_INDEX;
    if (bad && report) flag(a.status, bad);
    return !bad;
}

// The window tokens that token i of a window sees, as bits.
__device__ __forceinline__ unsigned ancestors_of(const AttendArgs &a, int row, int i, int len) {
    const unsigned all = 0xFFFFFFFFu >> (32 - len);
    return (a.ancestors ? __ldg(a.ancestors + row) : 0xFFFFFFFFu >> (31 - i)) & all;
}

template <typename T, typename C>
__global__ void __launch_bounds__(kAnyWarps * 32) attend_any_kernel(AttendArgs a) {
    __shared__ float part_o[kAnyWarps][DSPARK_MAX_HEAD_DIM];
    __shared__ float part_m[kAnyWarps], part_l[kAnyWarps];
    pdl_trigger();
    pdl_wait();
    const int row = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int D = a.cache.head_dim;
    if (row >= __ldg(a.cu + a.B)) return;
    int lo = 0, hi = a.B - 1;  // the last request that starts at or before the row
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(a.cu + mid) <= row) lo = mid;
        else hi = mid - 1;
    }
    const int r = lo;
    int row0, len, P;
    if (!window_of(a, r, &row0, &len, &P, threadIdx.x == 0) || row < row0) return;
    const unsigned bits = ancestors_of(a, row, row - row0, len);
    const int kh = h / (a.n_q_heads / a.cache.n_kv_heads);

    const T *q = static_cast<const T *>(a.q) + row * a.ld_q + (long long)h * D;
    float qv[kAnySteps], o[kAnySteps], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int t = 0; t < kAnySteps; ++t) {
        const int d = lane + 32 * t;
        qv[t] = d < D ? elem_value(q[d]) * a.scale : 0.0f;
        o[t] = 0.0f;
    }
    for (int p = warp; p < P + len; p += kAnyWarps) {
        if (p >= P && !(bits >> (p - P) & 1)) continue;
        int token;
        const int page = kv_page(a.cache, r, p, &token);
        if (page < 0) {
            if (lane == 0) flag(a.status, DSPARK_STATUS_BAD_INDEX);
            continue;
        }
        const long long at = kv_offset(a.cache, page, token, kh);
        const C *k = reinterpret_cast<const C *>(a.cache.k) + at;
        const C *v = reinterpret_cast<const C *>(a.cache.v) + at;
        float ks = 1.0f, vs = 1.0f;
        if (sizeof(C) == 1) {
            const long long s = kv_scale_offset(a.cache, page, token, kh);
            ks = __ldg(a.cache.k_scale + s);
            vs = __ldg(a.cache.v_scale + s);
        }
        float s = 0.0f, vv[kAnySteps];
#pragma unroll
        for (int t = 0; t < kAnySteps; ++t) {
            const int d = lane + 32 * t;
            vv[t] = d < D ? elem_value(v[d]) * vs : 0.0f;
            if (d < D) s = fmaf(qv[t], elem_value(k[d]) * ks, s);
        }
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(kFullMask, s, x);
        const float mn = fmaxf(m, s);
        const float base = mn == -INFINITY ? 0.0f : mn;
        const float keep = expf(m - base), w = expf(s - base);
        l = l * keep + w;
#pragma unroll
        for (int t = 0; t < kAnySteps; ++t) o[t] = o[t] * keep + w * vv[t];
        m = mn;
    }
#pragma unroll
    for (int t = 0; t < kAnySteps; ++t)
        if (lane + 32 * t < D) part_o[warp][lane + 32 * t] = o[t];
    if (lane == 0) {
        part_m[warp] = m;
        part_l[warp] = l;
    }
    __syncthreads();
    float M = -INFINITY, L = 0.0f, f[kAnyWarps];
#pragma unroll
    for (int w = 0; w < kAnyWarps; ++w) M = fmaxf(M, part_m[w]);
    const float base = M == -INFINITY ? 0.0f : M;
#pragma unroll
    for (int w = 0; w < kAnyWarps; ++w) {
        f[w] = expf(part_m[w] - base);
        L += part_l[w] * f[w];
    }
    T *out = static_cast<T *>(a.out) + row * a.ld_out + (long long)h * D;
    for (int d = threadIdx.x; d < D; d += kAnyWarps * 32) {
        float x = 0.0f;
#pragma unroll
        for (int w = 0; w < kAnyWarps; ++w) x += part_o[w][d] * f[w];
        elem_store(out + d, L == 0.0f ? 0.0f : x / L);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[(long long)row * a.n_q_heads + h] = L == 0.0f ? -INFINITY : base + logf(L);
}

template <typename T>
cudaError_t launch_any(const AttendArgs &a, int cache_dtype, cudaStream_t stream) {
    const dim3 grid(a.max_rows, a.n_q_heads), block(kAnyWarps * 32);
    if (cache_dtype == DSPARK_DTYPE_BF16)
        return launch_pdl(attend_any_kernel<T, __nv_bfloat16>, grid, block, 0, stream, a);
    if (cache_dtype == DSPARK_DTYPE_F32)
        return launch_pdl(attend_any_kernel<T, float>, grid, block, 0, stream, a);
    return launch_pdl(attend_any_kernel<T, e4m3>, grid, block, 0, stream, a);
}

}  // namespace dspark

using namespace dspark;

extern "C" size_t dspark_tree_attention_workspace_bytes(int32_t n_q_heads, int32_t head_dim) {
    if (n_q_heads < 1 || head_dim < 2 || head_dim > DSPARK_MAX_HEAD_DIM) return 0;
    return 256;
}

extern "C" int dspark_tree_attention(const void *q, int64_t ld_q, int32_t dtype, int32_t n_q_heads,
                                     int32_t max_rows, const int32_t *cu_seqlens,
                                     const int32_t *prefix_lens, int32_t B,
                                     const uint32_t *ancestors, float scale,
                                     const dspark_kv_cache *cache, void *out, int64_t ld_out,
                                     float *lse, void *workspace, size_t workspace_bytes,
                                     int32_t *status, void *stream) {
    const int rc = kv_check(cache);
    if (rc != DSPARK_OK) return rc;
    if (!q || !out || !cu_seqlens || !prefix_lens || !status || max_rows < 0 || B < 1 ||
        B > cache->n_requests || n_q_heads < 1 || n_q_heads % cache->n_kv_heads)
        return DSPARK_ERR_INVALID_ARG;
    if (dtype != DSPARK_DTYPE_BF16 && dtype != DSPARK_DTYPE_F32) return DSPARK_ERR_INVALID_ARG;
    const int64_t width = (int64_t)n_q_heads * cache->head_dim;
    if (ld_q < width || ld_out < width) return DSPARK_ERR_INVALID_ARG;
    if (!(scale - scale == 0.0f)) return DSPARK_ERR_INVALID_ARG;
    if (n_q_heads > 65535) return DSPARK_ERR_UNSUPPORTED;
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < dspark_tree_attention_workspace_bytes(n_q_heads, cache->head_dim))
        return DSPARK_ERR_WORKSPACE;
    if (max_rows == 0) return DSPARK_OK;
    AttendArgs a;
    a.q = q;
    a.ld_q = ld_q;
    a.out = out;
    a.ld_out = ld_out;
    a.lse = lse;
    a.cu = cu_seqlens;
    a.prefix = prefix_lens;
    a.ancestors = ancestors;
    a.B = B;
    a.n_q_heads = n_q_heads;
    a.max_rows = max_rows;
    a.scale = scale;
    a.cache = kv_view(*cache);
    a.status = status;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == DSPARK_DTYPE_BF16
                              ? launch_any<__nv_bfloat16>(a, cache->dtype, st)
                              : launch_any<float>(a, cache->dtype, st);
    return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
