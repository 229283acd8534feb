// prompt.cu -- causal attention of ragged prompts over keys and values of every head,
// with a key part that all heads share: the expanded form over a latent cache's rows.
//
// Query i of n over m keys sees keys j <= m - n + i.  With q = [q_k | q_s], of kv head g:
//   s_j = scale (q_k . k_jg + q_s . k_shared_j),  mx = max s_j,  l = sum exp(s_j - mx)
//   out = sum exp(s_j - mx) v_jg / l,             lse = mx + ln l
//
// prompt_any_kernel   any types, strides and dimensions, in 32 bits throughout: a CTA a
//   (row, query head), its four warps take every fourth key, each with a running maximum
//   and sum, joined at the end.

#include "kvcache.cuh"

namespace dspark {

struct PromptArgs {
    const void *q, *k, *shared, *v;
    long long ld_q, ld_k, hs_k, ld_shared, ld_v, hs_v;
    void *out;
    long long ld_out;
    float *lse;
    const int32_t *cu, *cu_k;
    int B, n_q_heads, group, key_dim, shared_dim, value_dim, max_rows, max_keys;
    float scale;
    int32_t *status;
};

// A request's queries [lo, hi) and keys [k0, k1).
struct PromptRange {
    int lo, hi, k0, k1;
};

__device__ __forceinline__ PromptRange load_range(const PromptArgs &a, int r) {
    return {__ldg(a.cu + r), __ldg(a.cu + r + 1), __ldg(a.cu_k + r), __ldg(a.cu_k + r + 1)};
}

// Whether a range has queries and can be used; with `report`, flags why not.
__device__ __forceinline__ bool usable(const PromptArgs &a, const PromptRange &w, bool report) {
    if (w.hi == w.lo) return false;
    const bool bad = w.lo < 0 || w.hi < w.lo || w.hi > a.max_rows || w.k0 < 0 || w.k1 < w.k0 || w.k1 > a.max_keys;
    if (bad && report) flag(a.status, DSPARK_STATUS_BAD_LEN);
    return !bad;
}

constexpr int kPromptWarps = 4;
constexpr int kPromptSteps = DSPARK_MAX_HEAD_DIM / 32;

template <typename T>
__global__ void __launch_bounds__(kPromptWarps * 32) prompt_any_kernel(PromptArgs a) {
    __shared__ float part_o[kPromptWarps][DSPARK_MAX_HEAD_DIM];
    __shared__ float part_m[kPromptWarps], part_l[kPromptWarps];
    pdl_trigger();
    pdl_wait();
    const int row = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (row == 0 && h == 0)
        for (int r = threadIdx.x; r < a.B; r += kPromptWarps * 32) usable(a, load_range(a, r), true);
    if (row >= __ldg(a.cu + a.B)) return;
    int first = 0, last = a.B - 1;  // the last request that starts at or before the row
    while (first < last) {
        const int mid = (first + last + 1) >> 1;
        if (__ldg(a.cu + mid) <= row) first = mid;
        else last = mid - 1;
    }
    const PromptRange w = load_range(a, first);
    if (!usable(a, w, false) || row < w.lo) return;
    const long long sees = (long long)(w.k1 - w.k0) - (w.hi - w.lo) + (row - w.lo) + 1;  // keys

    const int K = a.key_dim, S = a.shared_dim, V = a.value_dim, g = h / a.group;
    const T *q = static_cast<const T *>(a.q) + row * a.ld_q + (long long)h * (K + S);
    float qk[kPromptSteps], qs[kPromptSteps], o[kPromptSteps], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int i = 0; i < kPromptSteps; ++i) {
        const int d = lane + 32 * i;
        qk[i] = d < K ? elem_value(q[d]) * a.scale : 0.0f;
        qs[i] = d < S ? elem_value(q[K + d]) * a.scale : 0.0f;
        o[i] = 0.0f;
    }
    for (long long j = w.k0 + warp; j < w.k0 + sees; j += kPromptWarps) {
        const T *k = static_cast<const T *>(a.k) + j * a.ld_k + g * a.hs_k;
        const T *v = static_cast<const T *>(a.v) + j * a.ld_v + g * a.hs_v;
        const T *c = static_cast<const T *>(a.shared) + j * a.ld_shared;
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < kPromptSteps; ++i) {
            const int d = lane + 32 * i;
            if (d < K) s = fmaf(qk[i], elem_value(k[d]), s);
            if (d < S) s = fmaf(qs[i], elem_value(c[d]), s);
        }
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(kFullMask, s, x);
        const float mn = fmaxf(m, s);
        const float base = mn == -INFINITY ? 0.0f : mn;
        const float keep = expf(m - base), e = expf(s - base);
        l = l * keep + e;
#pragma unroll
        for (int i = 0; i < kPromptSteps; ++i) {
            const int d = lane + 32 * i;
            o[i] = o[i] * keep + e * (d < V ? elem_value(v[d]) : 0.0f);
        }
        m = mn;
    }
#pragma unroll
    for (int i = 0; i < kPromptSteps; ++i)
        if (lane + 32 * i < V) part_o[warp][lane + 32 * i] = o[i];
    if (lane == 0) {
        part_m[warp] = m;
        part_l[warp] = l;
    }
    __syncthreads();
    float M = -INFINITY, L = 0.0f, f[kPromptWarps];
#pragma unroll
    for (int i = 0; i < kPromptWarps; ++i) M = fmaxf(M, part_m[i]);
    const float base = M == -INFINITY ? 0.0f : M;
#pragma unroll
    for (int i = 0; i < kPromptWarps; ++i) {
        f[i] = expf(part_m[i] - base);
        L += part_l[i] * f[i];
    }
    T *out = static_cast<T *>(a.out) + row * a.ld_out + (long long)h * V;
    for (int d = threadIdx.x; d < V; d += kPromptWarps * 32) {
        float x = 0.0f;
#pragma unroll
        for (int i = 0; i < kPromptWarps; ++i) x += part_o[i][d] * f[i];
        elem_store(out + d, L == 0.0f ? 0.0f : x / L);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[(long long)row * a.n_q_heads + h] = L == 0.0f ? -INFINITY : base + logf(L);
}

}  // namespace dspark

using namespace dspark;

extern "C" int dspark_prompt_attention(const void *q, int64_t ld_q, const void *k, int64_t ld_k, int64_t hs_k,
                                       const void *k_shared, int64_t ld_shared, const void *v, int64_t ld_v,
                                       int64_t hs_v, int32_t dtype, int32_t n_q_heads, int32_t n_kv_heads,
                                       int32_t key_dim, int32_t shared_dim, int32_t value_dim, int32_t max_rows,
                                       int32_t max_keys, const int32_t *cu_seqlens, const int32_t *cu_keys,
                                       int32_t B, float scale, void *out, int64_t ld_out, float *lse,
                                       int32_t *status, void *stream) {
    if (!q || !k || !v || !out || !cu_seqlens || !cu_keys || !status || max_rows < 0 || max_keys < 0 || B < 1 ||
        n_q_heads < 1 || n_kv_heads < 1 || n_q_heads % n_kv_heads)
        return DSPARK_ERR_INVALID_ARG;
    if (dtype != DSPARK_DTYPE_BF16 && dtype != DSPARK_DTYPE_F32) return DSPARK_ERR_INVALID_ARG;
    if (key_dim < 1 || key_dim > DSPARK_MAX_HEAD_DIM || shared_dim < 0 || shared_dim > DSPARK_MAX_HEAD_DIM ||
        value_dim < 1 || value_dim > DSPARK_MAX_HEAD_DIM || n_q_heads > 65535)
        return DSPARK_ERR_UNSUPPORTED;
    if ((shared_dim > 0) != (k_shared != nullptr)) return DSPARK_ERR_INVALID_ARG;
    const int64_t width = (int64_t)n_q_heads * (key_dim + shared_dim), width_out = (int64_t)n_q_heads * value_dim;
    if (ld_q < width || ld_out < width_out || hs_k < key_dim || hs_v < value_dim ||
        ld_k < (n_kv_heads - 1) * hs_k + key_dim || ld_v < (n_kv_heads - 1) * hs_v + value_dim ||
        (k_shared && ld_shared < shared_dim))
        return DSPARK_ERR_INVALID_ARG;
    if (!(scale - scale == 0.0f)) return DSPARK_ERR_INVALID_ARG;
    if (max_rows == 0) return DSPARK_OK;
    const int64_t e_bytes = kv_elem_bytes(dtype);
    if (rows_overlap(q, ld_q * e_bytes, width * e_bytes, out, ld_out * e_bytes, width_out * e_bytes, max_rows))
        return DSPARK_ERR_INVALID_ARG;
    PromptArgs a;
    a.q = q;
    a.ld_q = ld_q;
    a.k = k;
    a.ld_k = ld_k;
    a.hs_k = hs_k;
    a.shared = k_shared;
    a.ld_shared = k_shared ? ld_shared : 0;
    a.v = v;
    a.ld_v = ld_v;
    a.hs_v = hs_v;
    a.out = out;
    a.ld_out = ld_out;
    a.lse = lse;
    a.cu = cu_seqlens;
    a.cu_k = cu_keys;
    a.B = B;
    a.n_q_heads = n_q_heads;
    a.group = n_q_heads / n_kv_heads;
    a.key_dim = key_dim;
    a.shared_dim = shared_dim;
    a.value_dim = value_dim;
    a.max_rows = max_rows;
    a.max_keys = max_keys;
    a.scale = scale;
    a.status = status;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const dim3 grid(max_rows, n_q_heads), block(kPromptWarps * 32);
    const cudaError_t e = dtype == DSPARK_DTYPE_BF16
                              ? launch_pdl(prompt_any_kernel<__nv_bfloat16>, grid, block, 0, st, a)
                              : launch_pdl(prompt_any_kernel<float>, grid, block, 0, st, a);
    return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
