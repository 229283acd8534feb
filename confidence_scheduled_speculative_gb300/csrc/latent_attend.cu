// latent_attend.cu -- attention of a verify window's drafted tokens over the paged
// latent cache that holds their requests' prefixes and the tokens themselves, in the
// absorbed form: every head's keys are a token's whole entry [c | r], its values c.
//
// For packed row i (token t of request r's window, query head h) over the positions p it
// sees, the prefix and the window tokens of its ancestor bits:
//   s_p = scale q . [c_p | r_p],  m = max s_p,  l = sum exp(s_p - m)
//   out = sum exp(s_p - m) c_p / l,     lse = m + ln l
//
// latent_any_kernel   any types, strides, dimensions and page sizes, in 32 bits
//   throughout: a CTA a (row, query head), its four warps take every fourth
//   position, each with a running maximum and sum, joined at the end.

#include "latentcache.cuh"
#include "schedule.cuh"

namespace dspark {

constexpr int kAnyWarps = 4;
constexpr int kValueSteps = DSPARK_MAX_LATENT_DIM / 32;
constexpr int kKeySteps = kValueSteps + DSPARK_MAX_LATENT_ROPE / 32;

struct LatentArgs {
    AttendArgs a;
    int latent_dim;
};

template <typename T, typename C>
__global__ void __launch_bounds__(kAnyWarps * 32) latent_any_kernel(LatentArgs t) {
    __shared__ float part_o[kAnyWarps][DSPARK_MAX_LATENT_DIM];
    __shared__ float part_m[kAnyWarps], part_l[kAnyWarps];
    pdl_trigger();
    pdl_wait();
    const AttendArgs &a = t.a;
    const int row = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int D = a.cache.head_dim, L = t.latent_dim;
    // (the requests' windows are looked at by one CTA: a window outside the rows has none)
    if (row == 0 && h == 0)
        for (int r = threadIdx.x; r < a.B; r += kAnyWarps * 32) usable(a, load_window(a, r), true);
    if (row >= __ldg(a.cu + a.B)) return;
    const int r = request_of(a, row);
    const Window win = load_window(a, r);
    if (!usable(a, win, false) || row < win.lo) return;
    const int len = win.hi - win.lo, P = win.P;
    const unsigned bits = ancestors_of(a, row, row - win.lo, len);

    const T *q = static_cast<const T *>(a.q) + row * a.ld_q + (long long)h * D;
    float qv[kKeySteps], o[kValueSteps], m = -INFINITY, l = 0.0f;
    // element d of the key, for a lane's step: those of c first, then those of r
    auto element = [&](int i) { return i < kValueSteps ? lane + 32 * i : L + lane + 32 * (i - kValueSteps); };
    auto there = [&](int i) { return element(i) < (i < kValueSteps ? L : D); };
#pragma unroll
    for (int i = 0; i < kKeySteps; ++i) qv[i] = there(i) ? elem_value(q[element(i)]) * a.scale : 0.0f;
#pragma unroll
    for (int i = 0; i < kValueSteps; ++i) o[i] = 0.0f;
    for (int p = warp; p < P + len; p += kAnyWarps) {
        if (p >= P && !(bits >> (p - P) & 1)) continue;
        int token;
        const int page = kv_page(a.cache, r, p, &token);
        if (page < 0) {
            if (lane == 0) flag(a.status, DSPARK_STATUS_BAD_INDEX);
            continue;
        }
        const C *kv = reinterpret_cast<const C *>(a.cache.k) + kv_offset(a.cache, page, token, 0);
        float s = 0.0f, v[kValueSteps];
#pragma unroll
        for (int i = 0; i < kKeySteps; ++i) {
            const float x = there(i) ? elem_value(kv[element(i)]) : 0.0f;
            if (i < kValueSteps) v[i] = x;
            if (there(i)) s = fmaf(qv[i], x, s);
        }
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(kFullMask, s, x);
        const float mn = fmaxf(m, s);
        const float base = mn == -INFINITY ? 0.0f : mn;
        const float keep = expf(m - base), w = expf(s - base);
        l = l * keep + w;
#pragma unroll
        for (int i = 0; i < kValueSteps; ++i) o[i] = o[i] * keep + w * v[i];
        m = mn;
    }
#pragma unroll
    for (int i = 0; i < kValueSteps; ++i)
        if (there(i)) part_o[warp][element(i)] = o[i];
    if (lane == 0) {
        part_m[warp] = m;
        part_l[warp] = l;
    }
    __syncthreads();
    float M = -INFINITY, sum = 0.0f, f[kAnyWarps];
#pragma unroll
    for (int w = 0; w < kAnyWarps; ++w) M = fmaxf(M, part_m[w]);
    const float base = M == -INFINITY ? 0.0f : M;
#pragma unroll
    for (int w = 0; w < kAnyWarps; ++w) {
        f[w] = expf(part_m[w] - base);
        sum += part_l[w] * f[w];
    }
    T *out = static_cast<T *>(a.out) + row * a.ld_out + (long long)h * L;
    for (int d = threadIdx.x; d < L; d += kAnyWarps * 32) {
        float x = 0.0f;
#pragma unroll
        for (int w = 0; w < kAnyWarps; ++w) x += part_o[w][d] * f[w];
        elem_store(out + d, sum == 0.0f ? 0.0f : x / sum);
    }
    if (a.lse && threadIdx.x == 0)
        a.lse[(long long)row * a.n_q_heads + h] = sum == 0.0f ? -INFINITY : base + logf(sum);
}

namespace {

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

template <typename T>
cudaError_t launch_any(const LatentArgs &t, int cache_dtype, cudaStream_t stream) {
    const dim3 grid(t.a.max_rows, t.a.n_q_heads), block(kAnyWarps * 32);
    if (cache_dtype == DSPARK_DTYPE_BF16)
        return launch_pdl(latent_any_kernel<T, __nv_bfloat16>, grid, block, 0, stream, t);
    return launch_pdl(latent_any_kernel<T, float>, grid, block, 0, stream, t);
}

}  // namespace

}  // namespace dspark

using namespace dspark;

extern "C" size_t dspark_latent_attention_workspace_bytes(int32_t n_q_heads, int32_t latent_dim) {
    if (n_q_heads < 1 || latent_dim < 2 || latent_dim > DSPARK_MAX_LATENT_DIM) return 0;
    return round256(1);
}

extern "C" int dspark_latent_attention(const void *q, int64_t ld_q, int32_t dtype, int32_t n_q_heads,
                                       int32_t max_rows, const int32_t *cu_seqlens,
                                       const int32_t *prefix_lens, int32_t B, const uint32_t *ancestors,
                                       float scale, const dspark_latent_cache *cache, void *out,
                                       int64_t ld_out, float *lse, void *workspace,
                                       size_t workspace_bytes, int32_t *status, void *stream) {
    const int rc = latent_check(cache);
    if (rc != DSPARK_OK) return rc;
    if (!q || !out || !cu_seqlens || !prefix_lens || !status || max_rows < 0 || B < 1 ||
        B > cache->n_requests || n_q_heads < 1)
        return DSPARK_ERR_INVALID_ARG;
    if (dtype != DSPARK_DTYPE_BF16 && dtype != DSPARK_DTYPE_F32) return DSPARK_ERR_INVALID_ARG;
    const int64_t width = (int64_t)n_q_heads * (cache->latent_dim + cache->rope_dim);
    const int64_t width_out = (int64_t)n_q_heads * cache->latent_dim;
    if (ld_q < width || ld_out < width_out) return DSPARK_ERR_INVALID_ARG;
    if (!(scale - scale == 0.0f)) return DSPARK_ERR_INVALID_ARG;
    if (n_q_heads > 65535) return DSPARK_ERR_UNSUPPORTED;
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < dspark_latent_attention_workspace_bytes(n_q_heads, cache->latent_dim))
        return DSPARK_ERR_WORKSPACE;
    if (max_rows == 0) return DSPARK_OK;
    // (a split job reads its queries again after another CTA has written its outputs)
    const int64_t e_bytes = kv_elem_bytes(dtype);
    if (rows_overlap(q, ld_q * e_bytes, width * e_bytes, out, ld_out * e_bytes, width_out * e_bytes, max_rows))
        return DSPARK_ERR_INVALID_ARG;
    LatentArgs t;
    AttendArgs &a = t.a;
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
    a.cache = latent_view(*cache);
    a.status = status;
    t.latent_dim = cache->latent_dim;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == DSPARK_DTYPE_BF16 ? launch_any<__nv_bfloat16>(t, cache->dtype, st)
                                                     : launch_any<float>(t, cache->dtype, st);
    return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
