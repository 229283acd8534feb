// latent.cu -- rows of latent vectors into their paged cache.
//
// The mathematics, for one row [x | r] and the query parts t_h of its heads, in 32 bits:
//   c = x / sqrt(mean(x^2) + eps) * w       (a, b) -> (a cos - b sin, b cos + a sin)
// the latter over the pairs of r and of every t_h.  Each element is read once and
// written once, so the bound is HBM bandwidth; for a few rows it is the launch.
//
// latent_append_kernel   a warp takes a row's cache entry, or a few steps of its query
//   heads (kSteps, all their loads in flight before the first use).  A unit of rotation is
//   eight pairs, sixteen elements in two 16-byte pieces, so that it stays in a lane; a lane
//   has the same pairs in every step and fetches its cosines and sines once.  Queries are
//   asked for before the row's position is known.  Windows of up to 17 tokens of 256
//   requests with 128 heads take 21 us, 3.9 TB/s: the chain row, position, angles is what
//   is left.  (With the queries asked for behind it 28 us; by the next kernel 81.)
// latent_append_any_kernel   any dimensions, strides and alignment: a warp a row's entry
//   or one head's part, one pair or element a lane and step.

#include "latentcache.cuh"

#include <type_traits>

namespace dspark {

constexpr int kLatentThreads = 128;
template <typename T>
constexpr int kSteps = 8 / sizeof(T);  // 32-byte or 64-byte units of a lane under way

struct LatentAppendArgs {
    const void *x;
    long long ld_x;
    const void *q;
    long long ld_q, hs_q;
    void *q_out;
    long long ld_q_out, hs_q_out;
    const void *weight;
    float eps;
    const float *cos_sin;
    int n_pos, interleaved, n_q_heads, latent_dim, rope_dim;
    const int32_t *req, *pos, *cache_pos, *totals;
    int max_rows;
    KvView cache;
    int32_t *status;
};

// Row w / parts and part w % parts of this warp's task; false behind the last row.
__device__ __forceinline__ bool latent_task(const LatentAppendArgs &a, long long warp, int parts, int *row,
                                            int *part) {
    const long long at = div_nonneg(warp, parts);
    *row = (int)at;
    *part = (int)(warp - at * parts);
    return at < (a.totals ? min(__ldg(a.totals), a.max_rows) : a.max_rows);
}

// The row's request and position; false if there is nothing to write (a pad row, a position
// that cannot be rotated, which the row's first part flags).
__device__ __forceinline__ bool latent_row(const LatentAppendArgs &a, int row, int part, int *r, int *p) {
    *r = __ldg(a.req + row);
    *p = __ldg(a.pos + row);
    if (*r < 0) return false;
    if (*p >= 0 && *p < a.n_pos) return true;
    if (part == 0 && (threadIdx.x & 31) == 0) flag(a.status, DSPARK_STATUS_BAD_INDEX);
    return false;
}

// Where the row's entry goes, in elements; -1, flagged, if it has no place.
__device__ __forceinline__ long long latent_place(const LatentAppendArgs &a, int row, int r, int p) {
    int token;
    const int page = kv_page(a.cache, r, a.cache_pos ? __ldg(a.cache_pos + row) : p, &token);
    if (page >= 0) return kv_offset(a.cache, page, token, 0);
    if ((threadIdx.x & 31) == 0) flag(a.status, DSPARK_STATUS_BAD_INDEX);
    return -1;
}

// Eight elements a lane, in pieces of 16 bytes, as they lie in memory and in 32 bits.
template <typename T>
struct Eight {
    uint4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Eight<T> raw8(const T *p) {
    Eight<T> x;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) x.v[i] = reinterpret_cast<const uint4 *>(p)[i];
    return x;
}
__device__ __forceinline__ void wide8(const Eight<__nv_bfloat16> &e, float (&x)[8]) {
    const unsigned w[4] = {e.v[0].x, e.v[0].y, e.v[0].z, e.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void wide8(const Eight<float> &e, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        x[4 * i] = __uint_as_float(e.v[i].x), x[4 * i + 1] = __uint_as_float(e.v[i].y);
        x[4 * i + 2] = __uint_as_float(e.v[i].z), x[4 * i + 3] = __uint_as_float(e.v[i].w);
    }
}
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&x)[8]) {
    wide8(raw8(p), x);
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&x)[8]) {
    unsigned w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 two = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const unsigned *>(&two);
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(float *p, const float (&x)[8]) {
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

// A unit's sixteen elements u, v as they lie in memory, rotated: pairs (u_i, v_i), or
// interleaved, neighbours.
__device__ __forceinline__ void rotate8(float (&u)[8], float (&v)[8], const float (&c)[8], const float (&s)[8],
                                        bool interleaved) {
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = u[2 * i], b = u[2 * i + 1], d = v[2 * i], e = v[2 * i + 1];
            u[2 * i] = a * c[i] - b * s[i], u[2 * i + 1] = b * c[i] + a * s[i];
            v[2 * i] = d * c[4 + i] - e * s[4 + i], v[2 * i + 1] = e * c[4 + i] + d * s[4 + i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = u[i], b = v[i];
            u[i] = a * c[i] - b * s[i], v[i] = b * c[i] + a * s[i];
        }
    }
}

template <typename T, typename C>
__global__ void __launch_bounds__(kLatentThreads) latent_append_kernel(LatentAppendArgs a, int parts) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    int row, part, r, p;
    if (!latent_task(a, ((long long)blockIdx.x * kLatentThreads + threadIdx.x) >> 5, parts, &row, &part)) return;
    // this lane's pairs, and where its unit's two pieces lie in a rotated part
    const int R = a.rope_dim, units = R / 16, unit = lane % units;
    const int first = a.interleaved ? 16 * unit : 8 * unit, second = a.interleaved ? first + 8 : first + R / 2;
    const int heads = 32 / units;  // a step
    const int h0 = (part - 1) * kSteps<T> * heads + lane / units;
    // the queries first: they do not wait for the row's position
    Eight<T> u[kSteps<T>], v[kSteps<T>];
    if (part > 0) {
        const T *q = static_cast<const T *>(a.q) + row * a.ld_q;
#pragma unroll
        for (int i = 0; i < kSteps<T>; ++i) {
            const int h = h0 + i * heads;
            if (h >= a.n_q_heads) continue;
            u[i] = raw8(q + h * a.hs_q + first);
            v[i] = raw8(q + h * a.hs_q + second);
        }
    }
    if (!latent_row(a, row, part, &r, &p)) return;
    float c[8], s[8];
    const float *angles = a.cos_sin + (long long)p * R + 8 * unit;
    load8(angles, c);
    load8(angles + R / 2, s);
    if (part == 0) {
        const long long at = latent_place(a, row, r, p);
        if (at < 0) return;
        const T *x = static_cast<const T *>(a.x) + row * a.ld_x;
        C *out = reinterpret_cast<C *>(a.cache.k) + at;
        constexpr int kPieces = DSPARK_MAX_LATENT_DIM / 256;
        float e[kPieces][8], key[2][8], sum = 0.0f;
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int d = (lane + 32 * i) * 8;
            if (d < a.latent_dim) load8(x + d, e[i]);
        }
        if (lane < units) {
            load8(x + a.latent_dim + first, key[0]);
            load8(x + a.latent_dim + second, key[1]);
        }
        if (a.weight) {
#pragma unroll
            for (int i = 0; i < kPieces; ++i)
                if ((lane + 32 * i) * 8 < a.latent_dim)
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum = fmaf(e[i][j], e[i][j], sum);
            for (int m = 16; m; m >>= 1) sum += __shfl_xor_sync(kFullMask, sum, m);
            const float inv = 1.0f / sqrtf(sum / a.latent_dim + a.eps);
#pragma unroll
            for (int i = 0; i < kPieces; ++i) {
                const int d = (lane + 32 * i) * 8;
                if (d >= a.latent_dim) continue;
                float w[8];
                load8(static_cast<const T *>(a.weight) + d, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) e[i][j] = e[i][j] * inv * w[j];
            }
        }
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int d = (lane + 32 * i) * 8;
            if (d < a.latent_dim) store8(out + d, e[i]);
        }
        if (lane < units) {
            rotate8(key[0], key[1], c, s, a.interleaved);
            store8(out + a.latent_dim + first, key[0]);
            store8(out + a.latent_dim + second, key[1]);
        }
        return;
    }
    T *out = static_cast<T *>(a.q_out) + row * a.ld_q_out;
#pragma unroll
    for (int i = 0; i < kSteps<T>; ++i) {
        const int h = h0 + i * heads;
        if (h >= a.n_q_heads) continue;
        float x[8], y[8];
        wide8(u[i], x);
        wide8(v[i], y);
        rotate8(x, y, c, s, a.interleaved);
        store8(out + h * a.hs_q_out + first, x);
        store8(out + h * a.hs_q_out + second, y);
    }
}

template <typename T, typename O>
__device__ __forceinline__ void rotate_part(const T *x, O *out, const float *angles, int R, int interleaved) {
    for (int i = threadIdx.x & 31; i < R / 2; i += 32) {
        const int m = interleaved ? 2 * i : i, n = interleaved ? 2 * i + 1 : i + R / 2;
        const float a = elem_value(x[m]), b = elem_value(x[n]), c = angles[i], s = angles[R / 2 + i];
        elem_store(out + m, a * c - b * s);
        elem_store(out + n, b * c + a * s);
    }
}

template <typename T, typename C>
__global__ void __launch_bounds__(kLatentThreads) latent_append_any_kernel(LatentAppendArgs a) {
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, R = a.rope_dim;
    int row, part, r, p;
    if (!latent_task(a, ((long long)blockIdx.x * kLatentThreads + threadIdx.x) >> 5, 1 + a.n_q_heads, &row, &part) ||
        !latent_row(a, row, part, &r, &p))
        return;
    const float *angles = a.cos_sin + (long long)p * R;
    if (part > 0) {
        rotate_part(static_cast<const T *>(a.q) + row * a.ld_q + (part - 1) * a.hs_q,
                    static_cast<T *>(a.q_out) + row * a.ld_q_out + (part - 1) * a.hs_q_out, angles, R,
                    a.interleaved);
        return;
    }
    const long long at = latent_place(a, row, r, p);
    if (at < 0) return;
    const T *x = static_cast<const T *>(a.x) + row * a.ld_x, *w = static_cast<const T *>(a.weight);
    C *out = reinterpret_cast<C *>(a.cache.k) + at;
    float inv = 1.0f;
    if (w) {
        float sum = 0.0f;
        for (int d = lane; d < a.latent_dim; d += 32) sum = fmaf(elem_value(x[d]), elem_value(x[d]), sum);
        for (int m = 16; m; m >>= 1) sum += __shfl_xor_sync(kFullMask, sum, m);
        inv = 1.0f / sqrtf(sum / a.latent_dim + a.eps);
    }
    for (int d = lane; d < a.latent_dim; d += 32)
        elem_store(out + d, w ? elem_value(x[d]) * inv * elem_value(w[d]) : elem_value(x[d]));
    rotate_part(x + a.latent_dim, out + a.latent_dim, angles, R, a.interleaved);
}

namespace {

// Whether every piece of 16 bytes that the first kernel touches is aligned, and a part's
// units divide a warp.
bool append_pieces(const LatentAppendArgs &a, int dtype, const dspark_latent_cache &c) {
    const int e = kv_elem_bytes(dtype), ce = kv_elem_bytes(c.dtype), units = a.rope_dim / 16;
    bool ok = a.latent_dim % 8 == 0 && a.rope_dim % 16 == 0 && 32 % units == 0;
    ok = ok && aligned(a.x, 16) && aligned(a.weight, 16) && aligned(a.cos_sin, 16) && aligned(a.q, 16) &&
         aligned(a.q_out, 16) && aligned(c.data, 16);
    for (long long s : {a.ld_x, a.ld_q, a.hs_q, a.ld_q_out, a.hs_q_out}) ok = ok && s * e % 16 == 0;
    return ok && c.page_stride * ce % 16 == 0 && c.token_stride * ce % 16 == 0;
}

// Whether the queries' outputs are the queries themselves, or share no element with them:
// rows side by side or apart in any strides, or, with the strides of the queries, parts of
// the same rows' heads.
bool same_or_apart(const LatentAppendArgs &a, int dtype) {
    const int64_t e = kv_elem_bytes(dtype), part = a.rope_dim * e, H = a.n_q_heads;
    const char *q = static_cast<const char *>(a.q), *out = static_cast<const char *>(a.q_out);
    const bool rows_alike = a.ld_q == a.ld_q_out || a.max_rows == 1, heads_alike = a.hs_q == a.hs_q_out || H == 1;
    if (q == out && rows_alike && heads_alike) return true;
    const int64_t span = (H - 1) * a.hs_q * e + part, span_out = (H - 1) * a.hs_q_out * e + part;
    if (!rows_overlap(q, a.ld_q * e, span, a.max_rows, out, a.ld_q_out * e, span_out, a.max_rows)) return true;
    if (!rows_alike || !heads_alike) return false;
    for (int64_t h = 1 - H; h < H; ++h)
        if (rows_overlap(q, a.ld_q * e, part, a.max_rows, out + h * a.hs_q * e, a.ld_q * e, part, a.max_rows))
            return false;
    return true;
}

template <typename T, typename C>
cudaError_t launch_latent_append(const LatentAppendArgs &a, bool pieces, cudaStream_t stream) {
    const int step = pieces ? 32 / (a.rope_dim / 16) * kSteps<T> : 1;
    const int parts = 1 + (a.n_q_heads + step - 1) / step;
    constexpr int kWarps = kLatentThreads / 32;
    const long long grid = ((long long)a.max_rows * parts + kWarps - 1) / kWarps;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    if (pieces)
        return launch_pdl(latent_append_kernel<T, C>, dim3((unsigned)grid), dim3(kLatentThreads), 0, stream, a,
                          parts);
    return launch_pdl(latent_append_any_kernel<T, C>, dim3((unsigned)grid), dim3(kLatentThreads), 0, stream, a);
}

template <typename T>
cudaError_t launch_latent_append(const LatentAppendArgs &a, int cache_dtype, bool pieces, cudaStream_t stream) {
    if (cache_dtype == DSPARK_DTYPE_BF16) return launch_latent_append<T, __nv_bfloat16>(a, pieces, stream);
    return launch_latent_append<T, float>(a, pieces, stream);
}

}  // namespace

}  // namespace dspark

using namespace dspark;

extern "C" int dspark_latent_append(const void *x, int64_t ld_x, const void *q, int64_t ld_q, int64_t hs_q,
                                    int32_t dtype, int32_t n_q_heads, const dspark_latent_cache *cache,
                                    const dspark_norm_rope *nr, const int32_t *req, const int32_t *pos,
                                    const int32_t *cache_pos, const int32_t *totals, int32_t max_rows,
                                    void *q_out, int64_t ld_q_out, int64_t hs_q_out, int32_t *status,
                                    void *stream) {
    const int rc = latent_check(cache);
    if (rc != DSPARK_OK) return rc;
    if (!x || !nr || !nr->cos_sin || nr->q_weight || !req || !pos || !status || max_rows < 0 || n_q_heads < 0)
        return DSPARK_ERR_INVALID_ARG;
    if (dtype != DSPARK_DTYPE_BF16 && dtype != DSPARK_DTYPE_F32) return DSPARK_ERR_INVALID_ARG;
    if (!(nr->eps >= 0.0f) || nr->rope_dim != cache->rope_dim || nr->n_pos < 0) return DSPARK_ERR_INVALID_ARG;
    if (ld_x < cache->latent_dim + cache->rope_dim) return DSPARK_ERR_INVALID_ARG;
    if ((n_q_heads > 0) != (q != nullptr) || (q != nullptr) != (q_out != nullptr)) return DSPARK_ERR_INVALID_ARG;
    if (q && (hs_q < cache->rope_dim || hs_q_out < cache->rope_dim ||
              ld_q < (n_q_heads - 1) * hs_q + cache->rope_dim ||
              ld_q_out < (n_q_heads - 1) * hs_q_out + cache->rope_dim))
        return DSPARK_ERR_INVALID_ARG;
    if (max_rows == 0) return DSPARK_OK;
    LatentAppendArgs a;
    a.x = x;
    a.ld_x = ld_x;
    a.q = q;
    a.ld_q = q ? ld_q : 0;
    a.hs_q = q ? hs_q : 0;
    a.q_out = q_out;
    a.ld_q_out = q ? ld_q_out : 0;
    a.hs_q_out = q ? hs_q_out : 0;
    a.weight = nr->k_weight;
    a.eps = nr->eps;
    a.cos_sin = nr->cos_sin;
    a.n_pos = nr->n_pos;
    a.interleaved = nr->interleaved != 0;
    a.n_q_heads = n_q_heads;
    a.latent_dim = cache->latent_dim;
    a.rope_dim = cache->rope_dim;
    a.req = req;
    a.pos = pos;
    a.cache_pos = cache_pos;
    a.totals = totals;
    a.max_rows = max_rows;
    a.cache = latent_view(*cache);
    a.status = status;
    if (q && !same_or_apart(a, dtype)) return DSPARK_ERR_INVALID_ARG;
    const bool pieces = append_pieces(a, dtype, *cache);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == DSPARK_DTYPE_BF16
                              ? launch_latent_append<__nv_bfloat16>(a, cache->dtype, pieces, st)
                              : launch_latent_append<float>(a, cache->dtype, pieces, st);
    return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
