// cache.cu -- norms and rotation of queries and keys, the write of keys and
// values into a paged cache (quantised to E4M3 on the way, if it is one), and
// the reading of cache entries back into rows.
//
// The mathematics, for one row and head x in R^D, all in 32 bits:
//   y = x / sqrt(mean(x^2) + eps) * w          (queries and keys, if a weight is given)
//   (a, b) -> (a c - b s, b c + a s)           (the pairs of the first rope_dim elements)
//   E4M3: scale = max(max|y| / 448, 2^-100), code = e4m3(y / scale)
// Each element is read once and written once and costs some ten operations,
// so the bound is HBM bandwidth; for a window of a few rows it is the launch.
//
// append_kernel   a warp takes one row, or a part of its heads where rows are few, and
//   steps through them a few heads a lane group at a time, the next ones'
//   loads in flight.  The row's position, slot, cosines and sines are fetched once.
//   A head is D / 8 lanes of eight elements: four and the four that they rotate with,
//   so that the rotation stays in a lane and a head's sum and maximum are a few
//   shuffles; nothing is read twice.  Eight prompts of 4096 tokens, 32 and 8 heads of
//   128: 455 MB in 77 us (5.9 TB/s, 0.86 of a copy); the rotation alone of four with 64
//   heads 62 us (6.1 TB/s, 0.89); 256 windows of up to 17 tokens into E4M3 20 us (4.6
//   TB/s: a row's chain of dependent loads and the arithmetic, in two waves of CTAs, 1776
//   where 912 fit; 84 to 96 bytes of spills in the kernels from bfloat16 into E4M3).
// append_any_kernel   any alignment, stride and even head size: one warp a
//   (row, head), one element a lane and step.
// read_kernel     a CTA takes 16 output rows: their slots are looked up by one
//   warp (binary search in cu_rows, then the block table), then all threads
//   stream the rows' elements.  32 prefixes of up to 8192 tokens from E4M3 into
//   bfloat16 rows: 839 MB in 131 us (6.4 TB/s, 0.94 of a copy).

#include "kvcache.cuh"
#include "pairs.cuh"

#include <type_traits>

namespace dspark {

constexpr int kAppendThreads = 128;
// heads a lane group has in flight: 64 bytes a lane
template <typename T>
constexpr int kHeadsPerLane = 16 / sizeof(T) / 2;
// Warps an SM before a warp takes all heads of a row: a window of 256 requests of up to
// 17 tokens takes 20 us at 48, 26 at 24 and below, 26 at 96.
constexpr int kWarpsWanted = 48;
constexpr int kReadThreads = 256;
constexpr int kReadRows = 16;  // long prefixes 132 us; of 32 rows 137, of 64 139

struct NoCache {};

struct AppendArgs {
    const void *in[3];  // q, k, v
    long long ld_in[3];
    int heads[3];
    void *out[2];  // q_out, k_out (no cache)
    long long ld_out[2];
    const void *weight[2];
    float eps;
    const float *cos_sin;  // null: no rotation
    int n_pos, rope_dim, interleaved;
    const int32_t *req, *pos, *cache_pos, *totals;
    int max_rows, head_dim;
    KvView cache;
    int32_t *status;
};

// Four elements as they lie in memory, as numbers, and back.
template <typename T>
struct Four;
template <>
struct Four<__nv_bfloat16> {
    using Raw = uint2;
    __device__ static void unpack(const Raw &v, float *x) {
        x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xFFFF0000u);
        x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xFFFF0000u);
    }
    __device__ static Raw pack(const float *x) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
        return make_uint2(*reinterpret_cast<const unsigned *>(&a), *reinterpret_cast<const unsigned *>(&b));
    }
};
template <>
struct Four<float> {
    using Raw = float4;
    __device__ static void unpack(const Raw &v, float *x) {
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    }
    __device__ static Raw pack(const float *x) { return make_float4(x[0], x[1], x[2], x[3]); }
};

// Eight elements as numbers, and back.
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float *x) {
    const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p));
    Four<__nv_bfloat16>::unpack(make_uint2(v.x, v.y), x);
    Four<__nv_bfloat16>::unpack(make_uint2(v.z, v.w), x + 4);
}
__device__ __forceinline__ void load8(const float *p, float *x) {
    Four<float>::unpack(__ldg(reinterpret_cast<const float4 *>(p)), x);
    Four<float>::unpack(__ldg(reinterpret_cast<const float4 *>(p) + 1), x + 4);
}
__device__ __forceinline__ void load8(const e4m3 *p, float *x) {
    const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const unsigned w = i < 2 ? v.x : v.y;
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * (i & 1))), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float *x) {
    const uint2 a = Four<__nv_bfloat16>::pack(x), b = Four<__nv_bfloat16>::pack(x + 4);
    *reinterpret_cast<uint4 *>(p) = make_uint4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store8(float *p, const float *x) {
    reinterpret_cast<float4 *>(p)[0] = Four<float>::pack(x);
    reinterpret_cast<float4 *>(p)[1] = Four<float>::pack(x + 4);
}

__device__ __forceinline__ int rows_of(const AppendArgs &a) {
    if (!a.totals) return a.max_rows;
    return max(0, min(__ldg(a.totals), a.max_rows));
}

// The slot of a row's key and value: false for a pad row or a bad one (flagged).
__device__ __forceinline__ bool row_slot(const AppendArgs &a, int row, int *page, int *token) {
    const int r = __ldg(a.req + row);
    if (r < 0) return false;
    *page = kv_page(a.cache, r, __ldg((a.cache_pos ? a.cache_pos : a.pos) + row), token);
    if (*page < 0) flag(a.status, DSPARK_STATUS_BAD_INDEX);
    return *page >= 0;
}

// The row's position in the rotation's table: false when it is outside (flagged).
__device__ __forceinline__ bool row_angle(const AppendArgs &a, int row, int *p) {
    *p = 0;
    if (!a.cos_sin) return true;
    if (a.req && __ldg(a.req + row) < 0) return false;
    *p = __ldg(a.pos + row);
    const bool ok = *p >= 0 && *p < a.n_pos;
    if (!ok) flag(a.status, DSPARK_STATUS_BAD_INDEX);
    return ok;
}

template <typename T, typename C, int kLanes>
__global__ void __launch_bounds__(kAppendThreads, 6) append_kernel(AppendArgs a, int parts) {
    constexpr bool kCache = !std::is_same<C, NoCache>::value;
    constexpr int kHeads = kHeadsPerLane<T>;
    using Raw = typename Four<T>::Raw;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, D = a.head_dim;
    const unsigned unit = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    const int row = unit / (unsigned)parts, part = unit - row * parts;
    if (row >= a.max_rows) return;
    constexpr int groups = 32 / kLanes, step = groups * kHeads;  // kLanes lanes a head
    const int group = lane / kLanes, chunk = lane % kLanes;
    const int H = a.heads[0] + a.heads[1] + a.heads[2];
    const int per = ((H + step - 1) / step + parts - 1) / parts * step;  // heads a part
    const int begin = part * per, end = min(begin + per, H);
    const bool has = chunk * 8 < D;  // a lane past a head that is not a power of two

    // where this lane's two fours of a head lie: an element and its partner, which
    // is R / 2 on in the first R, or the next one in neighbouring pairs; the rest
    // lie anywhere
    const int R = a.cos_sin ? a.rope_dim : 0;
    int at0 = chunk * 8, at1 = at0 + 4;
    bool turned = at0 < R;
    if (!a.interleaved && R) {
        turned = chunk * 4 < R / 2;
        const int rest = chunk * 4 - R / 2;
        at0 = turned ? chunk * 4 : R + rest;
        at1 = turned ? at0 + R / 2 : R + (D - R) / 2 + rest;
    }

    // the heads of one step of a kind, as they lie in memory
    Raw raw[kHeads][2];
    auto fetch = [&](const T *p, int h, int last) {
#pragma unroll
        for (int i = 0; i < kHeads; ++i) {
            raw[i][0] = raw[i][1] = Raw{};
            if (h + i * groups < last && has) {
                raw[i][0] = *reinterpret_cast<const Raw *>(p + i * groups * D);
                raw[i][1] = *reinterpret_cast<const Raw *>(p + i * groups * D + (at1 - at0));
            }
        }
    };
    // the part's heads of a kind: [from, to), and where the group's first lies
    auto from = [&](int kind) {
        const int before = kind == 0 ? 0 : (kind == 1 ? a.heads[0] : a.heads[0] + a.heads[1]);
        return max(begin - before, 0);
    };
    auto to = [&](int kind) {
        const int before = kind == 0 ? 0 : (kind == 1 ? a.heads[0] : a.heads[0] + a.heads[1]);
        return min(end - before, a.heads[kind]);
    };
    auto source = [&](int kind) {
        return static_cast<const T *>(a.in[kind]) + row * a.ld_in[kind] + (from(kind) + group) * D + at0;
    };
    if (begin >= end) return;
    const int kind0 = begin < a.heads[0] ? 0 : (begin < a.heads[0] + a.heads[1] ? 1 : 2);
    fetch(source(kind0), from(kind0) + group, to(kind0));
    const int total = a.totals ? __ldg(a.totals) : a.max_rows;
    const int r = a.req ? __ldg(a.req + row) : 0;
    const int position = a.pos ? __ldg(a.pos + row) : 0;
    const int place = a.cache_pos ? __ldg(a.cache_pos + row) : position;
    if (row >= total || r < 0) return;
    const bool angle = !R || (position >= 0 && position < a.n_pos);
    if (!angle) flag(a.status, DSPARK_STATUS_BAD_INDEX);
    int page = -1, token = 0;
    if (kCache && end > a.heads[0]) {
        page = kv_page(a.cache, r, place, &token);
        if (page < 0) flag(a.status, DSPARK_STATUS_BAD_INDEX);
    }
    // (a, b) -> (a c - b s, b c + a s), two elements an instruction: of the lane's four
    // pairs of elements the cosines, and the sines that the partners come with
    float2 cos2[4], sin2[4];
    turned = turned && angle;
    if (turned) {
        const float *cs = a.cos_sin + (long long)position * R + chunk * 4;
        const float4 c = __ldg(reinterpret_cast<const float4 *>(cs));
        const float4 s = __ldg(reinterpret_cast<const float4 *>(cs + R / 2));
        if (a.interleaved) {
            cos2[0] = make_float2(c.x, c.x), cos2[1] = make_float2(c.y, c.y);
            cos2[2] = make_float2(c.z, c.z), cos2[3] = make_float2(c.w, c.w);
            sin2[0] = make_float2(-s.x, s.x), sin2[1] = make_float2(-s.y, s.y);
            sin2[2] = make_float2(-s.z, s.z), sin2[3] = make_float2(-s.w, s.w);
        } else {
            cos2[0] = cos2[2] = make_float2(c.x, c.y), cos2[1] = cos2[3] = make_float2(c.z, c.w);
            sin2[0] = make_float2(-s.x, -s.y), sin2[1] = make_float2(-s.z, -s.w);
            sin2[2] = make_float2(s.x, s.y), sin2[3] = make_float2(s.z, s.w);
        }
    }

    // queries, keys and values one kind after the other, each its own code
    const float share = 1.0f / (float)D;
    auto run = [&](auto kind_c) {
        constexpr int kKind = decltype(kind_c)::value;
        const int first = from(kKind), last = to(kKind);
        if (first >= last) return;
        const T *in = source(kKind);
        if (kKind != kind0) fetch(in, first + group, last);
        T *out = nullptr;
        if (kKind < 2 && (!kCache || kKind == 0))
            out = static_cast<T *>(a.out[kKind < 2 ? kKind : 0]) + row * a.ld_out[kKind < 2 ? kKind : 0] +
                  (first + group) * D + at0;
        const T *weight = kKind < 2 ? static_cast<const T *>(a.weight[kKind < 2 ? kKind : 0]) : nullptr;
        // (zero where a lane has no elements, whose products count for the largest one)
        float2 w[4] = {};
        if (weight && has) {
            Four<T>::unpack(__ldg(reinterpret_cast<const Raw *>(weight + at0)), reinterpret_cast<float *>(w));
            Four<T>::unpack(__ldg(reinterpret_cast<const Raw *>(weight + at1)), reinterpret_cast<float *>(w + 2));
        }
        [[maybe_unused]] unsigned char *stored = kKind == 1 ? a.cache.k : a.cache.v;
        [[maybe_unused]] float *scales = kKind == 1 ? a.cache.k_scale : a.cache.v_scale;
        long long slot = kv_offset(a.cache, page, token, first + group);
        long long scale_slot = kv_scale_offset(a.cache, page, token, first + group);
        for (int h0 = first + group; h0 - group < last; h0 += step) {
            Raw now[kHeads][2];
#pragma unroll
            for (int i = 0; i < kHeads; ++i) now[i][0] = raw[i][0], now[i][1] = raw[i][1];
            in += step * D;
            if (h0 - group + step < last) fetch(in, h0 + step, last);
#pragma unroll
            for (int i = 0; i < kHeads; ++i) {
                // the shuffles are the whole warp's: every lane goes through them
                const bool mine = h0 + i * groups < last && has;
                float2 y[4];
                Four<T>::unpack(now[i][0], reinterpret_cast<float *>(y));
                Four<T>::unpack(now[i][1], reinterpret_cast<float *>(y + 2));
                if (kKind < 2 && weight) {
                    float2 sum = mul2(y[0], y[0]);
#pragma unroll
                    for (int e = 1; e < 4; ++e) sum = fma2(y[e], y[e], sum);
                    float ss = sum.x + sum.y;
#pragma unroll
                    for (int o = kLanes / 2; o; o >>= 1) ss += __shfl_xor_sync(kFullMask, ss, o);
                    const float inv = rsqrtf(fmaf(ss, share, a.eps));
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = mul2(mul2(y[e], make_float2(inv, inv)), w[e]);
                }
                if (kKind < 2 && turned) {
                    float2 z[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 other = a.interleaved ? make_float2(y[e].y, y[e].x) : y[e ^ 2];
                        z[e] = fma2(y[e], cos2[e], mul2(other, sin2[e]));
                    }
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = z[e];
                }
                const float *x = reinterpret_cast<const float *>(y);
                if (kKind < 2 && (!kCache || kKind == 0)) {
                    if (mine && angle) {
                        T *p = out + i * groups * D;
                        *reinterpret_cast<Raw *>(p) = Four<T>::pack(x);
                        *reinterpret_cast<Raw *>(p + (at1 - at0)) = Four<T>::pack(x + 4);
                    }
                } else if constexpr (kCache) {
                    const bool write = mine && page >= 0 && angle;
                    const long long at = slot + (long long)i * groups * a.cache.head_stride;
                    if constexpr (std::is_same<C, e4m3>::value) {
                        unsigned m = 0;
#pragma unroll
                        for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e]) & 0x7FFFFFFFu);
#pragma unroll
                        for (int o = kLanes / 2; o; o >>= 1)
                            m = max(m, __shfl_xor_sync(kFullMask, m, o));
                        if (write) {
                            // y / scale, correctly rounded, by Markstein's method: the
                            // rounded reciprocal's product, and one correction by the
                            // exact remainder (which is only inexact for quotients far
                            // below the smallest code).  Eight divisions by the same
                            // number are dear (8 prompts of 4096 into E4M3: 97 us
                            // with them, 85 so; a window of 256 requests 22.5 and 20.5).
                            const float scale = e4m3_scale(m), r = __frcp_rn(scale);
                            unsigned codes[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float2 q = mul2(y[e], make_float2(r, r));
                                const float2 rest = fma2(q, make_float2(-scale, -scale), y[e]);
                                const float2 z = fma2(rest, make_float2(r, r), q);
                                codes[e] = e4m3_pair(z.x, z.y);
                            }
                            *reinterpret_cast<unsigned *>(stored + at + at0) = codes[0] | codes[1] << 16;
                            *reinterpret_cast<unsigned *>(stored + at + at1) = codes[2] | codes[3] << 16;
                            if (chunk == 0) {
                                scales[scale_slot + (long long)i * groups * a.cache.page_size] = scale;
                                if (m >= 0x7F800000u) flag(a.status, DSPARK_STATUS_BAD_INPUT);
                            }
                        }
                    } else if (write) {
                        using Stored = typename Four<C>::Raw;
                        C *p = reinterpret_cast<C *>(stored) + at;
                        *reinterpret_cast<Stored *>(p + at0) = Four<C>::pack(x);
                        *reinterpret_cast<Stored *>(p + at1) = Four<C>::pack(x + 4);
                    }
                }
            }
            if (out) out += step * D;
            slot += (long long)step * a.cache.head_stride;
            scale_slot += (long long)step * a.cache.page_size;
        }
    };
    run(std::integral_constant<int, 0>{});
    run(std::integral_constant<int, 1>{});
    if constexpr (kCache) run(std::integral_constant<int, 2>{});
}

// Any layout: one warp a (row, head).  Every element and its rotation partner
// are read before the first is written, so the call may run in place.
template <typename T, typename C>
__global__ void __launch_bounds__(kAppendThreads) append_any_kernel(AppendArgs a) {
    constexpr bool kCache = !std::is_same<C, NoCache>::value;
    constexpr int kSteps = DSPARK_MAX_HEAD_DIM / 32;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31, D = a.head_dim;
    const int H = a.heads[0] + a.heads[1] + a.heads[2];
    const long long unit = (long long)blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);
    const long long row64 = div_nonneg(unit, H);
    if (row64 >= rows_of(a)) return;
    const int row = (int)row64;
    int head = (int)(unit - row64 * H), kind = 0;
    while (head >= a.heads[kind]) head -= a.heads[kind++];
    if (a.req && __ldg(a.req + row) < 0) return;
    int p;
    if (!row_angle(a, row, &p)) return;
    int page = -1, token = 0;
    if (kCache && kind > 0 && !row_slot(a, row, &page, &token)) return;

    const T *src = static_cast<const T *>(a.in[kind]) + row * a.ld_in[kind] + (long long)head * D;
    const T *w = kind < 2 ? static_cast<const T *>(a.weight[kind]) : nullptr;
    const int R = kind < 2 && a.cos_sin ? a.rope_dim : 0;
    float y[kSteps], other[kSteps], ss = 0.0f;
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
        const int d = lane + 32 * t;
        y[t] = d < D ? elem_value(src[d]) : 0.0f;
        ss = fmaf(y[t], y[t], ss);
        const int o = a.interleaved ? d ^ 1 : (d < R / 2 ? d + R / 2 : d - R / 2);
        other[t] = d < R ? elem_value(src[o]) * (w ? elem_value(w[o]) : 1.0f) : 0.0f;
        if (d < D && w) y[t] *= elem_value(w[d]);
    }
    float inv = 1.0f;
    if (w) {
        for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(kFullMask, ss, o);
        inv = 1.0f / sqrtf(ss / (float)D + a.eps);
    }
    unsigned m = 0;
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
        const int d = lane + 32 * t;
        y[t] *= inv;
        if (d < R) {
            const int i = a.interleaved ? d >> 1 : (d < R / 2 ? d : d - R / 2);
            const bool first = a.interleaved ? !(d & 1) : d < R / 2;
            const float *cs = a.cos_sin + (long long)p * R;
            const float c = __ldg(cs + i), s = __ldg(cs + R / 2 + i);
            y[t] = y[t] * c + (first ? -1.0f : 1.0f) * (other[t] * inv) * s;
        }
        m = max(m, __float_as_uint(y[t]) & 0x7FFFFFFFu);
    }
    __syncwarp();
    if (!kCache || kind == 0) {
        T *dst = static_cast<T *>(a.out[kind]) + row * a.ld_out[kind] + (long long)head * D;
#pragma unroll
        for (int t = 0; t < kSteps; ++t)
            if (lane + 32 * t < D) elem_store(dst + lane + 32 * t, y[t]);
        return;
    }
    if constexpr (kCache) {
        unsigned char *base = kind == 1 ? a.cache.k : a.cache.v;
        const long long at = kv_offset(a.cache, page, token, head);
        float scale = 1.0f;
        if constexpr (std::is_same<C, e4m3>::value) {
            for (int o = 16; o; o >>= 1) m = max(m, __shfl_xor_sync(kFullMask, m, o));
            scale = e4m3_scale(m);
            if (lane == 0) {
                (kind == 1 ? a.cache.k_scale
                           : a.cache.v_scale)[kv_scale_offset(a.cache, page, token, head)] = scale;
                if (m >= 0x7F800000u) flag(a.status, DSPARK_STATUS_BAD_INPUT);
            }
        }
#pragma unroll
        for (int t = 0; t < kSteps; ++t) {
            const int d = lane + 32 * t;
            if (d >= D) continue;
            if constexpr (std::is_same<C, e4m3>::value)
                base[at + d] = (unsigned char)(e4m3_pair(__fdiv_rn(y[t], scale), 0.0f) & 0xFF);
            else
                elem_store(reinterpret_cast<C *>(base) + at + d, y[t]);
        }
    }
}

struct ReadArgs {
    KvView cache;
    const int32_t *start, *cu;
    int B, max_rows;
    void *out[2];
    long long ld_out;
    int32_t *status;
};

// kVec elements a thread and step: 8 where rows, slots and head size allow
// 16-byte loads (8-byte ones of E4M3 codes), else 1.
template <typename C, typename T, int kVec>
__global__ void __launch_bounds__(kReadThreads) read_kernel(ReadArgs a) {
    __shared__ int pages[kReadRows], tokens[kReadRows];
    pdl_trigger();
    pdl_wait();
    const int row0 = blockIdx.x * kReadRows;
    const int total = __ldg(a.cu + a.B);
    if (blockIdx.x == 0 && threadIdx.x == 0 && total > a.max_rows)
        flag(a.status, DSPARK_STATUS_CAPACITY);
    const int rows = min(total, a.max_rows);
    if (row0 >= rows) return;
    if (threadIdx.x < kReadRows) {
        const int row = row0 + threadIdx.x;
        int page = -1, token = 0;
        if (row < rows) {
            // the last request that starts at or before the row
            int lo = 0, hi = a.B - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (__ldg(a.cu + mid) <= row) lo = mid;
                else hi = mid - 1;
            }
            page = kv_page(a.cache, lo, (long long)__ldg(a.start + lo) + (row - __ldg(a.cu + lo)), &token);
            if (page < 0) flag(a.status, DSPARK_STATUS_BAD_INDEX);
        }
        pages[threadIdx.x] = page;
        tokens[threadIdx.x] = token;
    }
    __syncthreads();
    const int D = a.cache.head_dim, per_head = D / kVec, per_row = a.cache.n_kv_heads * per_head;
    const int n = min(kReadRows, rows - row0) * per_row;
    const C *src[2] = {reinterpret_cast<const C *>(a.cache.k), reinterpret_cast<const C *>(a.cache.v)};
    const float *scales[2] = {a.cache.k_scale, a.cache.v_scale};
#pragma unroll 2
    for (int i = threadIdx.x; i < n; i += kReadThreads) {
        const int j = i / per_row, at = i - j * per_row, head = at / per_head;
        const int page = pages[j];
        if (page < 0) continue;
        const int d = (at - head * per_head) * kVec;
        const long long from = kv_offset(a.cache, page, tokens[j], head) + d;
        const long long to = (row0 + j) * a.ld_out + (long long)head * D + d;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            float scale = 1.0f;
            if constexpr (std::is_same<C, e4m3>::value)
                scale = __ldg(scales[which] + kv_scale_offset(a.cache, page, tokens[j], head));
            T *dst = static_cast<T *>(a.out[which]) + to;
            if constexpr (kVec == 8) {
                float x[8];
                load8(src[which] + from, x);
                if constexpr (std::is_same<C, e4m3>::value) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] *= scale;
                }
                store8(dst, x);
            } else {
                float x = elem_value(src[which][from]);
                if constexpr (std::is_same<C, e4m3>::value) x *= scale;
                elem_store(dst, x);
            }
        }
    }
}

template <typename T, typename C>
cudaError_t launch_append(const AppendArgs &a, bool vec, cudaStream_t stream) {
    const int H = a.heads[0] + a.heads[1] + a.heads[2];
    constexpr int kWarps = kAppendThreads / 32;
    if (vec) {
        // a warp a row streams best; few rows are split over their heads until every
        // SM has kWarpsWanted warps
        const int lanes = a.head_dim <= 64 ? 8 : (a.head_dim <= 128 ? 16 : 32);
        const int step = 32 / lanes * kHeadsPerLane<T>, steps = (H + step - 1) / step;
        const long long want = (long long)kWarpsWanted * sm_count();
        const int parts = (int)max(1ll, min((long long)steps, want / a.max_rows));
        const long long grid = ((long long)a.max_rows * parts + kWarps - 1) / kWarps;
        if (grid > 0x7FFFFFFF / kWarps) return cudaErrorInvalidConfiguration;
        return launch_pdl(lanes == 8    ? append_kernel<T, C, 8>
                          : lanes == 16 ? append_kernel<T, C, 16>
                                        : append_kernel<T, C, 32>,
                          dim3((unsigned)grid), dim3(kAppendThreads), 0, stream, a, parts);
    }
    const long long grid = ((long long)a.max_rows * H + kWarps - 1) / kWarps;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    return launch_pdl(append_any_kernel<T, C>, dim3((unsigned)grid), dim3(kAppendThreads), 0,
                      stream, a);
}

template <typename T>
cudaError_t launch_append_cache(const AppendArgs &a, int cache_dtype, bool vec, cudaStream_t st) {
    if (cache_dtype < 0) return launch_append<T, NoCache>(a, vec, st);
    if (cache_dtype == DSPARK_DTYPE_BF16) return launch_append<T, __nv_bfloat16>(a, vec, st);
    if (cache_dtype == DSPARK_DTYPE_F32) return launch_append<T, float>(a, vec, st);
    return launch_append<T, e4m3>(a, vec, st);
}

template <typename C, typename T>
cudaError_t launch_read(const ReadArgs &a, bool vec, cudaStream_t stream) {
    const dim3 grid((a.max_rows + kReadRows - 1) / kReadRows), block(kReadThreads);
    if (vec) return launch_pdl(read_kernel<C, T, 8>, grid, block, 0, stream, a);
    return launch_pdl(read_kernel<C, T, 1>, grid, block, 0, stream, a);
}

template <typename C>
cudaError_t launch_read_out(const ReadArgs &a, int out_dtype, bool vec, cudaStream_t stream) {
    if (out_dtype == DSPARK_DTYPE_BF16) return launch_read<C, __nv_bfloat16>(a, vec, stream);
    return launch_read<C, float>(a, vec, stream);
}

namespace {

// Whether p and a stride of ld elements keep accesses of n elements (16 bytes at
// most) aligned.
bool aligned_to(const void *p, long long ld, int n, int elem_bytes) {
    const int bytes = n * elem_bytes < 16 ? n * elem_bytes : 16;
    return aligned(p, bytes) && ld * elem_bytes % bytes == 0;
}

bool cache_aligned(const dspark_kv_cache &c, int n) {
    const int e = kv_elem_bytes(c.dtype);
    return c.head_dim % n == 0 && aligned_to(c.k, c.page_stride, n, e) &&
           aligned_to(c.v, c.token_stride, n, e) && aligned_to(c.k, c.head_stride, n, e);
}

// The checks that the two writing calls share; fills the arguments they share.
int fill_append(AppendArgs &a, const void *q, int64_t ld_q, const void *k, int64_t ld_k,
                int32_t dtype, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                const dspark_norm_rope *nr, const int32_t *pos, const int32_t *totals,
                int32_t max_rows, void *q_out, int64_t ld_q_out, int32_t *status) {
    if (!status || max_rows < 0 || n_q_heads < 0 || n_kv_heads < 0) return DSPARK_ERR_INVALID_ARG;
    if (dtype != DSPARK_DTYPE_BF16 && dtype != DSPARK_DTYPE_F32) return DSPARK_ERR_INVALID_ARG;
    if (head_dim < 2 || head_dim > DSPARK_MAX_HEAD_DIM || head_dim % 2)
        return DSPARK_ERR_UNSUPPORTED;
    if ((n_q_heads > 0) != (q != nullptr) || (q != nullptr) != (q_out != nullptr))
        return DSPARK_ERR_INVALID_ARG;
    if ((n_kv_heads > 0) != (k != nullptr)) return DSPARK_ERR_INVALID_ARG;
    if (q && (ld_q < (int64_t)n_q_heads * head_dim || ld_q_out < (int64_t)n_q_heads * head_dim))
        return DSPARK_ERR_INVALID_ARG;
    if (k && ld_k < (int64_t)n_kv_heads * head_dim) return DSPARK_ERR_INVALID_ARG;
    a = AppendArgs{};
    if (nr) {
        if (!(nr->eps >= 0.0f)) return DSPARK_ERR_INVALID_ARG;
        if (nr->cos_sin) {
            if (!pos || nr->n_pos < 0 || nr->rope_dim < 2 || nr->rope_dim > head_dim ||
                nr->rope_dim % 2)
                return DSPARK_ERR_INVALID_ARG;
            a.cos_sin = nr->cos_sin;
            a.n_pos = nr->n_pos;
            a.rope_dim = nr->rope_dim;
            a.interleaved = nr->interleaved != 0;
        }
        a.weight[0] = nr->q_weight;
        a.weight[1] = nr->k_weight;
        a.eps = nr->eps;
    }
    a.in[0] = q;
    a.in[1] = k;
    a.ld_in[0] = ld_q;
    a.ld_in[1] = ld_k;
    a.heads[0] = n_q_heads;
    a.heads[1] = n_kv_heads;
    a.out[0] = q_out;
    a.ld_out[0] = ld_q_out;
    a.pos = pos;
    a.totals = totals;
    a.max_rows = max_rows;
    a.head_dim = head_dim;
    a.status = status;
    return DSPARK_OK;
}

// Whether the shared operands allow append_kernel: lanes of two fours.
bool append_fours(const AppendArgs &a, int dtype) {
    const int e = kv_elem_bytes(dtype);
    bool ok = a.head_dim % 8 == 0;
    for (int i = 0; i < 3; ++i) ok = ok && aligned_to(a.in[i], a.ld_in[i], 4, e);
    for (int i = 0; i < 2; ++i)
        ok = ok && aligned_to(a.out[i], a.ld_out[i], 4, e) && aligned(a.weight[i], 4 * e);
    if (a.cos_sin) ok = ok && aligned(a.cos_sin, 16) && a.rope_dim % 8 == 0;
    return ok;
}

}  // namespace

}  // namespace dspark

using namespace dspark;

extern "C" int dspark_qk_norm_rope(const void *q, int64_t ld_q, const void *k, int64_t ld_k,
                                   int32_t dtype, int32_t n_q_heads, int32_t n_kv_heads,
                                   int32_t head_dim, const dspark_norm_rope *nr,
                                   const int32_t *pos, const int32_t *totals, int32_t max_rows,
                                   void *q_out, int64_t ld_q_out, void *k_out, int64_t ld_k_out,
                                   int32_t *status, void *stream) {
    AppendArgs a;
    if (!nr || (!q && !k) || (k != nullptr) != (k_out != nullptr)) return DSPARK_ERR_INVALID_ARG;
    const int rc = fill_append(a, q, ld_q, k, ld_k, dtype, n_q_heads, n_kv_heads, head_dim, nr, pos,
                               totals, max_rows, q_out, ld_q_out, status);
    if (rc != DSPARK_OK) return rc;
    if (k && ld_k_out < (int64_t)n_kv_heads * head_dim) return DSPARK_ERR_INVALID_ARG;
    a.out[1] = k_out;
    a.ld_out[1] = ld_k_out;
    if (max_rows == 0) return DSPARK_OK;
    const bool vec = append_fours(a, dtype);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == DSPARK_DTYPE_BF16
                              ? launch_append_cache<__nv_bfloat16>(a, -1, vec, st)
                              : launch_append_cache<float>(a, -1, vec, st);
    return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

extern "C" int dspark_kv_append(const void *q, int64_t ld_q, const void *k, int64_t ld_k,
                                const void *v, int64_t ld_v, int32_t dtype, int32_t n_q_heads,
                                const dspark_kv_cache *cache, const dspark_norm_rope *nr,
                                const int32_t *req, const int32_t *pos, const int32_t *cache_pos,
                                const int32_t *totals, int32_t max_rows, void *q_out,
                                int64_t ld_q_out, int32_t *status, void *stream) {
    int rc = kv_check(cache);
    if (rc != DSPARK_OK) return rc;
    if (!k || !v || !req || (!pos && !cache_pos)) return DSPARK_ERR_INVALID_ARG;
    AppendArgs a;
    rc = fill_append(a, q, ld_q, k, ld_k, dtype, n_q_heads, cache->n_kv_heads, cache->head_dim, nr,
                     pos, totals, max_rows, q_out, ld_q_out, status);
    if (rc != DSPARK_OK) return rc;
    if (ld_v < (int64_t)cache->n_kv_heads * cache->head_dim) return DSPARK_ERR_INVALID_ARG;
    a.in[2] = v;
    a.ld_in[2] = ld_v;
    a.heads[2] = cache->n_kv_heads;
    a.req = req;
    a.cache_pos = cache_pos;
    a.cache = kv_view(*cache);
    if (max_rows == 0) return DSPARK_OK;
    const bool vec = append_fours(a, dtype) && cache_aligned(*cache, 4);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == DSPARK_DTYPE_BF16
                              ? launch_append_cache<__nv_bfloat16>(a, cache->dtype, vec, st)
                              : launch_append_cache<float>(a, cache->dtype, vec, st);
    return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

extern "C" int dspark_kv_read(const dspark_kv_cache *cache, const int32_t *start,
                              const int32_t *cu_rows, int32_t B, int32_t max_rows,
                              int32_t out_dtype, void *k_out, void *v_out, int64_t ld_out,
                              int32_t *status, void *stream) {
    const int rc = kv_check(cache);
    if (rc != DSPARK_OK) return rc;
    if (!start || !cu_rows || !k_out || !v_out || !status || max_rows < 0 || B < 1 ||
        B > cache->n_requests || ld_out < (int64_t)cache->n_kv_heads * cache->head_dim)
        return DSPARK_ERR_INVALID_ARG;
    if (out_dtype != DSPARK_DTYPE_BF16 && out_dtype != DSPARK_DTYPE_F32)
        return DSPARK_ERR_INVALID_ARG;
    if ((long long)cache->n_kv_heads * cache->head_dim * kReadRows > 0x7FFFFFFF)
        return DSPARK_ERR_UNSUPPORTED;
    ReadArgs a;
    a.cache = kv_view(*cache);
    a.start = start;
    a.cu = cu_rows;
    a.B = B;
    a.max_rows = max_rows;
    a.out[0] = k_out;
    a.out[1] = v_out;
    a.ld_out = ld_out;
    a.status = status;
    const int e = kv_elem_bytes(out_dtype);
    const bool vec = cache_aligned(*cache, 8) && aligned_to(k_out, ld_out, 8, e) && aligned_to(v_out, ld_out, 8, e);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (max_rows == 0) return DSPARK_OK;
    cudaError_t err;
    if (cache->dtype == DSPARK_DTYPE_BF16)
        err = launch_read_out<__nv_bfloat16>(a, out_dtype, vec, st);
    else if (cache->dtype == DSPARK_DTYPE_F32)
        err = launch_read_out<float>(a, out_dtype, vec, st);
    else
        err = launch_read_out<e4m3>(a, out_dtype, vec, st);
    return err == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
