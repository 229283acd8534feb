// fewrows.cuh -- few rows over the E4M3 cache: single tokens and short windows, whose
// query heads of a kv head are a few rows (included by attend.cu, which has the
// mathematics and joins the parts).
//
// The products are taken the other way round, with 16 positions as the rows of the
// matrix instruction and up to 8 query rows as its columns:
//   S^T [16 positions][8 rows]  = K [16][D] Q^T [D][8]
//   O^T [D][8 rows]            += V^T [D][16] P^T [16][8]
// so that keys and values are operands that stay in registers: the order in which a
// product sums its dimensions is free, hence a thread's part of K is 16 adjacent bytes
// of a token's row, and of V^T adjacent bytes of four tokens.  The codes become halves
// (exactly) on the way; only P^T, two 8 x 8 tiles of halves, changes hands inside a warp.
// mma.sync suits this: eight columns are all there are, and its operands are registers,
// while tcgen05.mma would want codes as halves in shared memory and 128 rows.
//
// A CTA's eight warps take the steps of a job in turn, each with a running maximum, sum
// and output of its own and its own copies in flight, so that nothing is waited for until
// the job's end.  A stage in shared memory is written and read by the same lanes, but for
// the scales.  32 requests of up to 8192 tokens, 4 heads a kv head, 286 MB: 75 us (3.8
// TB/s, 0.56 of a copy; 113 us in the kernel of 128 rows a tile).  What bounds it is the
// chain inside a warp: 445 instructions a step, issued in 44% of the cycles by the four
// warps a scheduler has room for.
#pragma once

#include "schedule.cuh"
#include "tensor.cuh"

namespace dspark {

constexpr int kFewWarps = 8;
constexpr int kFewChunk = 16;   // positions a step of a warp
constexpr int kFewStages = 3;   // steps in flight a warp
// What a job's begin and end cost, in tiles of its products: 32 requests of up to 8192
// tokens take 89, 82, 77, 75.5, 75.9 and 78 us at 1, 2, 4, 6, 8 and 12.
constexpr int kFewJobCost = 6;

template <int D>
struct FewShape {
    static constexpr int kCodes = kFewChunk * D;            // of K or V a stage
    static constexpr int kStage = 2 * kCodes + 2 * 4 * kFewChunk;  // and both scales
    static constexpr int kRing = kFewWarps * kFewStages * kStage;
    static_assert(kFewRows * D * 4 <= kStage, "a warp's output fits in a stage");
};
struct FewControl {
    Begin begin;
    Walk<kFewJobCost> walk;
    Segment seg[4];  // the present one, the next, and the one after
    unsigned nonfinite[2];  // window tokens whose values were zeroed, by segment
    int stage[kFewWarps];   // where the warps left their outputs
    float mx[kFewWarps][kFewRows], l[kFewWarps][kFewRows];
    long long scan[40];
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(in ? 8 : 0)
                 : "memory");
}
// x = a b + x: 16 x 16 halves times 16 x 8.
__device__ __forceinline__ void mma_16x8(float (&x)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// Off by at most one unit in the last place, for normal numbers.
__device__ __forceinline__ float reciprocal_approx(float x) {
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Off by at most 2^-22, for x in (1/2, 2), and by 2^-22 of itself elsewhere.
__device__ __forceinline__ float log2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_halves(float x, float y) {
    const __half2 two = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t *>(&two);
}

template <int D>
__global__ void __launch_bounds__(kFewWarps * 32, 2) attend_few_kernel(const TensorArgs t) {
    using S = FewShape<D>;
    constexpr int kSteps = D / 16;        // products along D; 16-row tiles of V^T
    constexpr int kWords = D / 64;        // 16-byte pieces of a token's key a thread
    extern __shared__ __align__(1024) unsigned char smem[];
    FewControl &ctl = *reinterpret_cast<FewControl *>(smem + S::kRing);
    const AttendArgs &a = t.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, c = lane & 3;
    pdl_wait();
    pdl_trigger();
    Deal deal;
    long long lo, hi;
    const int cta = blockIdx.x;
    if (!share_of<kFewWarps * 32, kFewJobCost, true>(t, &ctl.begin, ctl.scan, &deal, &lo, &hi)) return;
    __syncthreads();
    // one thread walks; the others read the segments it leaves
    auto leave = [&](unsigned k) {
        if (!ctl.walk.next(t, &ctl.seg[k & 3])) ctl.seg[k & 3].count = 0;
    };
    if (tid == 0) {
        ctl.walk.begin(t, ctl.begin, (int)(hi - lo));
        leave(0);
        leave(1);
        ctl.nonfinite[0] = ctl.nonfinite[1] = 0;
    }
    __syncthreads();

    unsigned char *ring = smem + warp * kFewStages * S::kStage;
    const uint32_t ring_at = smem_addr(ring);
    const float scale = copysignf(fmaxf(fabsf(a.scale) * kLog2e, 0x1p-100f), a.scale);

    // The copies run ahead of the products by up to kFewStages steps, into the next
    // segment too.  A warp takes every kFewWarps-th step of a segment.
    unsigned fetched = 0, used = 0, fk = 0;
    uint32_t f_stage = 0, stage = 0;  // of the next step to copy, to multiply: bytes
    int fi = 0, fn = 0, f_left = 0, f_page = -1, f_token = 0;
    long long f_head = 0, f_scale = 0;
    auto steps_of = [&](const Segment &s) {
        const int end = min((s.first + s.count) * kTile, s.q.P + s.q.len) - s.first * kTile;
        const int steps = (end + kFewChunk - 1) / kFewChunk;
        return s.count ? max(steps - warp + kFewWarps - 1, 0) / kFewWarps : 0;
    };
    auto enter = [&](unsigned k) {
        const Segment &s = ctl.seg[k & 3];
        fk = k;
        fi = 0;
        fn = steps_of(s);
        f_left = s.q.P + s.q.len - s.first * kTile - warp * kFewChunk;
        f_head = s.head * a.cache.head_stride;
        f_scale = (long long)s.head * a.cache.page_size;
    };
    enter(0);
    // this lane's part of a step: of K two tokens' bytes, of V four tokens', and of
    // the scales (eight lanes) four
    const long long k_lane = g * a.cache.token_stride + c * 16;
    const long long v_lane = 2 * c * a.cache.token_stride + g * (D / 8);
    const float *s_lane = (lane < 4 ? a.cache.k_scale : a.cache.v_scale) + 4 * c;
    auto copy_v = [](uint32_t dst, const void *src, bool in) {
        if (D == 128) copy16(dst, src, in);
        else copy8(dst, src, in);
    };
    auto fetch = [&](unsigned k) {  // one more step, of segment k or the next
        if (fi == fn && fk == k) enter(k + 1);
        if (fi == fn) return false;
        if (!(fi & 31)) {
            // where the next 32 steps lie, one a lane
            const Segment &s = ctl.seg[fk & 3];
            const int at = s.first * kTile + (warp + (fi + lane) * kFewWarps) * kFewChunk;
            f_page = -1;
            if (fi + lane < fn) {
                const int col = (unsigned)at / (unsigned)a.cache.page_size;
                f_token = at - col * a.cache.page_size;
                f_page = __ldg(a.cache.table + (long long)s.r * a.cache.table_width + col);
                if ((unsigned)f_page >= (unsigned)a.cache.n_pages) {
                    f_page = -1;
                    flag(a.status, DSPARK_STATUS_BAD_INDEX);
                }
            }
        }
        const int page = __shfl_sync(kFullMask, f_page, fi & 31);
        const int token = __shfl_sync(kFullMask, f_token, fi & 31);
        // a page outside the pool, as past the request's end, arrives as zeros
        const bool in = page >= 0;
        const long long from = in ? page * a.cache.page_stride + token * a.cache.token_stride + f_head : 0;
        const unsigned char *k_from = a.cache.k + from + k_lane, *v_from = a.cache.v + from + v_lane;
        const long long s_from =
            in ? (long long)page * a.cache.n_kv_heads * a.cache.page_size + f_scale + token : 0;
        const uint32_t to = ring_at + f_stage + lane * 16;
        const uint32_t v_to = ring_at + f_stage + S::kCodes + lane * (D / 8);
        const long long stride = a.cache.token_stride;
        if (in && f_left >= kFewChunk) {
#pragma unroll
            for (int j = 0; j < 2 * kWords; ++j)
                copy16(to + j * 512, k_from + j / kWords * 8 * stride + j % kWords * 64, true);
#pragma unroll
            for (int j = 0; j < 4; ++j) copy_v(v_to + j * 4 * D, v_from + ((j & 1) + 8 * (j >> 1)) * stride, true);
        } else {
            // tokens past the end as zeros: none of them is read
            const int left = in ? f_left : 0;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const bool some = g + 8 * h < left;
#pragma unroll
                for (int j = 0; j < kWords; ++j)
                    copy16(to + (h * kWords + j) * 512, k_from + (some ? h * 8 * stride : -k_lane) + j * 64, some);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const bool has = 2 * c + j + 8 * h < left;
                    copy_v(v_to + (2 * h + j) * 4 * D, v_from + (has ? (j + 8 * h) * stride : -v_lane), has);
                }
            }
        }
        if (lane < 8) copy16(to + 2 * S::kCodes, s_lane + s_from, in);
        asm volatile("cp.async.commit_group;" ::: "memory");
        ++fetched;
        f_stage = f_stage == (kFewStages - 1) * S::kStage ? 0 : f_stage + S::kStage;
        ++fi;
        f_left -= kFewWarps * kFewChunk;
        return true;
    };

    for (unsigned k = 0; ctl.seg[k & 3].count; ++k) {
        const Segment &s = ctl.seg[k & 3];
        const int n = s.q.P + s.q.len, P = s.q.P, token0 = s.row_tile * t.tokens;
        const int rows = min(t.tokens, s.q.len - token0) * t.group;
        const int steps = steps_of(s);
        const bool whole = s.count == s.q.tiles;
        if (fk < k) enter(k);

        // Query row g as the right operand, scaled by a power of two to halves: the
        // row's largest element to 2^14..2^15, so that any element down to 2^-31 of
        // it keeps its eight digits.
        uint32_t q[kSteps][2];
        float by_row[2];       // what rows 2c and 2c + 1 were divided by
        unsigned sees[2];      // and the window tokens that they see
        {
            const int m = min(g, rows - 1);
            const __nv_bfloat16 *from = static_cast<const __nv_bfloat16 *>(a.q) +
                                        (s.q.row0 + token0 + m / t.group) * a.ld_q +
                                        (long long)(s.head * t.group + m % t.group) * D;
            unsigned most = 0;
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
                const uint2 x = *reinterpret_cast<const uint2 *>(from + (j >> 2) * 64 + c * 16 + (j & 3) * 4);
                q[j][0] = x.x;
                q[j][1] = x.y;
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    most = max(most, max(q[j][e] & 0x7FFFu, q[j][e] >> 16 & 0x7FFFu));
            }
            most = max(most, __shfl_xor_sync(kFullMask, most, 1));
            most = max(most, __shfl_xor_sync(kFullMask, most, 2));
            const int exponent = min(max((int)(most >> 7), 16), 254) - 141;
            const float by = __int_as_float((127 - exponent) << 23);
#pragma unroll
            for (int j = 0; j < kSteps; ++j)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    q[j][e] = pack_halves(__uint_as_float(q[j][e] << 16) * by,
                                          __uint_as_float(q[j][e] & 0xFFFF0000u) * by);
            const float back = most >= 0x7F80u ? __int_as_float(0x7FC00000) : __int_as_float((exponent + 127) << 23);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                by_row[e] = __shfl_sync(kFullMask, back, (2 * c + e) * 4);
                const int token = token0 + min(2 * c + e, rows - 1) / t.group;
                sees[e] = ancestors_of(a, s.q.row0 + token, token, s.q.len);
            }
        }

        float o[kSteps][4], mx[2], l[2];
#pragma unroll
        for (int j = 0; j < kSteps; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.0f;
        mx[0] = mx[1] = -INFINITY;
        l[0] = l[1] = 0.0f;
        int pos = s.first * kTile + warp * kFewChunk;
#pragma unroll 1
        for (int i = 0; i < steps; ++i, ++used, pos += kFewWarps * kFewChunk) {
            while (fetched < used + kFewStages && fetch(k)) {}
            if (fetched - used > 2) asm volatile("cp.async.wait_group 2;" ::: "memory");
            else if (fetched - used > 1) asm volatile("cp.async.wait_group 1;" ::: "memory");
            else asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncwarp();  // the scales are other lanes' copies
            const unsigned char *at = ring + stage;
            stage = stage == (kFewStages - 1) * S::kStage ? 0 : stage + S::kStage;
            const float *ks = reinterpret_cast<const float *>(at + 2 * S::kCodes), *vs = ks + kFewChunk;
            const bool window = pos + kFewChunk > P;

            // scores of tokens g and g + 8 by rows 2c and 2c + 1
            float z[4] = {0.0f, 0.0f, 0.0f, 0.0f}, z2[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            {
                uint4 w[2][kWords];
#pragma unroll
                for (int j = 0; j < 2 * kWords; ++j)
                    w[j / kWords][j % kWords] = *reinterpret_cast<const uint4 *>(at + j * 512 + lane * 16);
#pragma unroll
                for (int j = 0; j < kSteps; ++j) {
                    const unsigned x = reinterpret_cast<const unsigned *>(w[0])[j];
                    const unsigned y = reinterpret_cast<const unsigned *>(w[1])[j];
                    uint32_t halves[4];
                    four_halves(x, &halves[0], &halves[2]);
                    four_halves(y, &halves[1], &halves[3]);
                    mma_16x8(j & 1 ? z2 : z, halves, q[j][0], q[j][1]);
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) z[x] += z2[x];
            }
            // Scores to base 2, plus log2 of the value's scale: the weights then are
            // those of the values' codes, and the sum divides it out again.
            float inv[2];
            bool odd = false;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float kf = ks[g + 8 * h], vf = vs[g + 8 * h];
                if (window && pos + g + 8 * h >= n) kf = vf = 1.0f;
                const bool fine = vf - vf == 0.0f;
                odd = odd || !fine || vf < 0.0f;
                // a NaN or infinite k_scale makes the score NaN
                kf = kf - kf == 0.0f ? kf * scale : __int_as_float(0x7FC00000);
                vf = fine ? fmaxf(fabsf(vf), 0x1p-100f) : 1.0f;
                const float log2v = log2_approx(vf);
                inv[h] = reciprocal_approx(vf);
#pragma unroll
                for (int e = 0; e < 2; ++e) z[2 * h + e] = fmaf(z[2 * h + e] * by_row[e], kf, log2v);
            }
            if (window) {
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const int p = pos + g + 8 * (x >> 1);
                    if (p >= P && (p >= n || !(sees[x & 1] >> (p - P) & 1))) z[x] = -INFINITY;
                }
            }
            // The maximum moves only when it grows by 2^kLazy: until then the
            // weights may pass 1, and sum and output stay as they are.
            float top[2] = {fmaxf(z[0], z[2]) - kHalfRoom, fmaxf(z[1], z[3]) - kHalfRoom};
            auto grows = [&](int e) { return top[e] > mx[e] + kLazy || (mx[e] == -INFINITY && top[e] > mx[e]); };
            if (__any_sync(kFullMask, grows(0) || grows(1))) {
                float f[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) top[e] = fmaxf(top[e], __shfl_xor_sync(kFullMask, top[e], x));
                    const bool grow = grows(e);
                    f[e] = grow ? exp2_approx(mx[e] - top[e]) : 1.0f;
                    if (grow) mx[e] = top[e];
                    l[e] *= f[e];
                }
#pragma unroll
                for (int j = 0; j < kSteps; ++j)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[j][e] *= f[e & 1];
            }
            uint32_t w[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float shift = mx[e] == -INFINITY ? 0.0f : mx[e];
                z[e] = exp2_approx(z[e] - shift);
                z[2 + e] = exp2_approx(z[2 + e] - shift);
                l[e] = fmaf(z[e], inv[0], fmaf(z[2 + e], inv[1], l[e]));
            }
            // the weights as halves, as the instruction takes them: rounded to 11
            // digits, eight times finer than the output
#pragma unroll
            for (int h = 0; h < 2; ++h) w[h] = transposed(pack_halves(z[2 * h], z[2 * h + 1]));

            // Negative and non-finite scales of values, and the window's tokens (of
            // which NaN and infinities become zeros: 0 x NaN would reach rows that do
            // not see them; those that do get them at the end).
            const bool special = window || __any_sync(kFullMask, odd);
            uint32_t sign[2];
            unsigned bad = 0;
            if (special) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float f[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int token = 2 * c + 8 * h + e;
                        f[e] = pos + token < n ? vs[token] : 1.0f;
                        if (f[e] - f[e] == 0.0f) f[e] = copysignf(1.0f, f[e]);
                    }
                    sign[h] = pack_halves(f[0], f[1]);
                }
            }
            uint4 v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (D == 128) {
                    v[j] = *reinterpret_cast<const uint4 *>(at + S::kCodes + j * 512 + lane * 16);
                } else {
                    const uint2 x = *reinterpret_cast<const uint2 *>(at + S::kCodes + j * 256 + lane * 8);
                    v[j] = make_uint4(x.x, x.y, 0, 0);
                }
            }
#pragma unroll
            for (int j = 0; j < kSteps; ++j) {
                // dimensions 2j and 2j + 1 of this thread's, tokens 2c, 2c + 1 and 8 on
                uint32_t halves[4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const unsigned x = reinterpret_cast<const unsigned *>(&v[2 * h])[j / 2];
                    const unsigned y = reinterpret_cast<const unsigned *>(&v[2 * h + 1])[j / 2];
                    four_halves(__byte_perm(x, y, j & 1 ? 0x7362 : 0x5140), &halves[2 * h], &halves[2 * h + 1]);
                }
                if (special) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const __half2 x = __hmul2(*reinterpret_cast<const __half2 *>(&halves[e]),
                                                  *reinterpret_cast<const __half2 *>(&sign[e >> 1]));
                        uint32_t y = *reinterpret_cast<const uint32_t *>(&x);
                        const int p = pos + 2 * c + 8 * (e >> 1);
                        if (p >= P && (y & 0x7C00u) == 0x7C00u) y &= 0xFFFF0000u, bad |= 1u << (p - P);
                        if (p + 1 >= P && (y & 0x7C000000u) == 0x7C000000u) y &= 0x0000FFFFu, bad |= 1u << (p + 1 - P);
                        halves[e] = y;
                    }
                }
                mma_16x8(o[j], halves, w[0], w[1]);
            }
            if (bad) atomicOr(&ctl.nonfinite[k & 1], bad);
            __syncwarp();
        }

        const uint32_t last = stage ? stage - S::kStage : (kFewStages - 1) * S::kStage;
        // The warps' parts meet in shared memory, in the stage that is free; then a
        // warp joins a row.
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) l[e] += __shfl_xor_sync(kFullMask, l[e], x);
            if (g == 0) {
                ctl.mx[warp][2 * c + e] = mx[e];
                ctl.l[warp][2 * c + e] = l[e];
            }
            float *to = reinterpret_cast<float *>(ring + last) +
                        (2 * c + e) * D + g * (D / 8);
#pragma unroll
            for (int j = 0; j < kSteps; j += 2)
                *reinterpret_cast<float4 *>(to + 2 * j) =
                    make_float4(o[j][e], o[j][2 + e], o[j + 1][e], o[j + 1][2 + e]);
        }
        if (lane == 0) ctl.stage[warp] = warp * kFewStages * S::kStage + last;
        __syncthreads();
        const int slot = 2 * cta + (k > 0), m = warp;
        if (m < rows) {
            float top = -INFINITY, sum = 0.0f;
#pragma unroll
            for (int i = 0; i < kFewWarps; ++i) top = fmaxf(top, ctl.mx[i][m]);
            const float shift = top == -INFINITY ? 0.0f : top;
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            const bool mine = lane < D / 4;
#pragma unroll
            for (int i = 0; i < kFewWarps; ++i) {
                const float f = exp2_approx(ctl.mx[i][m] - shift);
                sum = fmaf(f, ctl.l[i][m], sum);
                if (!mine) continue;
                const float4 y = *reinterpret_cast<const float4 *>(
                    smem + ctl.stage[i] + (m * D + lane * 4) * 4);
                x.x = fmaf(f, y.x, x.x), x.y = fmaf(f, y.y, x.y);
                x.z = fmaf(f, y.z, x.z), x.w = fmaf(f, y.w, x.w);
            }
            const int token = token0 + m / t.group, head = s.head * t.group + m % t.group;
            const int packed = s.q.row0 + token;
            for (unsigned e = ctl.nonfinite[k & 1] & ancestors_of(a, packed, token, s.q.len); e; e &= e - 1) {
                int tok;
                const int page = kv_page(a.cache, s.r, (long long)P + __ffs(e) - 1, &tok);
                if (page < 0 || !mine) continue;
                const unsigned char *v = a.cache.v + kv_offset(a.cache, page, tok, s.head) + lane * 4;
                const float f = __ldg(a.cache.v_scale + kv_scale_offset(a.cache, page, tok, s.head));
                float *to[4] = {&x.x, &x.y, &x.z, &x.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float y = e4m3_value(v[j]) * f;
                    if (!(y - y == 0.0f)) *to[j] += y;
                }
            }
            if (!whole) {
                if (mine)
                    reinterpret_cast<float4 *>(t.part_o)[((long long)slot * (D / 4) + lane) * kRowsPerTile + m] = x;
                if (lane == 0) {
                    t.part_ml[(long long)slot * 2 * kRowsPerTile + m] = top;
                    t.part_ml[((long long)slot * 2 + 1) * kRowsPerTile + m] = sum;
                }
            } else {
                const float by = sum == 0.0f ? 0.0f : 1.0f / sum;
                if (sum == 0.0f) x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                const __nv_bfloat162 u = __floats2bfloat162_rn(x.x * by, x.y * by);
                const __nv_bfloat162 v = __floats2bfloat162_rn(x.z * by, x.w * by);
                if (mine)
                    *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + packed * a.ld_out +
                                               (long long)head * D + lane * 4) =
                        make_uint2(*reinterpret_cast<const uint32_t *>(&u), *reinterpret_cast<const uint32_t *>(&v));
                if (lane == 0 && a.lse)
                    a.lse[(long long)packed * a.n_q_heads + head] =
                        sum == 0.0f ? -INFINITY : shift * kLn2 + logf(sum);
            }
        }
        if (tid == 0) {
            if (ctl.seg[k + 1 & 3].count == 0 && !whole) note_split(t, s, deal, lo, hi, k, token0, rows);
            leave(k + 2);
            ctl.nonfinite[k + 1 & 1] = 0;
        }
        __syncthreads();
    }
}

}  // namespace dspark
