// evict.cu -- a cache that is kept short: the attention weights that its positions gather
// step by step, and the eviction of the entries that gathered least.
//
// Gathering, for request r, kv head h and position p, over the window's rows that count
// and the head's query heads that see p:
//   weights_out_p = decay weights_p + sum exp(scale q . k_p - lse)
// with lse the rows' log sums that the attention left, so the terms are its softmax.
//
// weights_kernel   bfloat16 rows over bfloat16 or E4M3 keys of 64 or 128 elements, on the
//   matrix instruction of one warp, with positions as its rows and the window's (token,
//   head) rows as its columns, 64 at a time: a key is read once for all of them, and a
//   thread has the scores of few positions, so that the sum over rows is a sum in
//   registers.  The elements of a contraction may come in any order that both operands
//   share; here a thread's are contiguous, so that it copies what it multiplies itself, 16
//   bytes at a time and two steps ahead, and waits for no other thread.  Products are
//   exact in 32 bits: codes are halves as they are, and beside them queries are halves
//   brought to 2^14 by a power of two a row, so that what they lose is below 2^-39 of a
//   row's largest element.  A few rows leave most of the matrix instruction's rate unused:
//   tcgen05 would add barriers between warps.  Single tokens of 32 requests of up to 8192
//   over E4M3 keys, 8 kv heads (152 MB) take 45 us, 3.4 TB/s: a step's conversions and waits.
//   Windows of up to 9 over bfloat16 keys (287 MB) take 63 us, 4.5 TB/s, with HBM 57 % and
//   issue slots 47 % busy: neither is full, a warp's step and the uneven ends bound it.  (Loads into registers a step ahead instead of copies 66 and 81 us; three steps
//   under way, whose shared memory leaves one CTA an SM, 64 and 90.)
// weights_any_kernel   any types, strides, head and page sizes, in 32 bits throughout: a
//   warp a position, its key held in registers, one row and query head after another:
//   684 and 1097 us in those two cases.
//
// Eviction, for each (request, kv head): of n entries those `keep` stay that rank first by
// (fresh, weight, lower place).  An entry's rank is a 32-bit key (rank_key); the keep-th
// largest is found by its digits, and as many entries equal to it stay, in order, as are
// needed.  The entries that stay from place `keep` on then fill the places left below
// it, the i-th the i-th: so all reads lie at or behind place `keep` and all writes before
// it, entries move in any order and in parallel, and no more than have to.
//
// evict_select_kernel  a cluster of one to eight CTAs a (request, kv head), which hold the
//   ranks of its entries in shared memory: three passes for the digits (a histogram of each
//   beside them, integer counts, summed over the cluster), then entries equal to the border,
//   entries moved and the list of moves, each in the order of places by ballots and prefix
//   sums, and the ledger.  Latency bounds it (barriers and sums over the cluster, and an
//   SM's one CTA): 32 heads of 60000 to 131040 places take some 50 us of an eviction's 99 (with
//   the move).  That took 323 us with a CTA each that read them again in every pass, and 120
//   with ranks in the registers of eight CTAs, of which two in three clusters run at a time.
//   (Two histograms that lanes take in turns for the first digit: 102 us.)
// evict_select_any_kernel  a CTA a (request, kv head) of any length, which reads them again.
// evict_move_kernel    a CTA 128 moves of a (request, kv head): both slots looked up by a
//   thread, then the entries' pieces streamed by all.  HBM bounds it, 4.6 TB/s of reads and
//   writes of 128 bytes each here and there.  (64 moves a CTA 105 us for both, 256 98; eight
//   pieces of a thread under way 103.)

#include "kvcache.cuh"
#include "schedule.cuh"
#include "tensor.cuh"

namespace dspark {

// ------------------------------------------------------------- gathering

struct WeightsArgs {
    AttendArgs a;
    const float *lse;
    const int32_t *counts;
    float decay;
    const float *weights;
    float *weights_out;
    int length;
    const int32_t *pos;
    int32_t *positions;
    int span;  // positions of a CTA of weights_kernel
};

// How many rows of a window count, -1 if the request is left alone; with `report`,
// flags why.
__device__ __forceinline__ int counted(const WeightsArgs &t, const Window &w, int r, bool report) {
    if (w.hi != w.lo && !usable(t.a, w, report)) return -1;
    // (a request without rows still has a prefix that decays)
    const int n = t.counts ? __ldg(t.counts + r) : w.hi - w.lo;
    int bad = 0;
    if (n < 0 || n > w.hi - w.lo || w.P < 0) bad = DSPARK_STATUS_BAD_LEN;
    else if ((long long)w.P + n > t.length) bad = DSPARK_STATUS_CAPACITY;
    if (bad && report) flag(t.a.status, bad);
    return bad ? -1 : n;
}

constexpr int kWeightsWarps = 8;
constexpr int kWeightsPositions = 64;  // a CTA
constexpr int kWeightsSteps = DSPARK_MAX_HEAD_DIM / 32;

template <typename T, typename C>
__global__ void __launch_bounds__(kWeightsWarps * 32) weights_any_kernel(WeightsArgs t) {
    pdl_trigger();
    pdl_wait();
    const AttendArgs &a = t.a;
    const int r = blockIdx.z, kh = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Window w = load_window(a, r);
    const int n = counted(t, w, r, blockIdx.x == 0 && kh == 0 && threadIdx.x == 0);
    if (n < 0) return;
    const int D = a.cache.head_dim, G = a.n_q_heads / a.cache.n_kv_heads;
    const long long line = ((long long)r * a.cache.n_kv_heads + kh) * t.length;
    for (int i = warp; i < kWeightsPositions; i += kWeightsWarps) {
        const long long p = (long long)blockIdx.x * kWeightsPositions + i;
        if (p >= t.length) return;
        float sum = 0.0f;
        if (n > 0 && p < w.P + n) {
            int token;
            const int page = kv_page(a.cache, r, p, &token);
            if (page < 0 && lane == 0) flag(a.status, DSPARK_STATUS_BAD_INDEX);
            if (page >= 0) {
                const C *k = reinterpret_cast<const C *>(a.cache.k) + kv_offset(a.cache, page, token, kh);
                const float f =
                    sizeof(C) == 1 ? __ldg(a.cache.k_scale + kv_scale_offset(a.cache, page, token, kh)) : 1.0f;
                float kv[kWeightsSteps];
#pragma unroll
                for (int s = 0; s < kWeightsSteps; ++s) kv[s] = lane + 32 * s < D ? elem_value(k[lane + 32 * s]) * f : 0.0f;
                for (int j = 0; j < n; ++j) {
                    const int row = w.lo + j;
                    if (p >= w.P && !(ancestors_of(a, row, j, w.hi - w.lo) >> (p - w.P) & 1)) continue;
                    for (int g = 0; g < G; ++g) {
                        const int h = kh * G + g;
                        const T *q = static_cast<const T *>(a.q) + row * a.ld_q + (long long)h * D;
                        float s = 0.0f;
#pragma unroll
                        for (int e = 0; e < kWeightsSteps; ++e)
                            if (lane + 32 * e < D) s = fmaf(elem_value(q[lane + 32 * e]), kv[e], s);
                        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(kFullMask, s, x);
                        sum += expf(fmaf(s, a.scale, -t.lse[(long long)row * a.n_q_heads + h]));
                    }
                }
            }
        }
        if (lane == 0) {
            t.weights_out[line + p] = p < w.P ? fmaf(t.decay, t.weights[line + p], sum) : sum;
            if (t.positions && p >= w.P && p < w.P + n) t.positions[line + p] = __ldg(t.pos + w.lo + (p - w.P));
        }
    }
}

constexpr int kGatherWarps = 8, kGatherRows = 64;  // of a CTA; rows at a time
constexpr int kGatherStages = 2;                   // steps of a warp under way
constexpr int kGatherMost = 2048;                  // positions of a CTA

// x = a b + x: 16 x 16 times 16 x 8, halves or bfloat16.
template <bool kHalf>
__device__ __forceinline__ void mma_rows16(float (&x)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                           uint32_t b0, uint32_t b1) {
    if constexpr (kHalf)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%0,%1,%2,%3};"
            : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Shared memory of a CTA.  A step of a warp is kTiles times 16 positions, 4 KB at most.
template <int D, bool kQuant>
struct GatherShape {
    static constexpr int kTiles = kQuant ? 2 : 1, kStep = 16 * kTiles;
    static constexpr int kPieces = D / 32;                  // of eight query elements a lane
    static constexpr int kLoads = kQuant ? D / 64 : D / 32;  // of 16 bytes a lane and key
    uint4 keys[kGatherWarps][kGatherStages][2 * kTiles * kLoads][32];
    uint4 queries[kGatherRows / 8][kPieces][32];
    float lse[kGatherRows], factor[kGatherRows];
    unsigned seen[kGatherRows];  // the window's tokens that a row sees
    float scale[kGatherWarps][kGatherStages][32];
    float gathered[kGatherMost];  // by the rows before, where they are more than fit
};

template <int D, bool kQuant>
__global__ void __launch_bounds__(kGatherWarps * 32, 2) weights_kernel(WeightsArgs t) {
    using S = GatherShape<D, kQuant>;
    constexpr int kStep = S::kStep, kAll = kStep * kGatherWarps, kKeys = 2 * S::kTiles;
    extern __shared__ __align__(16) unsigned char smem[];
    S &sh = *reinterpret_cast<S *>(smem);
    pdl_trigger();
    pdl_wait();
    const AttendArgs &a = t.a;
    const int r = blockIdx.z, kh = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const Window w = load_window(a, r);
    const int n = counted(t, w, r, blockIdx.x == 0 && kh == 0 && tid == 0);
    if (n < 0) return;
    const int G = a.n_q_heads / a.cache.n_kv_heads, rows = n * G, len = w.hi - w.lo;
    const int first = blockIdx.x * t.span, last = min(first + t.span, t.length);
    const int end = n > 0 ? min(w.P + n, last) : first;  // from here on nothing is gathered
    const long long line = ((long long)r * a.cache.n_kv_heads + kh) * t.length;
    const int g = lane >> 2, q4 = lane & 3;  // a key's row of the matrix, its quarter of the elements

    // A position a lane.  The table's entry is loaded a step ahead of the key's copies.
    auto look_up = [&](int p) {
        return lane < kStep && p < end
                   ? __ldg(a.cache.table + (long long)r * a.cache.table_width + (unsigned)p / (unsigned)a.cache.page_size)
                   : -1;
    };
    // Starts the copies of keys g, g + 8, ... of the step, this lane's quarters; says which
    // positions have one.
    auto fetch = [&](int p, int page, int stage) {
        const bool in = lane < kStep && p < end, good = (unsigned)page < (unsigned)a.cache.n_pages;
        if (in && !good) flag(a.status, DSPARK_STATUS_BAD_INDEX);
        const int token = in ? (unsigned)p % (unsigned)a.cache.page_size : 0;
        const long long at = in && good ? kv_offset(a.cache, page, token, kh) : -1;
#pragma unroll
        for (int i = 0; i < kKeys; ++i) {
            const long long from = __shfl_sync(kFullMask, at, g + 8 * i);
            const unsigned char *k = a.cache.k + (from < 0 ? 0 : from) * (kQuant ? 1 : 2) + q4 * 16;
#pragma unroll
            for (int c = 0; c < S::kLoads; ++c)
                copy16(smem_addr(&sh.keys[warp][stage][i * S::kLoads + c][lane]), k + c * 64, from >= 0);
        }
        if constexpr (kQuant)
            copy4(smem_addr(&sh.scale[warp][stage][lane]),
                  a.cache.k_scale + (at < 0 ? 0 : kv_scale_offset(a.cache, page, token, kh)), at >= 0);
        copy16_commit();
        return __ballot_sync(kFullMask, at >= 0);
    };
    auto before = [&](int p) { return p < min(w.P, last) ? t.weights[line + p] : 0.0f; };
    auto put = [&](int p, float old, float sum) {
        if (p >= last) return;
        t.weights_out[line + p] = p < w.P ? fmaf(t.decay, old, sum) : sum;
        if (t.positions && p >= w.P && p < w.P + n) t.positions[line + p] = __ldg(t.pos + w.lo + (p - w.P));
    };

    const int own = first + warp * kStep;  // the warp's first position
    for (int row0 = 0; row0 < rows && first < end; row0 += kGatherRows) {
        const int count = min(rows - row0, kGatherRows), tiles = (count + 7) / 8;
        unsigned there[kGatherStages];  // of the stages' positions, those that have a key
        int page[kGatherStages + 1];
#pragma unroll
        for (int i = 0; i <= kGatherStages; ++i) page[i] = look_up(own + i * kAll + lane);
#pragma unroll
        for (int i = 0; i < kGatherStages; ++i) there[i] = fetch(own + i * kAll + lane, page[i], i);
        int next = page[kGatherStages];
        __syncthreads();
        for (int i = warp; i < tiles * 8; i += kGatherWarps) {
            // (places past the last row hold it again: against zeros, infinite keys would give NaN)
            const bool in = i < count;
            const int of = row0 + min(i, count - 1), token = of / G, row = w.lo + token, head = kh * G + of % G;
            const __nv_bfloat16 *q =
                static_cast<const __nv_bfloat16 *>(a.q) + (long long)row * a.ld_q + (long long)head * D;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (lane < D / 8) v = __ldg(reinterpret_cast<const uint4 *>(q) + lane);
            float by = 1.0f;
            if constexpr (kQuant) {
                const unsigned e[4] = {v.x, v.y, v.z, v.w};
                unsigned most = 0;
#pragma unroll
                for (int k = 0; k < 4; ++k) most = max(most, max(e[k] & 0x7FFFu, e[k] >> 16 & 0x7FFFu));
                most = __reduce_max_sync(kFullMask, most);
                // 2^(14 - its exponent); NaN and infinities stay what they are
                const int exponent = min(max((int)(most >> 7), 20), 254) - 127;
                const float up = __int_as_float((14 - exponent + 127) << 23);
                by = __int_as_float((exponent - 14 + 127) << 23);
                uint32_t h[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const __half2 two = __floats2half2_rn(__uint_as_float(e[k] << 16) * up,
                                                          __uint_as_float(e[k] & 0xFFFF0000u) * up);
                    h[k] = *reinterpret_cast<const uint32_t *>(&two);
                }
                v = make_uint4(h[0], h[1], h[2], h[3]);
            }
            // elements 8 lane.. are of the quarter (lane / 2) % 4 or lane % 4
            if (lane < D / 8) {
                const int quarter = kQuant ? lane / 2 % 4 : lane % 4;
                const int piece = kQuant ? lane / 8 * 2 + lane % 2 : lane / 4;
                sh.queries[i / 8][piece][i % 8 * 4 + quarter] = v;
            }
            if (lane == 0) {
                sh.lse[i] = in ? t.lse[(long long)row * a.n_q_heads + head] : INFINITY;
                sh.factor[i] = by;
                sh.seen[i] = in ? ancestors_of(a, row, token, len) : 0;
            }
        }
        __syncthreads();
        int stage = 0;
        for (int p0 = own; p0 < end; p0 += kAll) {
            const float old = before(p0 + lane);
            copy16_wait_but<kGatherStages - 1>();
            __syncwarp();  // (the scales are other lanes' copies)
            uint4 key[kKeys][S::kLoads];
            float scale[kKeys];
#pragma unroll
            for (int i = 0; i < kKeys; ++i) {
#pragma unroll
                for (int c = 0; c < S::kLoads; ++c) key[i][c] = sh.keys[warp][stage][i * S::kLoads + c][lane];
                scale[i] = kQuant ? sh.scale[warp][stage][g + 8 * i] : 1.0f;
            }
            __syncwarp();
            const unsigned now = there[0];
#pragma unroll
            for (int i = 0; i + 1 < kGatherStages; ++i) there[i] = there[i + 1];
            there[kGatherStages - 1] = fetch(p0 + kGatherStages * kAll + lane, next, stage);
            next = look_up(p0 + (kGatherStages + 1) * kAll + lane);
            if (++stage == kGatherStages) stage = 0;
            const bool in_window = p0 + kStep > w.P;
            float sum[kKeys] = {};
            for (int tile = 0; tile < tiles; ++tile) {
                float y[S::kTiles][4] = {};
#pragma unroll
                for (int c = 0; c < S::kLoads; ++c) {
                    if constexpr (kQuant) {
                        const uint4 b0 = sh.queries[tile][2 * c][lane], b1 = sh.queries[tile][2 * c + 1][lane];
#pragma unroll
                        for (int i = 0; i < S::kTiles; ++i) {
                            const uint4 u0 = eight_halves(make_uint2(key[2 * i][c].x, key[2 * i][c].y));
                            const uint4 v0 = eight_halves(make_uint2(key[2 * i + 1][c].x, key[2 * i + 1][c].y));
                            mma_rows16<true>(y[i], u0.x, v0.x, u0.y, v0.y, b0.x, b0.y);
                            mma_rows16<true>(y[i], u0.z, v0.z, u0.w, v0.w, b0.z, b0.w);
                            const uint4 u1 = eight_halves(make_uint2(key[2 * i][c].z, key[2 * i][c].w));
                            const uint4 v1 = eight_halves(make_uint2(key[2 * i + 1][c].z, key[2 * i + 1][c].w));
                            mma_rows16<true>(y[i], u1.x, v1.x, u1.y, v1.y, b1.x, b1.y);
                            mma_rows16<true>(y[i], u1.z, v1.z, u1.w, v1.w, b1.z, b1.w);
                        }
                    } else {
                        const uint4 b = sh.queries[tile][c][lane];
#pragma unroll
                        for (int i = 0; i < S::kTiles; ++i) {
                            const uint4 u = key[2 * i][c], v = key[2 * i + 1][c];
                            mma_rows16<false>(y[i], u.x, v.x, u.y, v.y, b.x, b.y);
                            mma_rows16<false>(y[i], u.z, v.z, u.w, v.w, b.z, b.w);
                        }
                    }
                }
                // scores of keys g + 8 i with rows 2 q4 and 2 q4 + 1 of the tile
                const int at_row = tile * 8 + 2 * q4;
                const float2 base = *reinterpret_cast<const float2 *>(&sh.lse[at_row]);
                const float2 by = *reinterpret_cast<const float2 *>(&sh.factor[at_row]);
                const uint2 sees = *reinterpret_cast<const uint2 *>(&sh.seen[at_row]);
#pragma unroll
                for (int i = 0; i < kKeys; ++i) {
                    float y0 = y[i / 2][i % 2 * 2], y1 = y[i / 2][i % 2 * 2 + 1];
                    if constexpr (kQuant) y0 *= by.x * scale[i], y1 *= by.y * scale[i];
                    // (the difference from lse before the change of base: where a term
                    // counts, it is small)
                    float e0 = exp2_approx(fmaf(y0, a.scale, -base.x) * kLog2e);
                    float e1 = exp2_approx(fmaf(y1, a.scale, -base.y) * kLog2e);
                    if (in_window) {
                        const int token = p0 + g + 8 * i - w.P;
                        if (token >= 0 && !(sees.x >> min(token, 31) & 1)) e0 = 0.0f;
                        if (token >= 0 && !(sees.y >> min(token, 31) & 1)) e1 = 0.0f;
                    }
                    sum[i] += e0 + e1;
                }
            }
            float mine = 0.0f;
#pragma unroll
            for (int i = 0; i < kKeys; ++i) {
                sum[i] += __shfl_xor_sync(kFullMask, sum[i], 1);
                sum[i] += __shfl_xor_sync(kFullMask, sum[i], 2);
                const float of = __shfl_sync(kFullMask, sum[i], lane % 8 * 4);
                if (lane / 8 == i) mine = of;
            }
            if (!(now >> lane & 1)) mine = 0.0f;
            const int p = p0 + lane;
            if (lane < kStep) {
                if (row0 > 0) mine += sh.gathered[p - first];
                if (row0 + kGatherRows < rows) sh.gathered[p - first] = mine;
                else put(p, old, mine);
            }
        }
        copy16_wait();
    }
    // positions of which no warp had one: all of them without rows
    for (int p = first + tid; p < last; p += kGatherWarps * 32)
        if (first + (p - first) / kStep * kStep >= end) put(p, before(p), 0.0f);
}

// -------------------------------------------------------------- eviction

struct EvictArgs {
    KvView cache;
    const int32_t *lens, *now;
    int B, keep, recent, length;
    const float *weights;
    float *weights_out;
    const int32_t *positions;
    int32_t *positions_out;
    int32_t *new_lens;
    int most;          // moves of a (request, kv head), at most
    int32_t *n_moves;  // [B][n_kv_heads]
    int32_t *cut;      // [B]: the new lengths, until every head has read the old
    int32_t *moves;    // [B][n_kv_heads][2][most]: places left, places they are filled from
    int32_t *status;
};

// Larger for what is to stay: the fresh first, then by weight, NaN last.
__device__ __forceinline__ unsigned rank_key(float w, int position, long long fresh_from) {
    if (position >= fresh_from) return 0xFFFFFFFFu;
    if (w != w) return 0;
    const unsigned b = __float_as_uint(w + 0.0f);  // (-0 is 0)
    return b >> 31 ? ~b : b | 0x80000000u;
}

constexpr int kSelectThreads = 1024, kSelectWarps = kSelectThreads / 32;
constexpr int kDigits = 2048;

__global__ void __launch_bounds__(kSelectThreads) evict_select_any_kernel(EvictArgs a) {
    __shared__ int hist[kDigits];
    __shared__ int scan[40], of_warp[2][kSelectWarps], found[2];
    pdl_trigger();
    pdl_wait();
    const int h = blockIdx.x, r = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int line = r * a.cache.n_kv_heads + h;
    const int n = __ldg(a.lens + r);
    const bool bad = n < 0 || n > a.length || n > (long long)a.cache.table_width * a.cache.page_size;
    const int end = bad ? n : min(n, a.keep);
    if (tid == 0) {
        a.n_moves[line] = 0;
        if (h == 0) a.cut[r] = end;
        if (bad && h == 0) flag(a.status, DSPARK_STATUS_BAD_LEN);
    }
    if (bad) return;
    const float *w_in = a.weights + (long long)line * a.length;
    const int32_t *p_in = a.positions + (long long)line * a.length;
    float *w_out = a.weights_out + (long long)line * a.length;
    int32_t *p_out = a.positions_out + (long long)line * a.length;
    const bool apart = a.weights_out != a.weights, apart_p = a.positions_out != a.positions;
    if (n > a.keep) {
        const long long fresh_from = (long long)__ldg(a.now + r) - a.recent;
        auto key = [&](int p) { return rank_key(w_in[p], p_in[p], fresh_from); };
        // the keep-th largest key, eleven, eleven and ten bits at a time
        unsigned border = 0;
        int need = a.keep;  // of the entries that agree with the border's digits so far
        bool nan = false;
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), bits = pass == 2 ? 10 : 11;
            for (int i = tid; i < kDigits; i += kSelectThreads) hist[i] = 0;
            __syncthreads();
#pragma unroll 4
            for (int p = tid; p < n; p += kSelectThreads) {
                const unsigned k = key(p);
                if (pass == 0) nan = nan || k == 0;
                else if (k >> (shift + bits) != border) continue;
                atomicAdd(&hist[k >> shift & ((1 << bits) - 1)], 1);
            }
            __syncthreads();
            // thread t holds the digits 2 t and 2 t + 1 from above
            const int digits = 1 << bits, top = digits - 1 - 2 * tid;
            const int c0 = top >= 0 ? hist[top] : 0, c1 = top >= 1 ? hist[top - 1] : 0;
            int total;
            const int above = block_exclusive_scan<int>(c0 + c1, scan, &total);
            if (above < need && above + c0 + c1 >= need) {
                const bool second = above + c0 < need;
                found[0] = second ? top - 1 : top;
                found[1] = need - above - (second ? c0 : 0);
            }
            __syncthreads();
            border = border << bits | (unsigned)found[0];
            need = found[1];
        }
        if (nan) flag(a.status, DSPARK_STATUS_BAD_INPUT);
        // each warp's run of places: how many keys equal the border before it
        const int run = (n + kSelectThreads - 1) / kSelectThreads * 32;
        const int from = min(warp * run, n), to = min(from + run, n);
        int mine = 0;
        for (int p = from + lane; p < to; p += 32) mine += key(p) == border;
        mine = __reduce_add_sync(kFullMask, mine);
        if (lane == 0) of_warp[0][warp] = mine;
        __syncthreads();
        int equal0 = 0;
        for (int i = 0; i < warp; ++i) equal0 += of_warp[0][i];
        __syncthreads();
        // whether the place of this lane's turn stays, in order along the run
        const unsigned before = lanemask_lt();
        auto stays = [&](int p, int *equal) {
            const unsigned k = p < to ? key(p) : 0;
            const bool eq = p < to && k == border;
            const unsigned eqs = __ballot_sync(kFullMask, eq);
            const bool yes = p < to && (k > border || (eq && *equal + __popc(eqs & before) < need));
            *equal += __popc(eqs);
            return yes;
        };
        int left = 0, moved = 0, equal = equal0;
        for (int p0 = from; p0 < to; p0 += 32) {
            const int p = p0 + lane;
            const bool yes = stays(p, &equal);
            left += __popc(__ballot_sync(kFullMask, p < min(to, a.keep) && !yes));
            moved += __popc(__ballot_sync(kFullMask, p >= a.keep && yes));
        }
        if (lane == 0) {
            of_warp[0][warp] = left;
            of_warp[1][warp] = moved;
        }
        __syncthreads();
        left = moved = 0;
        int total = 0;
        for (int i = 0; i < kSelectWarps; ++i) {
            if (i < warp) left += of_warp[0][i], moved += of_warp[1][i];
            total += of_warp[1][i];
        }
        int32_t *to_list = a.moves + (long long)line * 2 * a.most, *from_list = to_list + a.most;
        equal = equal0;
        for (int p0 = from; p0 < to; p0 += 32) {
            const int p = p0 + lane;
            const bool yes = stays(p, &equal);
            const bool is_left = p < min(to, a.keep) && !yes, is_moved = p >= a.keep && yes;
            const unsigned lefts = __ballot_sync(kFullMask, is_left), moves = __ballot_sync(kFullMask, is_moved);
            const int i = left + __popc(lefts & before), j = moved + __popc(moves & before);
            if (is_left && in_bounds(i, a.most, a.status)) to_list[i] = p;
            if (is_moved && in_bounds(j, a.most, a.status)) from_list[j] = p;
            left += __popc(lefts);
            moved += __popc(moves);
        }
        if (tid == 0) a.n_moves[line] = total;
        __syncthreads();
        // the ledger: entries that stay where they are, then those moved, then none
        if (apart || apart_p)
            for (int p = tid; p < end; p += kSelectThreads) {
                if (apart) w_out[p] = w_in[p];
                if (apart_p) p_out[p] = p_in[p];
            }
        __syncthreads();
        for (int i = tid; i < total; i += kSelectThreads) {
            const int p = to_list[i], of = from_list[i];
            w_out[p] = w_in[of];
            p_out[p] = p_in[of];
        }
        __syncthreads();
    } else if (apart || apart_p) {
        for (int p = tid; p < end; p += kSelectThreads) {
            if (apart) w_out[p] = w_in[p];
            if (apart_p) p_out[p] = p_in[p];
        }
    }
    for (int p = end + tid; p < a.length; p += kSelectThreads) {
        w_out[p] = 0.0f;
        p_out[p] = 0;
    }
}

// Places that a CTA holds, and the threads of one whose line is short, so that several
// fit an SM: 256 lines of 4113 places by 512 and by 1024 threads 19.4 and 29.3 us, 32 of them
// 15.5 and 16.8.
constexpr int kSelectPlaces = 48 * 1024, kShortPlaces = 8192, kShortThreads = 512;
constexpr int kSelectCtas = 8;  // of a cluster, at most

// The word of CTA `rank` of the cluster where this one has *own.
template <int kCtas>
__device__ __forceinline__ int word_of(const int *own, int rank) {
    return kCtas == 1 ? *own : (int)cluster_load(cluster_addr(smem_addr(own), rank));
}

template <int kCtas, int kThreads>
__global__ void __launch_bounds__(kThreads) evict_select_kernel(EvictArgs a) {
    extern __shared__ unsigned keys[];
    __shared__ int hist[2][kDigits];
    __shared__ long long wide[40];
    __shared__ int scan[40], found[2], counts[4];  // of this CTA: equal to the border; places left, moves
    pdl_trigger();
    pdl_wait();
    const int rank = blockIdx.x % kCtas, h = blockIdx.x / kCtas, r = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int line = r * a.cache.n_kv_heads + h;
    const int n = __ldg(a.lens + r);
    const bool bad = n < 0 || n > a.length || n > (long long)a.cache.table_width * a.cache.page_size;
    const int end = bad ? n : min(n, a.keep);
    if (tid == 0 && rank == 0) {
        a.n_moves[line] = 0;
        if (h == 0) a.cut[r] = end;
        if (bad && h == 0) flag(a.status, DSPARK_STATUS_BAD_LEN);
    }
    if (bad) return;  // (every CTA of the cluster)
    auto sync = [&]() {
        if constexpr (kCtas > 1) cluster_sync();
        else __syncthreads();
    };
    const float *w_in = a.weights + (long long)line * a.length;
    const int32_t *p_in = a.positions + (long long)line * a.length;
    float *w_out = a.weights_out + (long long)line * a.length;
    int32_t *p_out = a.positions_out + (long long)line * a.length;
    const bool apart = a.weights_out != a.weights, apart_p = a.positions_out != a.positions;
    const int whole = rank * kThreads + tid, threads = kCtas * kThreads;
    if (n > a.keep) {
        // this thread's places: from + 32 i, of the warp's run of consecutive ones, and
        // where their ranks lie
        const int per = (n + threads - 1) / threads, from = (whole - lane) * per + lane;
        const int have = min(max((n - from + 31) / 32, 0), per);
        unsigned *key = keys + warp * 32 * per + lane;
        const long long fresh_from = (long long)__ldg(a.now + r) - a.recent;
        // the keep-th largest key, eleven, eleven and ten bits at a time
        constexpr int kBits = 11, kLastBits = 10;
        static_assert(1 << kBits == kDigits && 2 * kBits + kLastBits == 32, "digits");
        for (int i = tid; i < kDigits; i += kThreads) hist[0][i] = 0;
        __syncthreads();
        int most = 0;  // (the fresh have one key, which is counted apart)
        bool nan = false;
        // (a short line's all at once: 256 lines of 4113 places 25 us at eight, 20.6 at sixteen)
        constexpr int kAhead = 16;
#pragma unroll 1
        for (int i = 0; i < have; i += kAhead) {
            float w[kAhead];
            int position[kAhead];
            const float *w_at = w_in + from + 32 * i;
            const int32_t *p_at = p_in + from + 32 * i;
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (i + k < have) {
                    w[k] = w_at[32 * k];
                    position[k] = p_at[32 * k];
                }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (i + k >= have) continue;
                const int p = from + 32 * (i + k);
                const unsigned rank = rank_key(w[k], position[k], fresh_from);
                key[32 * (i + k)] = rank;
                nan = nan || rank == 0;
                if (rank == 0xFFFFFFFFu) ++most;
                else atomicAdd(&hist[0][rank >> 32 - kBits], 1);
                // (the ledger of entries that stay where they are)
                if (apart && p < end) w_out[p] = w[k];
                if (apart_p && p < end) p_out[p] = position[k];
            }
        }
        if (nan) flag(a.status, DSPARK_STATUS_BAD_INPUT);
        auto there = [&](int i) { return i < have; };
        unsigned border = 0;
        int need = a.keep;  // of the entries that agree with the border's digits so far
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
            const int bits = pass == 2 ? kLastBits : kBits, shift = 32 - kBits * pass - bits;
            int *own = hist[pass & 1];
            if (pass > 0) {
                for (int i = tid; i < kDigits; i += kThreads) own[i] = 0;
                __syncthreads();
                most = 0;
#pragma unroll 4
                for (int i = 0; i < have; ++i) {
                    const unsigned k = key[32 * i];
                    if (k >> (shift + bits) != border) continue;
                    if (k == 0xFFFFFFFFu) ++most;
                    else atomicAdd(&own[k >> shift & ((1 << bits) - 1)], 1);
                }
            }
            most = __reduce_add_sync(kFullMask, most);
            if (lane == 0 && most) atomicAdd(&own[(1 << bits) - 1], most);
            sync();
            // thread t holds some digits in turn from above
            constexpr int kOwn = kDigits / kThreads;
            const int top = (1 << bits) - 1 - kOwn * tid;
            int c[kOwn] = {}, sum = 0;
            if (top >= 0)
#pragma unroll
                for (int k = 0; k < kOwn; ++k) {
#pragma unroll
                    for (int x = 0; x < kCtas; ++x) c[k] += word_of<kCtas>(&own[top - k], x);
                    sum += c[k];
                }
            int total, above = block_exclusive_scan<int>(sum, scan, &total);
#pragma unroll
            for (int k = 0; k < kOwn; ++k) {
                if (above < need && above + c[k] >= need) {
                    found[0] = top - k;
                    found[1] = need - above;
                }
                above += c[k];
            }
            __syncthreads();
            border = border << bits | (unsigned)found[0];
            need = found[1];
            __syncthreads();
        }
        // What comes before the warp's run in the cluster, in the order of places, by two
        // counts of each warp's (31 bits each: one scan), and the cluster's second count.
        auto before_warp = [&](long long mine, int which, int *all) {
            long long total;
            long long sum = block_exclusive_scan<long long>(lane == 0 ? mine : 0, wide, &total);
            sum = __shfl_sync(kFullMask, sum, 0);
            if (tid == 0) {
                counts[which] = (int)(total >> 32);
                counts[which + 1] = (int)total;
            }
            sync();
            *all = 0;
#pragma unroll
            for (int i = 0; i < kCtas; ++i) {
                const int a0 = word_of<kCtas>(&counts[which], i), a1 = word_of<kCtas>(&counts[which + 1], i);
                if (i < rank) sum += ((long long)a0 << 32) + a1;
                *all += a1;
            }
            return sum;
        };
        int mine = 0, all;
#pragma unroll 4
        for (int i = 0; i < per; ++i) mine += __popc(__ballot_sync(kFullMask, there(i) && key[32 * i] == border));
        int equal = (int)before_warp(mine, 0, &all);
        // which of the places stay: in the ranks' place
        const unsigned before = lanemask_lt();
        int left = 0, moved = 0;
#pragma unroll 4
        for (int i = 0; i < per; ++i) {
            const int p = from + 32 * i;
            const unsigned k = there(i) ? key[32 * i] : 0;
            const bool eq = there(i) && k == border;
            const unsigned eqs = __ballot_sync(kFullMask, eq);
            const bool yes = there(i) && (k > border || (eq && equal + __popc(eqs & before) < need));
            equal += __popc(eqs);
            if (there(i)) key[32 * i] = yes;
            left += __popc(__ballot_sync(kFullMask, there(i) && p < a.keep && !yes));
            moved += __popc(__ballot_sync(kFullMask, p >= a.keep && yes));
        }
        int total;
        const long long both = before_warp(((long long)left << 32) + moved, 2, &total);
        left = (int)(both >> 32);
        moved = (int)both;
        int32_t *to_list = a.moves + (long long)line * 2 * a.most, *from_list = to_list + a.most;
#pragma unroll 4
        for (int i = 0; i < per; ++i) {
            const int p = from + 32 * i;
            const bool yes = there(i) && key[32 * i];
            const bool is_left = there(i) && p < a.keep && !yes, is_moved = p >= a.keep && yes;
            const unsigned lefts = __ballot_sync(kFullMask, is_left), moves = __ballot_sync(kFullMask, is_moved);
            const int j = left + __popc(lefts & before), k = moved + __popc(moves & before);
            if (is_left && in_bounds(j, a.most, a.status)) to_list[j] = p;
            if (is_moved && in_bounds(k, a.most, a.status)) from_list[k] = p;
            left += __popc(lefts);
            moved += __popc(moves);
        }
        if (tid == 0 && rank == 0) a.n_moves[line] = total;
        sync();
        for (int i = whole; i < total; i += threads) {
            const int p = __ldcg(to_list + i), of = __ldcg(from_list + i);
            w_out[p] = w_in[of];
            p_out[p] = p_in[of];
        }
        sync();
    } else if (apart || apart_p) {
        for (int p = whole; p < end; p += threads) {
            if (apart) w_out[p] = w_in[p];
            if (apart_p) p_out[p] = p_in[p];
        }
    }
    for (int p = end + whole; p < a.length; p += threads) {
        w_out[p] = 0.0f;
        p_out[p] = 0;
    }
}

constexpr int kMoveThreads = 256, kMoves = 128;

// The entries' pieces of 16 bytes or of an element, four of a thread under way.
template <typename Piece>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(EvictArgs a, int elem_bytes) {
    __shared__ long long at[2][kMoves];
    pdl_trigger();
    pdl_wait();
    const int h = blockIdx.y, r = blockIdx.z, tid = threadIdx.x, line = r * a.cache.n_kv_heads + h;
    if (blockIdx.x == 0 && h == 0 && tid == 0) a.new_lens[r] = a.cut[r];
    const int n = min(a.n_moves[line] - (int)blockIdx.x * kMoves, kMoves);
    if (n <= 0) return;
    const KvView &c = a.cache;
    const int32_t *lists = a.moves + (long long)line * 2 * a.most + (long long)blockIdx.x * kMoves;
    if (tid < n) {
        int token[2], page[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            page[i] = kv_page(c, r, lists[(long long)i * a.most + tid], &token[i]);
            at[i][tid] = page[i] < 0 ? -1 : kv_offset(c, page[i], token[i], h) * elem_bytes;
        }
        if (page[0] < 0 || page[1] < 0) {
            flag(a.status, DSPARK_STATUS_BAD_INDEX);
            at[0][tid] = -1;
        } else if (c.k_scale) {
            const long long to = kv_scale_offset(c, page[0], token[0], h), of = kv_scale_offset(c, page[1], token[1], h);
            c.k_scale[to] = c.k_scale[of];
            c.v_scale[to] = c.v_scale[of];
        }
    }
    __syncthreads();
    const int pieces = c.head_dim * elem_bytes / (int)sizeof(Piece), all = n * 2 * pieces;
    constexpr int kAhead = 4;
    for (int base = tid; base < all; base += kAhead * kMoveThreads) {
        Piece x[kAhead];
        Piece *to[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = base + k * kMoveThreads;
            to[k] = nullptr;
            if (i >= all) continue;
            const int entry = i / (2 * pieces), rest = i - entry * 2 * pieces, v = rest >= pieces;
            if (at[0][entry] < 0) continue;
            unsigned char *pool = v ? c.v : c.k;
            to[k] = reinterpret_cast<Piece *>(pool + at[0][entry]) + (rest - v * pieces);
            x[k] = reinterpret_cast<const Piece *>(pool + at[1][entry])[rest - v * pieces];
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (to[k]) *to[k] = x[k];
    }
}

namespace {

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// Whether `out` is `in` itself, or shares none of its n words.
bool same_or_apart(const void *in, const void *out, int64_t n) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(in), y = reinterpret_cast<uintptr_t>(out), bytes = 4 * n;
    return x == y || x >= y + bytes || y >= x + bytes;
}

// Entries that can move: as many as are kept, or as lie behind them.
int most_moves(int keep, int length) { return length > keep ? min(keep, length - keep) : 0; }

// Whether weights_kernel takes a call's types, heads and layouts.
bool gather_fits(const AttendArgs &a, int dtype, const dspark_kv_cache &c) {
    if (dtype != DSPARK_DTYPE_BF16 || c.dtype == DSPARK_DTYPE_F32 || (c.head_dim != 64 && c.head_dim != 128))
        return false;
    const int e = kv_elem_bytes(c.dtype);
    for (int64_t s : {c.page_stride, c.token_stride, c.head_stride})
        if (s * e % 16) return false;
    return aligned(c.k, 16) && aligned(a.q, 16) && a.ld_q % 8 == 0;
}

template <int D, bool kQuant>
cudaError_t launch_gather(const WeightsArgs &t, cudaStream_t stream) {
    using S = GatherShape<D, kQuant>;
    cudaError_t e = ensure_smem(reinterpret_cast<const void *>(weights_kernel<D, kQuant>), sizeof(S),
                                29 + (D == 128) + 2 * kQuant);
    if (e != cudaSuccess) return e;
    // some four times as many CTAs as run at a time, of 256 to 2048 positions (32 requests,
    // twice, four and eight times as many: 53, 46 and 48 us; 8 windows 26, 26 and 30)
    const long long all = (long long)t.length * t.a.cache.n_kv_heads * t.a.B / (8 * sm_count());
    WeightsArgs u = t;
    u.span = (int)min(max((all + 255) / 256, 1ll), (long long)(kGatherMost / 256)) * 256;
    const dim3 grid((t.length + u.span - 1) / u.span, t.a.cache.n_kv_heads, t.a.B);
    return launch_pdl(weights_kernel<D, kQuant>, grid, dim3(kGatherWarps * 32), sizeof(S), stream, u);
}

template <typename T>
cudaError_t launch_weights(const WeightsArgs &t, int cache_dtype, cudaStream_t stream) {
    const dim3 grid((t.length + kWeightsPositions - 1) / kWeightsPositions, t.a.cache.n_kv_heads, t.a.B);
    const dim3 block(kWeightsWarps * 32);
    if (cache_dtype == DSPARK_DTYPE_BF16)
        return launch_pdl(weights_any_kernel<T, __nv_bfloat16>, grid, block, 0, stream, t);
    if (cache_dtype == DSPARK_DTYPE_F32) return launch_pdl(weights_any_kernel<T, float>, grid, block, 0, stream, t);
    return launch_pdl(weights_any_kernel<T, e4m3>, grid, block, 0, stream, t);
}

template <int kCtas, int kThreads>
cudaError_t launch_select(const EvictArgs &a, cudaStream_t stream) {
    constexpr int kMost = kThreads == kShortThreads ? kShortPlaces : kSelectPlaces;
    constexpr int kSlot = 33 + (kThreads == kShortThreads ? 0 : kCtas == 1 ? 1 : kCtas == 2 ? 2 : kCtas == 4 ? 3 : 4);
    // (a warp's run is whole, and as long as any other's)
    const int run = (a.length + kCtas * kThreads - 1) / (kCtas * kThreads);
    const size_t smem = (size_t)run * kThreads * 4;
    cudaError_t e = ensure_smem(reinterpret_cast<const void *>(evict_select_kernel<kCtas, kThreads>), 4 * kMost, kSlot);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.cache.n_kv_heads * kCtas, a.B);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {kCtas, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = kCtas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, evict_select_kernel<kCtas, kThreads>, a);
}

cudaError_t launch_select_any(const EvictArgs &a, cudaStream_t stream) {
    return launch_pdl(evict_select_any_kernel, dim3(a.cache.n_kv_heads, a.B), dim3(kSelectThreads), 0, stream, a);
}

template <typename Piece>
cudaError_t launch_moves(const EvictArgs &a, int elem_bytes, cudaStream_t stream) {
    const dim3 grid(max((a.most + kMoves - 1) / kMoves, 1), a.cache.n_kv_heads, a.B);
    return launch_pdl(evict_move_kernel<Piece>, grid, dim3(kMoveThreads), 0, stream, a, elem_bytes);
}

}  // namespace

}  // namespace dspark

using namespace dspark;

extern "C" int dspark_attention_weights(const void *q, int64_t ld_q, int32_t dtype, int32_t n_q_heads,
                                        int32_t max_rows, const int32_t *cu_seqlens, const int32_t *prefix_lens,
                                        int32_t B, const uint32_t *ancestors, float scale,
                                        const dspark_kv_cache *cache, const float *lse, const int32_t *counts,
                                        float decay, const float *weights, float *weights_out, int32_t length,
                                        const int32_t *pos, int32_t *positions, int32_t *status, void *stream) {
    const int rc = kv_check(cache);
    if (rc != DSPARK_OK) return rc;
    if (!q || !lse || !weights || !weights_out || !cu_seqlens || !prefix_lens || !status || max_rows < 0 ||
        B < 1 || B > cache->n_requests || n_q_heads < 1 || n_q_heads % cache->n_kv_heads || length < 1)
        return DSPARK_ERR_INVALID_ARG;
    if (dtype != DSPARK_DTYPE_BF16 && dtype != DSPARK_DTYPE_F32) return DSPARK_ERR_INVALID_ARG;
    if (ld_q < (int64_t)n_q_heads * cache->head_dim || (pos != nullptr) != (positions != nullptr))
        return DSPARK_ERR_INVALID_ARG;
    if (!(scale - scale == 0.0f) || !(decay - decay == 0.0f)) return DSPARK_ERR_INVALID_ARG;
    if (!same_or_apart(weights, weights_out, (int64_t)B * cache->n_kv_heads * length)) return DSPARK_ERR_INVALID_ARG;
    if (n_q_heads > 65535 || B > 65535 || length > (1 << 30)) return DSPARK_ERR_UNSUPPORTED;
    WeightsArgs t;
    AttendArgs &a = t.a;
    a.q = q;
    a.ld_q = ld_q;
    a.out = nullptr;
    a.ld_out = 0;
    a.lse = nullptr;
    a.cu = cu_seqlens;
    a.prefix = prefix_lens;
    a.ancestors = ancestors;
    a.B = B;
    a.n_q_heads = n_q_heads;
    a.max_rows = max_rows;
    a.scale = scale;
    a.cache = kv_view(*cache);
    a.status = status;
    t.lse = lse;
    t.counts = counts;
    t.decay = decay;
    t.weights = weights;
    t.weights_out = weights_out;
    t.length = length;
    t.pos = pos;
    t.positions = positions;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool quant = cache->dtype == DSPARK_DTYPE_E4M3, small = cache->head_dim == 64;
    cudaError_t e;
    if (gather_fits(a, dtype, *cache))
        e = quant ? small ? launch_gather<64, true>(t, st) : launch_gather<128, true>(t, st)
            : small ? launch_gather<64, false>(t, st)
                    : launch_gather<128, false>(t, st);
    else
        e = dtype == DSPARK_DTYPE_BF16 ? launch_weights<__nv_bfloat16>(t, cache->dtype, st)
                                       : launch_weights<float>(t, cache->dtype, st);
    return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}

extern "C" size_t dspark_kv_evict_workspace_bytes(int32_t B, int32_t n_kv_heads, int32_t length) {
    if (B < 1 || n_kv_heads < 1 || length < 1) return 0;
    const size_t lines = (size_t)B * n_kv_heads;
    return round256(B * 4) + round256(lines * 4) + round256(lines * 2 * (length / 2) * 4);
}

extern "C" int dspark_kv_evict(const dspark_kv_cache *cache, const int32_t *lens, const int32_t *now, int32_t B,
                               int32_t keep, int32_t recent, const float *weights, float *weights_out,
                               const int32_t *positions, int32_t *positions_out, int32_t length,
                               int32_t *new_lens, void *workspace, size_t workspace_bytes, int32_t *status,
                               void *stream) {
    const int rc = kv_check(cache);
    if (rc != DSPARK_OK) return rc;
    if (!lens || !now || !weights || !weights_out || !positions || !positions_out || !new_lens || !status ||
        B < 1 || B > cache->n_requests || length < 1 || keep < 1 || recent < 0 || recent > keep)
        return DSPARK_ERR_INVALID_ARG;
    const int64_t words = (int64_t)B * cache->n_kv_heads * length;
    if (!same_or_apart(weights, weights_out, words) || !same_or_apart(positions, positions_out, words))
        return DSPARK_ERR_INVALID_ARG;
    if (cache->n_kv_heads > 65535 || B > 65535 || length > (1 << 30)) return DSPARK_ERR_UNSUPPORTED;
    if (!workspace || !aligned(workspace, 256) ||
        workspace_bytes < dspark_kv_evict_workspace_bytes(B, cache->n_kv_heads, length))
        return DSPARK_ERR_WORKSPACE;
    EvictArgs a;
    a.cache = kv_view(*cache);
    if (cache->dtype != DSPARK_DTYPE_E4M3) a.cache.k_scale = a.cache.v_scale = nullptr;
    a.lens = lens;
    a.now = now;
    a.B = B;
    a.keep = keep;
    a.recent = recent;
    a.length = length;
    a.weights = weights;
    a.weights_out = weights_out;
    a.positions = positions;
    a.positions_out = positions_out;
    a.new_lens = new_lens;
    a.most = most_moves(keep, length);
    const size_t lines = (size_t)B * cache->n_kv_heads;
    unsigned char *w = static_cast<unsigned char *>(workspace);
    a.cut = reinterpret_cast<int32_t *>(w);
    a.n_moves = reinterpret_cast<int32_t *>(w + round256(B * 4));
    a.moves = reinterpret_cast<int32_t *>(w + round256(B * 4) + round256(lines * 4));
    a.status = status;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    // as few CTAs a line as hold it, or more while there are SMs for them and each has
    // kShortPlaces or more.  Eight lines of up to 131040 places by 4 and 8 CTAs 57 and 52 us,
    // 32 of them 99 and 156; 128 of up to 40000 by 1, 2, 4: 161, 176 and 210.
    int ctas = 1;
    while (ctas < kSelectCtas && ((long long)ctas * kSelectPlaces < length ||
                                  ((long long)2 * ctas * lines <= sm_count() && length >= 2 * ctas * kShortPlaces)))
        ctas *= 2;
    cudaError_t e = length <= kShortPlaces                          ? launch_select<1, kShortThreads>(a, st)
                    : (long long)ctas * kSelectPlaces < length ? launch_select_any(a, st)
                    : ctas == 1                                     ? launch_select<1, kSelectThreads>(a, st)
                    : ctas == 2                                     ? launch_select<2, kSelectThreads>(a, st)
                    : ctas == 4                                     ? launch_select<4, kSelectThreads>(a, st)
                                                                    : launch_select<8, kSelectThreads>(a, st);
    if (e == cudaSuccess) {
        const int elem = kv_elem_bytes(cache->dtype);
        const bool wide = cache->head_dim * elem % 16 == 0 && aligned(cache->k, 16) && aligned(cache->v, 16) &&
                          cache->page_stride * elem % 16 == 0 && cache->token_stride * elem % 16 == 0 &&
                          cache->head_stride * elem % 16 == 0;
        e = wide        ? launch_moves<uint4>(a, elem, st)
            : elem == 4 ? launch_moves<uint32_t>(a, elem, st)
            : elem == 2 ? launch_moves<uint16_t>(a, elem, st)
                        : launch_moves<uint8_t>(a, elem, st);
    }
    return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
