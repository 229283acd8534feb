// prompt.cu -- causal attention of ragged prompts over keys and values of every head,
// with a key part that all heads share: the expanded form over a latent cache's rows.
//
// Query i of n over m keys sees keys j <= m - n + i.  With q = [q_k | q_s], of kv head g:
//   s_j = scale (q_k . k_jg + q_s . k_shared_j),  mx = max s_j,  l = sum exp(s_j - mx)
//   out = sum exp(s_j - mx) v_jg / l,             lse = mx + ln l
//
// prompt_any_kernel   any types, strides and dimensions, and requests of few scores where most
//   are short; in 32 bits throughout: a CTA a (row, query head), its four warps take every
//   fourth key, each with a running maximum and sum, joined at the end.  Each reads its keys
//   itself: 4 prompts of up to 128 tokens 67 us (the next 14), two of 8192 with 32 heads 459
//   ms (1.33).
//
// prompt_tensor_kernel   bfloat16 with keys of 128 (and a shared part of 64 or none) and
//   values of 128, on the tensor cores of two CTAs at a time.  A job is a (request, query
//   head) and 512 of its queries, two tiles of 256, of which a CTA has 128 each; a step is
//   128 keys:  S = Q K^T into tensor memory, then
//     y = S c   m' = max(m, max y)   w = 2^(y - m')   l = l 2^(m - m') + sum w
//     O = O 2^(m - m') + W V
//   with W written over S in tensor memory and O kept there.  m moves only when a row's
//   maximum grows by 2^kLazy (until then w may pass 1, and O is not touched).  One tile's
//   softmax runs beside the other tile's products.  A CTA holds half of either product's
//   right operand (64 keys; 64 of the values' elements), so that it is fetched once for 512
//   queries and read from shared memory at three quarters of its bandwidth, not at all of it.
//   One warp copies (TMA), one of the first CTA issues, four a tile do the softmax, a thread
//   a row.  Jobs with the most keys come first.
//   Two prompts of up to 8192 new tokens behind up to 4000 earlier ones, 32 heads (1782
//   GFLOP) take 1315 to 1377 us, 1.29 to 1.36 PFLOP/s, 0.68 to 0.72 of the measured rate.
//   What bounds it: a step of two tiles takes 1.8 us, 3700 cycles, of which its products
//   are 2560 (20 of 16 x 256 x 128 a tile, 64 cycles each).  The rest is a tile's chain, 1400
//   cycles from scores to weights, its 1280 of products and the barriers between.  And some
//   25 us of every job are outside of that (begin, what the diagonal's steps add, the last
//   outputs): calls of one job a pair take 40, 85 and 256 us with 1024, 4096 and 16384 keys.
//   Here a pair has ten jobs and 586 steps, 1050 us of steps and 250 of jobs, before the
//   uneven end.  The tensor cores are busy for 61 % of the kernel.  (Weights handed to the
//   product in halves: 1510 us.  Half of the exponentials left out, in an experiment: 1232,
//   so it is not they.)

#include "kvcache.cuh"
#include "tensor.cuh"
#include "tensormap.cuh"

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
    int split;  // both kernels are launched: requests of few scores are the first's
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

// Where both kernels are launched, which one a request is for: by its scores, which cost
// the kernel without tensor cores 0.25 to 0.37 ns each (with all SMs, a head) and the other
// next to nothing beside its 150 ns a job.  256 requests of 16 heads, us, without and with:
//   20 queries over 20 keys 470 and 639, 22 over 23 569 and 638, 26 over 26 700 and 643
//   4 over 100 555 and 628, over 128 696 and 624;  one over 400 602 and 884, over 512 765 and
//   698, over 640 953 and 781
// so that about 512 the two differ by a tenth either way.
constexpr int kFewScores = 512;
__device__ __forceinline__ bool few_scores(const PromptRange &w) {
    return (long long)(w.hi - w.lo) * (w.k1 - w.k0) <= kFewScores;
}
// Other requests have at least so many queries and keys together (twice the root).
constexpr int kManyTokens = 46;

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
    if (!usable(a, w, false) || row < w.lo || (a.split && !few_scores(w))) return;
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

// --------------------------------------------------- tensor-core kernel

constexpr int kPromptTile = 256, kPromptBlock = 2 * kPromptTile;  // queries a tile, a job
constexpr int kPromptKeys = 128;                                  // a step
constexpr int kPromptDim = 128, kPromptShared = 64;
constexpr int kPromptStages = 3;
constexpr int kRowsChunk = 128 * 128, kKeysChunk = 64 * 128;  // bytes of 64 elements of 128 rows, of 64 keys
constexpr int kPromptThreads = 320, kPromptCopyWarp = 8, kPromptMatrixWarp = 9;
constexpr int kPromptScoreCol = 0, kPromptOutCol = 256;  // columns of tensor memory, a tile's 128 on
constexpr int kDiagonal = kPromptBlock / kPromptKeys + 1;  // steps of a job that some query sees a part of

// Shared memory of a CTA: the queries of both tiles, rings of keys and values, control.
template <bool kShared>
struct PromptShape {
    static constexpr int kParts = 2 + kShared;  // of 64 elements of a key
    static constexpr int kQBytes = kParts * kRowsChunk;
    static constexpr int kKeyBytes = kParts * kKeysChunk, kValueBytes = kPromptKeys * 128;
    static constexpr int kKeyAt = 2 * kQBytes;
    static constexpr int kValueAt = kKeyAt + kPromptStages * kKeyBytes;
    static constexpr int kControl = kValueAt + kPromptStages * kValueBytes;
    static constexpr int kTotal = kControl + 2048;
    static_assert(kTotal <= 227 * 1024, "shared memory");
};

// Barriers that the issuing warp waits on are the first CTA's; those that it commits to
// are each CTA's own.
struct alignas(16) PromptControl {
    unsigned long long q_full[2], key_full[kPromptStages], value_full[kPromptStages], p_ready[2];  // the first's
    unsigned long long key_empty[kPromptStages], value_empty[kPromptStages], s_full[2], o_done[2], value_seen, drain;
    unsigned tmem;
    int abort;
    int request, block;  // of the job
    unsigned nonfinite[kDiagonal][kPromptKeys / 32];  // keys whose values were zeroed in either CTA
    long long scan[40];
};
static_assert(sizeof(PromptControl) <= 2048, "control area");

// Whether a row's score of a key is -inf.
__device__ __noinline__ bool weightless(const PromptArgs &a, int row, int head, long long key) {
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + row * a.ld_q +
                             (long long)head * (a.key_dim + a.shared_dim);
    const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(a.k) + key * a.ld_k + head / a.group * a.hs_k;
    const __nv_bfloat16 *c = static_cast<const __nv_bfloat16 *>(a.shared) + key * a.ld_shared;
    float s = 0.0f;
    for (int i = 0; i < a.key_dim; ++i) s = fmaf(elem_value(q[i]), elem_value(k[i]), s);
    for (int i = 0; i < a.shared_dim; ++i) s = fmaf(elem_value(q[a.key_dim + i]), elem_value(c[i]), s);
    return s * a.scale == -INFINITY;
}

template <bool kShared>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPromptThreads, 1)
prompt_tensor_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_s, const __grid_constant__ CUtensorMap map_v,
                     const PromptArgs a) {
    using S = PromptShape<kShared>;
    extern __shared__ __align__(1024) unsigned char smem[];
    PromptControl &ctl = *reinterpret_cast<PromptControl *>(smem + S::kControl);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)cluster_rank(), head = blockIdx.x / 2 % a.n_q_heads;
    const long long cluster = blockIdx.x / 2 / a.n_q_heads;  // the job's place among all blocks of 512 queries
    const uint32_t base = smem_addr(smem);
    if (tid == 0) {
        for (int i = 0; i < kPromptStages; ++i) {
            mbar_init(smem_addr(&ctl.key_full[i]), 1);
            mbar_init(smem_addr(&ctl.value_full[i]), 1);
            mbar_init(smem_addr(&ctl.key_empty[i]), 1);
            mbar_init(smem_addr(&ctl.value_empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&ctl.q_full[i]), 1);
            mbar_init(smem_addr(&ctl.p_ready[i]), 8);
            mbar_init(smem_addr(&ctl.s_full[i]), 1);
            mbar_init(smem_addr(&ctl.o_done[i]), 1);
        }
        mbar_init(smem_addr(&ctl.value_seen), 1);
        mbar_init(smem_addr(&ctl.drain), 1);
        ctl.abort = 0;
        ctl.request = -1;
        fence_mbar_init();
        prefetch_map(&map_q);
        prefetch_map(&map_k);
        prefetch_map(&map_v);
        if (kShared) prefetch_map(&map_s);
    }
    for (int i = tid; i < kDiagonal * kPromptKeys / 32; i += kPromptThreads) (&ctl.nonfinite[0][0])[i] = 0;
    __syncthreads();
    pdl_wait();
    {  // the request: each thread counts the blocks of a run of them
        const int per = (a.B + kPromptThreads - 1) / kPromptThreads;
        auto blocks = [&](int r, bool report) {
            const PromptRange w = load_range(a, r);
            if (!usable(a, w, report) || (a.split && few_scores(w))) return 0;
            return (w.hi - w.lo + kPromptBlock - 1) / kPromptBlock;
        };
        long long mine = 0, total;
        for (int i = 0, r = tid * per; i < per && r < a.B; ++i, ++r) mine += blocks(r, blockIdx.x == 0);
        long long before = block_exclusive_scan<long long>(mine, ctl.scan, &total);
        if (cluster >= before && cluster < before + mine)
            for (int r = tid * per;; ++r) {
                const int n = blocks(r, false);
                if (cluster < before + n) {
                    ctl.request = r;
                    ctl.block = n - 1 - (int)(cluster - before);  // the last queries see most keys
                    break;
                }
                before += n;
            }
    }
    __syncthreads();
    if (ctl.request < 0) return;  // (both CTAs)
    if (warp == kPromptMatrixWarp) tmem_alloc_pair(smem_addr(&ctl.tmem), 512);
    pdl_trigger();
    __syncthreads();
    cluster_sync();  // both CTAs' barriers are there
    tmem_fence_after();
    const uint32_t tmem = ctl.tmem;
    volatile int *abort = &ctl.abort;
    bool ok = true;
    auto wait = [&](unsigned long long *bar, unsigned parity) {
        return ok = warp_wait(ok, smem_addr(bar), parity, abort, a.status);
    };
    auto first_cta = [&](unsigned long long *bar) { return cluster_addr(smem_addr(bar), 0); };
    const PromptRange w = load_range(a, ctl.request);
    const int n = w.hi - w.lo, m = w.k1 - w.k0, row0 = ctl.block * kPromptBlock;
    // query i sees keys 0..i + ahead
    const int ahead = m - n;
    // steps of tile t: up to the last key that its last query sees
    auto steps_of = [&](int t) {
        const int last = min(row0 + (t + 1) * kPromptTile, n) - 1;
        return last < row0 + t * kPromptTile ? 0 : max(last + ahead + kPromptKeys, 0) / kPromptKeys;
    };
    const int steps[2] = {steps_of(0), steps_of(1)}, most = max(steps[0], steps[1]);
    // from this step on some query does not see all keys
    const int diagonal = max(row0 + ahead + 1, 0) / kPromptKeys;

    if (warp == kPromptCopyWarp) {
        // ------------------------------------------------ copy warp
        const int group = head / a.group;
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
            if (!steps[t]) continue;
            if (rank == 0 && lane == 0) mbar_expect(smem_addr(&ctl.q_full[t]), 2 * S::kQBytes);
            __syncwarp();
            if (lane < S::kParts)
                tma_load_4d_pair(base + t * S::kQBytes + lane * kRowsChunk, &map_q, lane * 64,
                                 w.lo + row0 + t * kPromptTile + rank * 128, head, 0, first_cta(&ctl.q_full[t]));
        }
        int stage = 0;
        unsigned parity = 1;
        for (int j = 0; j < most; ++j) {
            if (!wait(&ctl.key_empty[stage], parity)) break;
            if (rank == 0 && lane == 0) mbar_expect(smem_addr(&ctl.key_full[stage]), 2 * S::kKeyBytes);
            __syncwarp();
            const int key = w.k0 + j * kPromptKeys;
            if (lane < S::kParts)
                tma_load_4d_pair(base + S::kKeyAt + stage * S::kKeyBytes + lane * kKeysChunk,
                                 lane < 2 ? &map_k : &map_s, lane < 2 ? lane * 64 : 0, key + rank * 64,
                                 lane < 2 ? group : 0, 0, first_cta(&ctl.key_full[stage]));
            if (!wait(&ctl.value_empty[stage], parity)) break;
            if (rank == 0 && lane == 0) mbar_expect(smem_addr(&ctl.value_full[stage]), 2 * S::kValueBytes);
            __syncwarp();
            if (lane == 0)
                tma_load_4d_pair(base + S::kValueAt + stage * S::kValueBytes, &map_v, rank * 64, key, group, 0,
                                 first_cta(&ctl.value_full[stage]));
            if (++stage == kPromptStages) stage = 0, parity ^= 1;
        }
        if (!ok && rank == 0 && lane == 0) {
            // copies still under way write the pair's buffers (each wait ends by itself; the
            // CTAs leave together)
            for (int t = 0; t < 2; ++t)
                if (steps[t]) mbar_wait(smem_addr(&ctl.q_full[t]), 0, kWaitLimitNs / 4);
            for (int p = 0; p < 2; ++p)
                for (int i = 0; i < kPromptStages; ++i) {
                    mbar_wait(smem_addr(&ctl.key_full[i]), p, kWaitLimitNs / 4);
                    mbar_wait(smem_addr(&ctl.value_full[i]), p, kWaitLimitNs / 4);
                }
        }
    } else if (warp == kPromptMatrixWarp) {
        // ---------------------------------------------- matrix warp
        // Keeps step as a whole, so that addresses stay in uniform registers; one lane
        // issues.  A tile's products of a step: its output with the last step's weights, then
        // its scores, while the other tile's weights are computed.
        if (rank == 0) {
            constexpr uint32_t score_word = mma_word(true, kPromptKeys, false) + kPairOf128;
            constexpr uint32_t value_word = mma_word(true, kPromptDim, true) + kPairOf128;
            const uint32_t ubase = __shfl_sync(kFullMask, base, 0), utmem = __shfl_sync(kFullMask, tmem, 0);
            const bool leader = elect_one();
            const uint64_t desc_q = smem_operand(ubase, 16, 128);
            const uint64_t desc_k = smem_operand(ubase + S::kKeyAt, 16, 128);
            const uint64_t desc_v = smem_operand(ubase + S::kValueAt, 16, 128);
            int key_stage = 0, value_stage = 0;
            unsigned key_parity = 0, value_parity = 0;
            for (int j = 0; j <= most && ok; ++j) {
                // step j - 1's weights and values, step j's keys
#pragma unroll 1
                for (int t = 0; t < 2; ++t) {
                    if (j > 0 && j <= steps[t]) {
                        const bool first = t == 0 || steps[0] < j, last = t == 1 || steps[1] < j;
                        if (first) {
                            if (!wait(&ctl.value_full[value_stage], value_parity)) break;
                            if (lane < 2) cluster_arrive(cluster_addr(smem_addr(&ctl.value_seen), lane));
                        }
                        if (!wait(&ctl.p_ready[t], j - 1)) break;
                        tmem_fence_after();
                        const uint64_t v = desc_v + value_stage * (S::kValueBytes >> 4);
                        if (leader) {
#pragma unroll
                            for (int k = 0; k < kPromptKeys / 16; ++k)
                                mma_pair_ts(utmem + kPromptOutCol + t * 128, utmem + kPromptScoreCol + t * 128 + k * 8,
                                            v + (k * 16 * 128 >> 4), value_word, j > 1 || k > 0);
                            if (last) mma_pair_commit(smem_addr(&ctl.value_empty[value_stage]));
                            if (j == steps[t]) mma_pair_commit(smem_addr(&ctl.o_done[t]));
                        }
                        __syncwarp();
                        if (last && ++value_stage == kPromptStages) value_stage = 0, value_parity ^= 1;
                    }
                    if (j < steps[t]) {
                        const bool first = t == 0 || steps[0] <= j, last = t == 1 || steps[1] <= j;
                        if (j == 0 && !wait(&ctl.q_full[t], 0)) break;
                        if (first && !wait(&ctl.key_full[key_stage], key_parity)) break;
                        tmem_fence_after();
                        const uint64_t q = desc_q + t * (S::kQBytes >> 4);
                        const uint64_t key = desc_k + key_stage * (S::kKeyBytes >> 4);
                        if (leader) {
#pragma unroll
                            for (int k = 0; k < 4 * S::kParts; ++k)
                                mma_pair_ss(utmem + kPromptScoreCol + t * 128,
                                            q + (k / 4 * kRowsChunk + k % 4 * 32 >> 4),
                                            key + (k / 4 * kKeysChunk + k % 4 * 32 >> 4), score_word, k > 0);
                            mma_pair_commit(smem_addr(&ctl.s_full[t]));
                            if (last) mma_pair_commit(smem_addr(&ctl.key_empty[key_stage]));
                        }
                        __syncwarp();
                        if (last && ++key_stage == kPromptStages) key_stage = 0, key_parity ^= 1;
                    }
                }
            }
            // after a timeout: products still under way write tensor memory and barriers of
            // the pair
            if (!ok && leader) {
                mma_pair_commit(smem_addr(&ctl.drain));
                mbar_wait(smem_addr(&ctl.drain), 0);
            }
            __syncwarp();
        }
    } else {
        // --------------------------------------------- softmax warps
        const int t = warp >> 2, count = steps[t];
        const uint32_t lanes = tmem + ((uint32_t)(warp % 4 * 32) << 16);
        const uint32_t scores = lanes + kPromptScoreCol + t * 128, outputs = lanes + kPromptOutCol + t * 128;
        const float c = fmaxf(fabsf(a.scale) * kLog2e, 0x1p-100f);  // 0 would turn -inf into NaN
        const bool negative = a.scale < 0.0f;
        const int row = row0 + t * kPromptTile + rank * 128 + tid % 128;  // of the request's queries
        const int sees = row + ahead + 1;                                 // keys
        float mx = -INFINITY, l = 0.0f;  // running maximum (to base 2), sum
        for (int j = 0; j < count; ++j) {
            if (!wait(&ctl.s_full[t], j)) break;
            tmem_fence_after();
            uint32_t x[128];
#pragma unroll
            for (int k = 0; k < 4; ++k) tmem_load32(scores + 32 * k, x + 32 * k);
#pragma unroll
            for (int k = 0; k < 4; ++k) tmem_wait_load(x + 32 * k);
            if (negative) {
#pragma unroll
                for (int k = 0; k < 128; ++k) x[k] ^= 0x80000000u;
            }
            const int there = sees - j * kPromptKeys;  // of the step's keys
            if (j >= diagonal) {
#pragma unroll
                for (int k = 0; k < 128; ++k)
                    if (k >= there) x[k] = 0xFF800000u;
            }
            float part[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                part[k] = fmaxf(__uint_as_float(x[k]), __uint_as_float(x[k + 4]));
#pragma unroll
                for (int e = 8 + k; e < 128; e += 4) part[k] = fmaxf(part[k], __uint_as_float(x[e]));
            }
            const float top = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3])) * c;
            // The maximum moves only when it grows by 2^kLazy: until then the weights
            // may pass 1, and sum and output stay as they are.  (The scores' barrier says that
            // the last step's output is done too.)
            const bool grow = top > mx + kLazy || (mx == -INFINITY && top > mx);
            if (__any_sync(kFullMask, grow)) {
                const float f = grow ? exp2_approx(mx - top) : 1.0f;
                if (grow) mx = top;
                l *= f;
                if (j > 0)
#pragma unroll 1
                    for (int d = 0; d < kPromptDim; d += 16) {
                        uint32_t o[16];
                        tmem_load16(outputs + d, o);
                        tmem_wait_load16(o);
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                        tmem_store16(outputs + d, o);
                    }
            }
            const float shift = mx == -INFINITY ? 0.0f : mx;
            float2 sum[2] = {};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int at = 32 * k + 2 * e;
                    const float2 y = fma2(make_float2(__uint_as_float(x[at]), __uint_as_float(x[at + 1])),
                                          make_float2(c, c), make_float2(-shift, -shift));
                    const float2 u = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                    sum[e & 1] = add2(sum[e & 1], u);
                    // (bfloat16, 8 digits, as the values are: a product takes operands of one
                    // type.  The sum keeps all digits, for lse)
                    const __nv_bfloat162 two = __floats2bfloat162_rn(u.x, u.y);
                    x[16 * k + e] = *reinterpret_cast<const uint32_t *>(&two);
                }
                tmem_store16(scores + 16 * k, x + 16 * k);  // over scores that have been read
            }
            l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            if (j >= diagonal && (t == 0 || steps[0] <= j)) {
                // NaN and infinities of values that some query does not see become zeros (0 x
                // NaN would reach it); the rows that do see them get them at the end.  Each
                // CTA does so for the elements that it holds.
                wait(&ctl.value_seen, j);
                unsigned char *values = smem + S::kValueAt + j % kPromptStages * S::kValueBytes;
                if (ok)
                    for (int i = tid % 128; i < kPromptKeys * 8; i += 128) {
                        uint4 *at = reinterpret_cast<uint4 *>(values + i / 8 * 128 + ((i % 8 ^ (i / 8 & 7)) << 4));
                        uint4 v = *at;
                        unsigned *e = reinterpret_cast<unsigned *>(&v);
                        bool bad = false;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const bool lo16 = (e[k] & 0x7F80u) == 0x7F80u;
                            const bool hi16 = (e[k] & 0x7F800000u) == 0x7F800000u;
                            bad = bad || lo16 || hi16;
                            if (lo16) e[k] &= 0xFFFF0000u;
                            if (hi16) e[k] &= 0x0000FFFFu;
                        }
                        if (!bad) continue;
                        *at = v;
                        const int key = i / 8;
                        if (j * kPromptKeys + key < m)
                            for (int k = 0; k < 2; ++k)
                                cluster_or(cluster_addr(smem_addr(&ctl.nonfinite[j - diagonal][key / 32]), k),
                                           1u << key % 32);
                    }
                cluster_fence();
                fence_async_proxy();
            }
            tmem_wait_store();
            tmem_fence_before();
            __syncwarp();
            if (!ok) break;
            if (lane == 0) cluster_arrive(first_cta(&ctl.p_ready[t]));
        }
        if (count) wait(&ctl.o_done[t], 0);
        tmem_fence_after();
        const bool valid = row < n && ok;
        if (__any_sync(kFullMask, valid)) {
            const float shift = mx == -INFINITY ? 0.0f : mx, inv = l == 0.0f ? 0.0f : 1.0f / l;
            __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + (long long)(w.lo + row) * a.ld_out +
                                 (long long)head * kPromptDim;
            if (count) cluster_fence();  // (the noted keys)
#pragma unroll 1
            for (int d = 0; d < kPromptDim; d += 32) {
                uint32_t o[32] = {};
                if (count) {
                    tmem_load32(outputs + d, o);
                    tmem_wait_load(o);
                }
                for (int j = diagonal; valid && j < most; ++j)
                    for (int i = 0; i < kPromptKeys / 32; ++i) {
                        const int left = sees - j * kPromptKeys - 32 * i;
                        unsigned bits = *(volatile unsigned *)&ctl.nonfinite[j - diagonal][i];
                        bits = left >= 32 ? bits : left > 0 ? bits & ((1u << left) - 1) : 0;
                        for (; bits; bits &= bits - 1) {
                            const long long key = w.k0 + j * kPromptKeys + 32 * i + __ffs(bits) - 1;
                            const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v) + key * a.ld_v +
                                                     head / a.group * a.hs_v + d;
                            const bool gone = weightless(a, w.lo + row, head, key);  // (0 times infinity is NaN)
#pragma unroll
                            for (int k = 0; k < 32; ++k) {
                                const float y = elem_value(v[k]);
                                if (y - y == 0.0f) continue;
                                o[k] = __float_as_uint(gone ? NAN : __uint_as_float(o[k]) + y);
                            }
                        }
                    }
                if (!valid) continue;
                uint32_t p[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    float u = __uint_as_float(o[2 * k]) * inv, v = __uint_as_float(o[2 * k + 1]) * inv;
                    if (l == 0.0f) u = v = 0.0f;
                    const __nv_bfloat162 two = __floats2bfloat162_rn(u, v);
                    p[k] = *reinterpret_cast<const uint32_t *>(&two);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    reinterpret_cast<uint4 *>(out + d)[k] =
                        make_uint4(p[4 * k], p[4 * k + 1], p[4 * k + 2], p[4 * k + 3]);
            }
            if (valid && a.lse)
                a.lse[(long long)(w.lo + row) * a.n_q_heads + head] =
                    l == 0.0f ? -INFINITY : shift * kLn2 + logf(l);
        }
        tmem_fence_before();
    }
    __syncthreads();
    cluster_sync();  // the other CTA may arrive on, or multiply from, what is here
    if (warp == kPromptMatrixWarp) tmem_free_pair(tmem, 512);
}

namespace {

// Whether a call runs on the tensor cores: the dimensions that the kernel is laid out for,
// and the strides and bases that TMA and the 16-byte accesses take.
bool prompt_tensor_fits(const PromptArgs &a, int dtype) {
    if (dtype != DSPARK_DTYPE_BF16 || a.key_dim != kPromptDim || a.value_dim != kPromptDim || a.max_keys < 1)
        return false;
    if (a.shared_dim != 0 && a.shared_dim != kPromptShared) return false;
    for (long long s : {a.ld_q, a.ld_k, a.hs_k, a.ld_v, a.hs_v, a.ld_out, a.ld_shared})
        if (s % 8 || s * 2 >= (1ll << 40)) return false;
    return aligned(a.q, 16) && aligned(a.k, 16) && aligned(a.v, 16) && aligned(a.out, 16) && aligned(a.shared, 16);
}

// How many requests can have more than few_scores.
long long many_requests(const PromptArgs &a) { return ((long long)a.max_rows + a.max_keys) / kManyTokens; }

template <typename T>
cudaError_t launch_prompt_any(const PromptArgs &a, cudaStream_t stream) {
    const dim3 grid(a.max_rows, a.n_q_heads), block(kPromptWarps * 32);
    return launch_pdl(prompt_any_kernel<T>, grid, block, 0, stream, a);
}

template <bool kShared>
cudaError_t launch_prompt_tensor(const PromptArgs &a, cudaStream_t stream) {
    using S = PromptShape<kShared>;
    const int width = a.key_dim + a.shared_dim, n_kv_heads = a.n_q_heads / a.group;
    // [head][row][element]
    auto map = [&](CUtensorMap *to, const void *p, int dim, int rows, int heads, long long ld, long long hs, int box) {
        const int64_t dims[4] = {dim, rows, heads, 1}, strides[3] = {ld, hs, ld};
        return encode(to, p, 2, 64, true, dims, strides, box, 1);
    };
    CUtensorMap map_q, map_k, map_s = {}, map_v;
    if (!map(&map_q, a.q, width, a.max_rows, a.n_q_heads, a.ld_q, width, 128) ||
        !map(&map_k, a.k, a.key_dim, a.max_keys, n_kv_heads, a.ld_k, a.hs_k, 64) ||
        !map(&map_v, a.v, a.value_dim, a.max_keys, n_kv_heads, a.ld_v, a.hs_v, kPromptKeys) ||
        (kShared && !map(&map_s, a.shared, a.shared_dim, a.max_keys, 1, a.ld_shared, a.ld_shared, 64)))
        return cudaErrorUnknown;
    cudaError_t e = ensure_smem(reinterpret_cast<const void *>(prompt_tensor_kernel<kShared>), S::kTotal,
                                27 + kShared);
    if (e != cudaSuccess) return e;
    // every request has one block that is not full at most
    const long long jobs = min(a.split ? many_requests(a) : (long long)a.B, (long long)a.max_rows);
    const long long grid = 2ll * a.n_q_heads * (a.max_rows / kPromptBlock + jobs);
    if (grid == 0) return cudaSuccess;
    if (grid > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
    return launch_pdl(prompt_tensor_kernel<kShared>, dim3((unsigned)grid), dim3(kPromptThreads), S::kTotal, stream,
                      map_q, map_k, map_s, map_v, a);
}

}  // namespace

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
    // (other CTAs read the inputs after one has written its outputs)
    const int64_t e_bytes = kv_elem_bytes(dtype);
    auto under_out = [&](const void *p, int64_t ld, int64_t n, int64_t rows) {
        return rows_overlap(p, ld * e_bytes, n * e_bytes, rows, out, ld_out * e_bytes, width_out * e_bytes, max_rows);
    };
    bool over = under_out(q, ld_q, width, max_rows) || (k_shared && under_out(k_shared, ld_shared, shared_dim, max_keys));
    for (int g = 0; g < n_kv_heads; ++g)
        over = over || under_out(static_cast<const char *>(k) + g * hs_k * e_bytes, ld_k, key_dim, max_keys) ||
               under_out(static_cast<const char *>(v) + g * hs_v * e_bytes, ld_v, value_dim, max_keys);
    if (over) return DSPARK_ERR_INVALID_ARG;
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
    cudaError_t e;
    a.split = 0;
    if (prompt_tensor_fits(a, dtype)) {
        // A job takes a pair of CTAs some 11 us, however few its queries.  Where requests are
        // short on average, those of few scores go to the other kernel, which needs a second
        // launch and a CTA a row and head.  Jobs alone and split, us, 16 heads: 256 prompts of 1
        // token 601 and 20, of up to 8 603 and 74, of up to 32 630 and 402; 32 of up to 32 81 and
        // 57.  Of up to 64 (643, or 1216 without tensor cores) they stay.
        a.split = many_requests(a) < B;
        e = shared_dim ? launch_prompt_tensor<true>(a, st) : launch_prompt_tensor<false>(a, st);
        if (e == cudaSuccess && a.split) e = launch_prompt_any<__nv_bfloat16>(a, st);
    } else {
        e = dtype == DSPARK_DTYPE_BF16 ? launch_prompt_any<__nv_bfloat16>(a, st) : launch_prompt_any<float>(a, st);
    }
    return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
