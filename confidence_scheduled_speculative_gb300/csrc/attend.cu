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
//
// attend_tensor_kernel   bfloat16 rows over a bfloat16 or E4M3 cache on the tensor
//   cores.  A job is a (request, kv head) and up to 128 of its rows (window tokens with
//   their heads, so that keys and values are read once for all of them), a step 64
//   positions:  S = Q K^T into tensor memory, then
//     y = S c   m' = max(m, max y)   w = 2^(y - m')   l = l 2^(m - m') + sum w
//     O = O 2^(m - m') + W V
//   with W written over S in tensor memory and O kept there.  m moves only when a row's
//   maximum grows by 2^kLazy (until then w may pass 1, and O is not touched).
//   Over E4M3, K is an operand as it is, with the queries split into two E4M3 parts
//   (split_pair); V's codes become halves on the way.  Scales go with the scores: k's as
//   a factor, v's as an addend log2 v to y, divided out of l again by 1 / v.
//   One warp each copies (TMA), issues the first product and issues the second, four do
//   the softmax; over E4M3 another prepares scales and four convert.  Two CTAs an SM, so
//   that one's softmax runs beside the other's products; the tiles of all jobs are dealt
//   evenly to them (schedule.cuh), so jobs are split along the positions where there are
//   few, and attend_join_kernel adds the parts in a fixed order.
//   Over bfloat16 the bound is HBM: 32 requests of up to 8192 tokens with windows of up
//   to nine and 32 query heads, 557 MB, in 98 to 102 us by box (5.5 TB/s, 0.81 of a copy);
//   256 requests with up to 17 and 64 heads, 4.4 GB, in 763 to 787 us (5.6 to 5.8 TB/s, 0.83).
//   Over E4M3 half the bytes take the same steps, and the bound is a step's softmax and
//   conversions with the waits between them: two requests of up to 131040 tokens, 80 and
//   160 rows a kv head, the latter in two passes, 522 MB in 289 us (1.81 TB/s, 0.27; issue
//   slots half used).
//   There few rows go to attend_few_kernel (fewrows.cuh).

#include "fewrows.cuh"
#include "kvcache.cuh"
#include "schedule.cuh"
#include "tensor.cuh"

#include <atomic>
#include <type_traits>

namespace dspark {

constexpr int kAnyWarps = 4;
constexpr int kAnySteps = DSPARK_MAX_HEAD_DIM / 32;

template <typename T, typename C>
__global__ void __launch_bounds__(kAnyWarps * 32) attend_any_kernel(AttendArgs a) {
    __shared__ float part_o[kAnyWarps][DSPARK_MAX_HEAD_DIM];
    __shared__ float part_m[kAnyWarps], part_l[kAnyWarps];
    pdl_trigger();
    pdl_wait();
    const int row = blockIdx.x, h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int D = a.cache.head_dim;
    // (the requests' windows are looked at by one CTA: a window outside the rows has none)
    if (row == 0 && h == 0)
        for (int r = threadIdx.x; r < a.B; r += kAnyWarps * 32) usable(a, load_window(a, r), true);
    if (row >= __ldg(a.cu + a.B)) return;
    int lo = 0, hi = a.B - 1;  // the last request that starts at or before the row
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldg(a.cu + mid) <= row) lo = mid;
        else hi = mid - 1;
    }
    const int r = lo;
    const Window win = load_window(a, r);
    if (!usable(a, win, false) || row < win.lo) return;
    const int row0 = win.lo, len = win.hi - win.lo, P = win.P;
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

// ------------------------------------------------- tensor-core kernel

// Shared memory and warps of a CTA.
//   16-bit cache: one ring of buffers, into which keys and values are copied and
//     from which they are multiplied.
//   E4M3 cache: the keys' codes are operands as they are (their ring: kBufs), the
//     values' codes are staged (kStages) and converted by four warps into two
//     buffers of halves.
template <int D, bool kQuant>
struct TensorShape {
    static constexpr int kQBytes = kRowsPerTile * D * 2;
    static constexpr int kBufBytes = kTile * D * (kQuant ? 1 : 2);
    static constexpr int kBufs = kQuant ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 9);
    static constexpr int kStages = kQuant ? (D == 128 ? 2 : 6) : 0;
    static constexpr int kStageAt = kQBytes + kBufs * kBufBytes;
    static constexpr int kOpBytes = kTile * D * 2;
    static constexpr int kOpAt = kStageAt + kStages * kBufBytes;
    static constexpr int kControl = kOpAt + (kQuant ? 2 * kOpBytes : 0);
    static constexpr int kTotal = kControl + (kQuant ? 5120 : 1024);
    static constexpr int kCopyWarp = kQuant ? 8 : 4;
    static constexpr int kScoreWarp = kCopyWarp + 1, kValueWarp = kCopyWarp + 2, kScaleWarp = 11;
    static constexpr int kThreads = kQuant ? 384 : 224;
    // of a job's begin and end, in tiles (1, 2 and 4: windows 104, 104 and 106 us, long
    // trees over E4M3 302, 295 and 305)
    static constexpr int kJobCost = 2;
    static_assert(kTotal <= 113 * 1024, "two CTAs an SM");
};

// The barriers and words behind the buffers.  A wait tells a phase from the next
// one only; the barriers that come in twos serve every other tile, so that a
// role one tile behind another still waits for the phase it means.
struct alignas(16) Control {
    unsigned long long full[9], empty[9], stage_full[6], stage_empty[6], op_full[2], op_empty[2];
    unsigned long long s_full[2], p_ready[2], o_done[2], scales[2];
    unsigned long long q_raw[2], q_full[2], q_empty[2], drain[2];
    unsigned tmem;
    unsigned nonfinite[4];  // window tokens whose values were zeroed, by segment
    int abort;
    Begin begin;
    long long scan[40];
};
// What the scales of a tile's tokens become (E4M3), for every other tile.
struct TileScales {
    float k[2][kTile];       // k_scale times the scores' factor, to base 2
    float v_log2[2][kTile];  // log2 v_scale: part of a weight's exponent
    float v_inv[2][kTile];   // 1 / v_scale: takes it out of the sum of weights
    float v[2][kTile];       // v_scale itself
    int odd[2];              // whether a v_scale is negative, NaN or infinite
    int pad[2];
    float q[4][kRowsPerTile];  // what the queries were divided by, by segment
};
static_assert(sizeof(Control) <= 1024 && sizeof(Control) + sizeof(TileScales) <= 5120, "control area");

// A place in a ring of `slots` barriers and buffers, and the parity of its phase.
struct Ring {
    unsigned slot, parity;
    __device__ __forceinline__ void step(unsigned slots) {
        if (++slot == slots) {
            slot = 0;
            parity ^= 1;
        }
    }
};

// Where a position lies, for a lane that steps through the tiles of a segment:
// the table's entry is loaded ahead of its use.
struct Place {
    int col, token;
    __device__ __forceinline__ void begin(const KvView &c, int pos) {
        col = (unsigned)pos / (unsigned)c.page_size;
        token = pos - col * c.page_size;
    }
    __device__ __forceinline__ void step(const KvView &c) {
        token += kTile;
        while (token >= c.page_size) {
            token -= c.page_size;
            ++col;
        }
    }
    // the entry; the pool's size, a page it does not have, past the end
    __device__ __forceinline__ int entry(const KvView &c, int r, bool in) const {
        return in ? __ldg(c.table + (long long)r * c.table_width + col) : c.n_pages;
    }
};

// Two E4M3 values' worth of a query: x = hi + lo.  A bfloat16 has 8 significant
// digits; hi takes the upper four, and what remains of x has at most four more, so
// that hi + lo = x exactly while lo's last digit is at least E4M3's smallest step, 2^-9:
// from 2^-2 on.  Below it half a step is lost, 2^-10, which is at most 2^-17 of a row's
// largest element (brought to 128..256).
__device__ __forceinline__ void split_pair(float x0, float x1, unsigned *hi, unsigned *lo) {
    *hi = e4m3_pair(x0, x1);
    const float2 h = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)*hi, __NV_E4M3)));
    *lo = e4m3_pair(x0 - h.x, x1 - h.y);
}

// Where 16-byte chunk c of row r lies in rows of `row_bytes` (64 or 128) under the
// swizzle of that width.
template <int kRowBytes>
__device__ __forceinline__ int swizzled(int r, int c) {
    return kRowBytes == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ (r >> 1 & 3)) << 4);
}

template <int D, bool kQuant>
__global__ void __launch_bounds__(TensorShape<D, kQuant>::kThreads, 2)
attend_tensor_kernel(const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v,
                     const __grid_constant__ CUtensorMap map_q,
                     const __grid_constant__ CUtensorMap map_few, const TensorArgs t) {
    using S = TensorShape<D, kQuant>;
    constexpr int kThreads = S::kThreads;
    constexpr int kHalves = D / 64;       // 128-byte column blocks of a row
    constexpr int kChunks = D / 8;        // 16-byte chunks of a row
    constexpr int kHalfBytes = kTile * 128;
    extern __shared__ __align__(1024) unsigned char smem[];
    Control &ctl = *reinterpret_cast<Control *>(smem + S::kControl);
    TileScales &sc = *reinterpret_cast<TileScales *>(smem + S::kControl + sizeof(Control));
    const AttendArgs &a = t.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = smem_addr(smem);
    const uint32_t ring = base + S::kQBytes;

    // Behind fewrows.cuh's kernel, which may do the call.  That one lets this one start
    // only after its own wait, so the lengths are there to read; and if it does the call,
    // one CTA waits for it, as the join waits for these only, and the others make room.
    if (kQuant && t.choose) {
        pdl_trigger();
        Request q;
        long long dearer = 0;
        for (int r = tid; r < a.B; r += kThreads)
            if (to_request(t, load_window(a, r), &q, false)) dearer += few_dearer(t, q);
        if (block_sum<long long>(dearer, ctl.scan) <= 0) {
            if (blockIdx.x == 0) pdl_wait();
            return;
        }
    }
    if (tid == 0) {
        for (int i = 0; i < S::kBufs; ++i) {
            mbar_init(smem_addr(&ctl.full[i]), 1);
            mbar_init(smem_addr(&ctl.empty[i]), 1);
        }
        for (int i = 0; i < S::kStages; ++i) {
            mbar_init(smem_addr(&ctl.stage_full[i]), 1);
            mbar_init(smem_addr(&ctl.stage_empty[i]), 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&ctl.s_full[i]), kQuant ? 2 : 1);  // the product; the scales
            mbar_init(smem_addr(&ctl.p_ready[i]), 4);
            mbar_init(smem_addr(&ctl.o_done[i]), 1);
            mbar_init(smem_addr(&ctl.scales[i]), 1);
            mbar_init(smem_addr(&ctl.op_full[i]), 4);
            mbar_init(smem_addr(&ctl.op_empty[i]), 1);
            mbar_init(smem_addr(&ctl.q_raw[i]), 1);
            mbar_init(smem_addr(&ctl.q_full[i]), 4);
            mbar_init(smem_addr(&ctl.q_empty[i]), 1);
            mbar_init(smem_addr(&ctl.drain[i]), 1);
        }
        ctl.abort = 0;
        for (int i = 0; i < 4; ++i) ctl.nonfinite[i] = 0;
        fence_mbar_init();
        prefetch_map(&map_k);
        prefetch_map(&map_v);
        prefetch_map(&map_q);
        prefetch_map(&map_few);
    }
    if (warp == S::kScoreWarp) tmem_alloc(smem_addr(&ctl.tmem), kTmemCols);
    pdl_wait();
    pdl_trigger();

    Deal deal;
    long long lo, hi;
    const int cta = blockIdx.x;
    if (!share_of<kThreads, S::kJobCost, false>(t, &ctl.begin, ctl.scan, &deal, &lo, &hi)) {
        if (warp == S::kScoreWarp) {
            __syncwarp();
            tmem_free(*(volatile unsigned *)&ctl.tmem, kTmemCols);
        }
        return;
    }
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = ctl.tmem;
    volatile int *abort = &ctl.abort;
    Walk<S::kJobCost> walk;
    walk.begin(t, ctl.begin, (int)(hi - lo));
    Segment s = {};
    Ring ring_at = {0, 0};
    // The queries of a segment whose rows fit in 64 take one half of their buffer
    // and the next such segment's the other, so that they are there in time.
    auto few_rows = [&](const Segment &s) { return s.q.len - s.row_tile * t.tokens <= t.few; };
    auto q_offset = [&](const Segment &s, unsigned seg) { return few_rows(s) ? (seg & 1) * 8192u : 0u; };

    // Over E4M3 the softmax warps take registers from the others: of 80 a thread at
    // launch in each of three warpgroups, 112, 72 and 56.
    if (warp >= S::kCopyWarp) {
        if constexpr (kQuant) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == S::kCopyWarp) {
            // -------------------------------------------- copy warp
            constexpr int kParts = kQuant ? 1 : kHalves;  // boxes side by side
            const int boxes = kTile / t.box, box = lane / kParts, half = lane % kParts;
            const bool issues = box < boxes;
            const uint32_t dst = ring + half * kHalfBytes + box * t.box * (kQuant ? D : 128);
            Ring stage_at = {0, 0};  // the values' ring, over E4M3
            unsigned seg = 0;
            bool ok = true, few_before = false;
            auto wait = [&](unsigned long long *bar, unsigned parity) {
                return ok = warp_wait(ok, smem_addr(bar), parity, abort, a.status);
            };
            while (ok && walk.next(t, &s)) {
                // this lane's box of each tile; a page outside the pool, as past
                // the request's end, arrives as zeros
                const int n = s.q.P + s.q.len;
                int pos = s.first * kTile + box * t.box;
                Place at;
                at.begin(a.cache, issues ? pos : 0);
                auto entry = [&](bool in) { return at.entry(a.cache, s.r, issues && in && pos < n); };
                int page = 0, token = 0, page1 = entry(true), token1;  // of the values and the keys
                // In the order of use: K0, K1, V0, K2, V1, ..., V(n-1)
                for (int i = 0; i <= s.count; ++i) {
                    token1 = at.token;
                    if (i < s.count) {
                        if (issues && pos < n && (unsigned)page1 >= (unsigned)a.cache.n_pages) {
                            flag(a.status, DSPARK_STATUS_BAD_INDEX);
                            page1 = a.cache.n_pages;
                        }
                    }
                    pos += kTile;
                    at.step(a.cache);
                    const int page2 = entry(i + 1 < s.count);
#pragma unroll 1
                    for (int which = 0; which < 2; ++which) {  // keys of tile i, values of tile i - 1
                        if (which == 0 ? i == s.count : i == 0) continue;
                        const bool staged = kQuant && which == 1;
                        Ring &r = staged ? stage_at : ring_at;
                        if (!wait((staged ? ctl.stage_empty : ctl.empty) + r.slot, r.parity ^ 1)) break;
                        const uint32_t bar = smem_addr((staged ? ctl.stage_full : ctl.full) + r.slot);
                        if (lane == 0) mbar_expect(bar, S::kBufBytes);
                        __syncwarp();
                        if (issues)
                            tma_load_4d(dst + (staged ? S::kStageAt - S::kQBytes : 0) + r.slot * S::kBufBytes,
                                        which == 0 ? &map_k : &map_v, half * 64, which == 0 ? token1 : token,
                                        s.head, which == 0 ? page1 : page, bar);
                        if (staged) stage_at.step(S::kStages > 0 ? S::kStages : 1);
                        else ring_at.step(S::kBufs);
                    }
                    if (!ok) break;
                    if (i == 0) {
                        // the queries, once the products with the ones there before
                        // are done: the last segment's, or the ones before those
                        const bool few = few_rows(s);
                        if (seg > 1 && !wait(&ctl.q_empty[seg & 1], (seg - 2) >> 1)) break;
                        if (seg > 0 && !(few && few_before) && !wait(&ctl.q_empty[(seg - 1) & 1], (seg - 1) >> 1))
                            break;
                        const uint32_t bar = smem_addr(&ctl.q_raw[seg & 1]);
                        if (lane == 0) mbar_expect(bar, t.group * (few ? t.few : t.tokens) * D * 2);
                        __syncwarp();
                        if (lane < kHalves)
                            tma_load_4d(base + lane * kRowsPerTile * 128 + q_offset(s, seg), few ? &map_few : &map_q,
                                        lane * 64, 0, s.head, s.q.row0 + s.row_tile * t.tokens, bar);
                        few_before = few;
                        ++seg;
                    }
                    page = page1;
                    token = token1;
                    page1 = page2;
                }
            }
            if (!ok && lane == 0) {
                // copies still under way write this block's buffers: the last load
                // of each slot, complete or never begun
                for (int i = 0; i < S::kBufs; ++i)
                    mbar_wait(smem_addr(&ctl.full[i]), i < (int)ring_at.slot ? ring_at.parity : ring_at.parity ^ 1);
                for (int i = 0; i < S::kStages; ++i)
                    mbar_wait(smem_addr(&ctl.stage_full[i]),
                              i < (int)stage_at.slot ? stage_at.parity : stage_at.parity ^ 1);
                for (unsigned i = seg > 2 ? seg - 2 : 0; i < seg; ++i)
                    mbar_wait(smem_addr(&ctl.q_raw[i & 1]), i >> 1 & 1);
            }
        } else if (warp == S::kScoreWarp || warp == S::kValueWarp) {
            // ---------------------------------------- matrix warps
            // One issues the products of queries and keys, the other those of weights
            // and values: issuing a tile's products, with the waits before and the
            // commits behind them, takes one warp longer than the products take.  Each
            // warp keeps step as a whole, so that addresses stay in uniform registers;
            // one lane issues.
            const bool scores = warp == S::kScoreWarp;
            const uint32_t ubase = __shfl_sync(kFullMask, base, 0);
            const uint32_t utmem = __shfl_sync(kFullMask, tmem, 0);
            const bool leader = elect_one();
            unsigned done = 0, seg = 0;  // tiles and segments so far
            bool ok = true;
            auto wait = [&](unsigned long long *bar, unsigned parity) {
                return ok = warp_wait(ok, smem_addr(bar), parity, abort, a.status);
            };
            // over E4M3 keys have a ring of their own; else the loads lie in one, K0, K1,
            // V0, K2, V1, ..., V(n-1)
            auto skip = [&](int n) {
                for (; n > 0; --n) ring_at.step(S::kBufs);
            };
            if (scores) {
                // over E4M3: codes times the queries' two parts
                constexpr uint32_t all_rows = kQuant ? mma_word_e4m3(kTile) : mma_word(true, kTile, false);
                constexpr int kKeyRow = kQuant ? D : 128;  // bytes of a row
                const uint64_t desc_q = smem_operand(ubase, 16, kKeyRow);
                const uint64_t desc_k = smem_operand(ubase + S::kQBytes, 16, kKeyRow);
                unsigned long long *queries = kQuant ? ctl.q_full : ctl.q_raw;
                while (ok && walk.next(t, &s)) {
                    if (!wait(queries + (seg & 1), seg >> 1)) break;
                    const bool few = few_rows(s);
                    const uint32_t word = all_rows - (few ? kHalfRows : 0);
                    const uint64_t queries_at = desc_q + (q_offset(s, seg) >> 4);
                    // their second parts, over E4M3
                    const unsigned part = (D == 64 && few ? 4096 : S::kQBytes / 2) >> 4;
                    const int count = __shfl_sync(kFullMask, s.count, 0);
                    for (int i = 0; i < count; ++i) {
                        // in the place of the weights of tile - 2
                        const unsigned tile = done + i;
                        if (tile > 1 && !wait(&ctl.o_done[tile & 1], (tile - 2) >> 1)) break;
                        if (!wait(&ctl.full[ring_at.slot], ring_at.parity)) break;
                        tmem_fence_after();
                        const uint64_t buf = desc_k + ring_at.slot * (S::kBufBytes >> 4);
                        const uint32_t d = utmem + (tile & 1) * kTile;
                        if (leader) {
                            if constexpr (kQuant) {
#pragma unroll
                                for (int k = 0; k < D / 16; ++k)  // 32 codes a step, for either part
                                    mma_ss_e4m3(d, queries_at + k % 2 * part + (k / 2 * 32 >> 4),
                                                buf + (k / 2 * 32 >> 4), word, k > 0);
                            } else {
#pragma unroll
                                for (int k = 0; k < D / 16; ++k)
                                    mma_ss(d, queries_at + ((k / 4 * kRowsPerTile * 128 + k % 4 * 32) >> 4),
                                           buf + ((k / 4 * kHalfBytes + k % 4 * 32) >> 4), word, k > 0);
                            }
                            mma_commit(smem_addr(&ctl.s_full[tile & 1]));
                            mma_commit(smem_addr(&ctl.empty[ring_at.slot]));
                            if (i + 1 == count) mma_commit(smem_addr(&ctl.q_empty[seg & 1]));
                        }
                        __syncwarp();
                        skip(kQuant ? 1 : (i == 0 ? 1 : 2) + (i + 1 == count));
                    }
                    done += count;
                    ++seg;
                }
            } else {
                constexpr uint32_t all_rows = mma_word(!kQuant, D, true);
                const uint64_t desc_v = smem_operand(ubase + (kQuant ? S::kOpAt : S::kQBytes), kHalfBytes, 128);
                while (ok && walk.next(t, &s)) {
                    const uint32_t word = all_rows - (few_rows(s) ? kHalfRows : 0);
                    const int count = __shfl_sync(kFullMask, s.count, 0);
                    if (!kQuant) skip(count > 1 ? 2 : 1);
                    for (int i = 0; i < count; ++i) {
                        const unsigned tile = done + i;
                        const unsigned slot = kQuant ? tile & 1 : ring_at.slot;
                        if (!wait(kQuant ? &ctl.op_full[slot] : &ctl.full[slot],
                                  kQuant ? tile >> 1 : ring_at.parity))
                            break;
                        if (!wait(&ctl.p_ready[tile & 1], tile >> 1)) break;
                        tmem_fence_after();
                        const uint64_t buf = desc_v + slot * (S::kOpBytes >> 4);
                        const uint32_t w = utmem + (tile & 1) * kTile;
                        if (leader) {
#pragma unroll
                            for (int k = 0; k < kTile / 16; ++k)
                                mma_ts(utmem + 2 * kTile, w + k * 8, buf + (k * 16 * 128 >> 4), word,
                                       i > 0 || k > 0);
                            mma_commit(smem_addr(&ctl.o_done[tile & 1]));
                            mma_commit(smem_addr(kQuant ? &ctl.op_empty[slot] : &ctl.empty[slot]));
                        }
                        __syncwarp();
                        if (!kQuant) skip(i + 2 < count ? 2 : 1);
                    }
                    done += count;
                }
            }
            // after a timeout: products still under way write tensor memory and
            // barriers of this block
            if (!ok && leader) {
                mma_commit(smem_addr(&ctl.drain[scores]));
                mbar_wait(smem_addr(&ctl.drain[scores]), 0);
            }
            __syncwarp();
        } else if (kQuant && warp == S::kScaleWarp) {
            // ------------------------------------------- scale warp
            if constexpr (kQuant) {
                const float c = copysignf(fmaxf(fabsf(a.scale) * kLog2e, 0x1p-100f), a.scale);
                unsigned done = 0;
                bool ok = true;
                while (ok && walk.next(t, &s)) {
                    // a lane's two tokens, 32 apart: the table's entries two tiles
                    // ahead, the scales one
                    const int n = s.q.P + s.q.len;
                    int pos = s.first * kTile + lane;
                    Place at[2];
                    at[0].begin(a.cache, pos);
                    at[1].begin(a.cache, pos + 32);
                    float ks[2], vs[2];
                    int page[2];
                    auto entries = [&](bool in) {
                        page[0] = at[0].entry(a.cache, s.r, in && pos < n);
                        page[1] = at[1].entry(a.cache, s.r, in && pos + 32 < n);
                    };
                    auto fetch = [&]() {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const bool in = (unsigned)page[i] < (unsigned)a.cache.n_pages;
                            const long long from =
                                in ? kv_scale_offset(a.cache, page[i], at[i].token, s.head) : 0;
                            ks[i] = in ? __ldg(a.cache.k_scale + from) : 1.0f;
                            vs[i] = in ? __ldg(a.cache.v_scale + from) : 1.0f;
                        }
                        pos += kTile;
                        at[0].step(a.cache);
                        at[1].step(a.cache);
                    };
                    entries(true);
                    fetch();
                    entries(s.count > 1);
                    for (int i = 0; i < s.count; ++i) {
                        const unsigned tile = done + i, b = tile & 1;
                        float k[2], log2v[2], inv[2], raw[2];
                        bool odd = false;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const bool fine = vs[j] - vs[j] == 0.0f;
                            // a NaN or infinite k_scale makes the score NaN
                            k[j] = ks[j] - ks[j] == 0.0f ? ks[j] * c : __int_as_float(0x7FC00000);
                            const float f = fine ? fmaxf(fabsf(vs[j]), 0x1p-100f) : 1.0f;
                            log2v[j] = __log2f(f);
                            inv[j] = __frcp_rn(f);
                            raw[j] = vs[j];
                            odd = odd || !fine || vs[j] < 0.0f;
                        }
                        odd = __any_sync(kFullMask, odd);
                        if (i + 1 < s.count) {
                            fetch();
                            entries(i + 2 < s.count);
                        }
                        // the tile before last is through with its scales
                        if (tile >= 2)
                            ok = warp_wait(ok, smem_addr(&ctl.o_done[b]), (tile >> 1) + 1, abort, a.status);
                        if (!ok) break;
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            sc.k[b][lane + 32 * j] = k[j];
                            sc.v_log2[b][lane + 32 * j] = log2v[j];
                            sc.v_inv[b][lane + 32 * j] = inv[j];
                            sc.v[b][lane + 32 * j] = raw[j];
                        }
                        if (lane == 0) sc.odd[b] = odd;
                        __syncwarp();
                        if (lane == 0) {
                            mbar_arrive(smem_addr(&ctl.s_full[b]));
                            mbar_arrive(smem_addr(&ctl.scales[b]));
                        }
                    }
                    done += s.count;
                }
            }
        }
    } else if (kQuant && warp >= 4) {
        // --------------------------------------------- converting warps
        if constexpr (kQuant) {
            asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
            constexpr int kUnits = D / 16;  // 16 codes a thread and step
            constexpr int kSteps = kTile * kUnits / 128;
            const int ct = tid - 128;
            unsigned done = 0, seg = 0;
            bool ok = true;
            auto wait = [&](unsigned long long *bar, unsigned parity) {
                return ok = warp_wait(ok, smem_addr(bar), parity, abort, a.status);
            };
            // Their place is chunks 2 part and 2 part + 1 of the token's row.  Lanes of one
            // half start with the one, of the other with the other, so that eight lanes
            // cover the eight chunk columns of shared memory.  A thread's tokens are
            // 128 / kUnits apart, a multiple of eight: its places differ by whole rows.
            const int part = ct % kUnits, own = ct / kUnits;
            const unsigned flip = part / 4 & 1;
            const unsigned place = S::kOpAt + part / 4 * kHalfBytes + own * 128;
            const unsigned first = place + (((part % 4 * 2 + flip) ^ (own & 7)) << 4);
            const unsigned last = place + (((part % 4 * 2 + 1 - flip) ^ (own & 7)) << 4);
            for (;;) {
                // a warp that gave up still comes to the four warps' barriers
                ok = named_all(2, 128, ok);
                if (!ok || !walk.next(t, &s)) break;
                const int n = s.q.P + s.q.len;
                // The tile's queries, a row a thread, as two E4M3 values an element
                // (split_pair): each part a K-major operand of its own, in the place
                // of the bfloat16 rows.  A power of two brings a row's largest element
                // to 128..256; a row with a NaN or an infinity gets NaN scores.
                wait(&ctl.q_raw[seg & 1], seg >> 1);
                const bool few = few_rows(s), mine = ct < (few ? 64 : 128);
                unsigned char *rows = smem + q_offset(s, seg);
                unsigned char *second = rows + (D == 64 && few ? 4096 : S::kQBytes / 2);
                unsigned most = 0;
                if (mine) {
#pragma unroll 4
                    for (int j = 0; j < D / 8; ++j) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(
                            rows + j / 8 * kRowsPerTile * 128 + swizzled<128>(ct, j % 8));
                        const unsigned w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k) most = max(most, max(w[k] & 0x7FFFu, w[k] >> 16 & 0x7FFFu));
                    }
                }
                const int exponent = min(max((int)(most >> 7), 8), 254) - 134;
                const float by = __int_as_float((127 - exponent) << 23);
                sc.q[seg & 3][ct] =
                    most >= 0x7F80u ? __int_as_float(0x7FC00000) : __int_as_float((exponent + 127) << 23);
                uint4 kept[4];  // the low parts of the first 64 elements: their place is not free yet
#pragma unroll 1
                for (int h = 0; h < kHalves; ++h) {
                    uint4 v[8];
                    if (mine) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            v[j] = *reinterpret_cast<const uint4 *>(rows + h * kRowsPerTile * 128 +
                                                                    swizzled<128>(ct, j));
                    }
                    if (D == 64) named_sync(2, 128);  // shorter rows: in the place of other threads' ones
                    if (!mine) continue;
                    uint4 low[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const unsigned w[8] = {v[2 * j].x,     v[2 * j].y,     v[2 * j].z,     v[2 * j].w,
                                               v[2 * j + 1].x, v[2 * j + 1].y, v[2 * j + 1].z, v[2 * j + 1].w};
                        unsigned hi[4], lo[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            unsigned h0, h1, l0, l1;
                            split_pair(__uint_as_float(w[2 * k] << 16) * by,
                                       __uint_as_float(w[2 * k] & 0xFFFF0000u) * by, &h0, &l0);
                            split_pair(__uint_as_float(w[2 * k + 1] << 16) * by,
                                       __uint_as_float(w[2 * k + 1] & 0xFFFF0000u) * by, &h1, &l1);
                            hi[k] = h0 | h1 << 16;
                            lo[k] = l0 | l1 << 16;
                        }
                        *reinterpret_cast<uint4 *>(rows + swizzled<D>(ct, 4 * h + j)) =
                            make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        low[j] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                    if (h + 1 < kHalves) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) kept[j] = low[j];
                        continue;
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (kHalves == 2) *reinterpret_cast<uint4 *>(second + swizzled<D>(ct, j)) = kept[j];
                        *reinterpret_cast<uint4 *>(second + swizzled<D>(ct, 4 * h + j)) = low[j];
                    }
                }
                fence_async_proxy();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&ctl.q_full[seg & 1]));
                for (int i = 0; i < s.count; ++i) {
                    const unsigned tile = done + i, b = tile & 1, stage = ring_at.slot;
                    if (!wait(&ctl.scales[b], tile >> 1)) break;
                    if (!wait(&ctl.stage_full[stage], ring_at.parity)) break;
                    if (!wait(&ctl.op_empty[b], (tile >> 1) + 1)) break;
                    const unsigned char *src = smem + S::kStageAt + stage * S::kBufBytes;
                    unsigned char *dst = smem + S::kOpAt + b * S::kOpBytes;
                    const int p0 = (s.first + i) * kTile;
                    if (p0 + kTile <= s.q.P && !*(volatile int *)&sc.odd[b]) {
                        const unsigned char *from = src + ct * 16;
                        unsigned char *to = smem + b * S::kOpBytes;
#pragma unroll 1
                        for (int k = 0; k < kSteps; ++k) {
                            const uint2 v0 = *reinterpret_cast<const uint2 *>(from + flip * 8);
                            const uint2 v1 = *reinterpret_cast<const uint2 *>(from + 8 - flip * 8);
                            *reinterpret_cast<uint4 *>(to + first) =
                                eight_halves(v0);
                            *reinterpret_cast<uint4 *>(to + last) =
                                eight_halves(v1);
                            from += 2048;
                            to += 128 / kUnits * 128;
                        }
                    } else {
                        // Scales that are not plain numbers (or negative) go into the
                        // values; values past the request's end become zeros, and so
                        // do NaN and infinities of the window, which the rows that see
                        // them get at the end.
#pragma unroll 1
                        for (int k = ct; k < kTile * kUnits; k += 128) {
                            const int tok = k / kUnits, pos = p0 + tok;
                            const float f = sc.v[b][tok];
                            const float g = f - f == 0.0f ? copysignf(1.0f, f) : f;
                            bool bad = false;
#pragma unroll 1
                            for (int e = 0; e < 8; ++e) {
                                const unsigned w = reinterpret_cast<const unsigned short *>(src + k * 16)[e];
                                float x[2] = {e4m3_value(w & 0xFF) * g, e4m3_value(w >> 8) * g};
#pragma unroll
                                for (int y = 0; y < 2; ++y) {
                                    if (pos >= n) x[y] = 0.0f;
                                    if (pos >= s.q.P && !(x[y] - x[y] == 0.0f)) x[y] = 0.0f, bad = true;
                                }
                                const __half2 two = __floats2half2_rn(x[0], x[1]);
                                unsigned char *row = dst + k % kUnits / 4 * kHalfBytes + tok * 128;
                                const int ch = k % kUnits % 4 * 2 + e / 4;
                                *reinterpret_cast<__half2 *>(row + ((ch ^ (tok & 7)) << 4) + e % 4 * 4) = two;
                            }
                            if (bad) atomicOr(&ctl.nonfinite[seg & 3], 1u << (pos - s.q.P));
                        }
                    }
                    fence_async_proxy();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(smem_addr(&ctl.op_full[b]));
                        mbar_arrive(smem_addr(&ctl.stage_empty[stage]));
                    }
                    ring_at.step(S::kStages);
                }
                done += s.count;
                ++seg;
            }
        }
    } else {
        // --------------------------------------------- softmax warps
        if constexpr (kQuant) asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
        const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
        const float c = fmaxf(fabsf(a.scale) * kLog2e, 0x1p-100f);  // 0 would turn -inf into NaN
        const bool negative = a.scale < 0.0f;
        unsigned loads = 0;  // of the segments before
        unsigned done = 0, seg = 0;
        bool ok = true;
        auto wait = [&](unsigned long long *bar, unsigned parity) {
            return ok = warp_wait(ok, smem_addr(bar), parity, abort, a.status);
        };
        for (;;) {
            // a warp that gave up still comes to the four warps' barriers
            ok = named_all(1, 128, ok);
            if (!ok || !walk.next(t, &s)) break;
            // 64 rows or fewer are 16 a warp, so that each has half the work (18 rows a kv
            // head over E4M3, 32 requests: 139 -> 123 us)
            const bool few = few_rows(s), own = !few || lane < 16;
            const int first_row = warp * (few ? 16 : 32), m = first_row + lane;
            // row m: head m % group of the tile's token m / group
            const int n = s.q.P + s.q.len, token0 = s.row_tile * t.tokens;
            const int rows = min(t.tokens, s.q.len - token0) * t.group;
            const bool valid = own && m < rows, active = first_row < rows;
            const int mm = min(m, rows - 1), token = token0 + mm / t.group;
            const int head = s.head * t.group + mm % t.group, packed = s.q.row0 + token;
            const unsigned bits = ancestors_of(a, packed, token, s.q.len);
            if (tid == 0) ctl.nonfinite[(seg + 3) & 3] = 0;  // the segment's before

            // The scores are taken as fragments: of the warp's rows a thread has
            // four, 16 h + 8 k + lane / 4, and of each sixteen columns.  16 rows or
            // fewer are one half's work, and few scales serve a thread.
            const int halves = !few && rows - first_row > 16 ? 2 : 1;
            struct Row {
                float mx, l, factor;  // running maximum (to base 2), sum; query's power of two
                unsigned seen;        // ancestor bits
            } now[2], other[2];       // of the half at hand, and of the other
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                auto row_of = [&](int h) -> Row {
                    const int token_k = token0 + min(first_row + 16 * h + 8 * k + lane / 4, rows - 1) / t.group;
                    return {-INFINITY, 0.0f, 1.0f,
                            active ? ancestors_of(a, s.q.row0 + token_k, token_k, s.q.len) : 0u};
                };
                now[k] = row_of(0);
                other[k] = row_of(1);
            }
            for (int i = 0; i < s.count; ++i) {
                const unsigned tile = done + i, b = tile & 1;
                const int p0 = (s.first + i) * kTile;
                if (!wait(&ctl.s_full[b], tile >> 1)) break;
                if (active) {
                    tmem_fence_after();
                    const bool prefix_only = p0 + kTile <= s.q.P;
                    // (a loop, not two copies: the warps of a scheduler run several kinds
                    // of code in turn, and all of it is to stay in the instruction cache)
#pragma unroll 1
                    for (int h = 0; h < halves; ++h) {
                        const uint32_t at = lanes + ((uint32_t)(16 * h) << 16);
                        const int column = 2 * (lane & 3);
                        uint32_t x[32];
                        tmem_load_rows16(at + b * kTile, x);
                        // (all of the scales' loads before the first use: one after the
                        // other their latencies are most of a tile's time)
                        [[maybe_unused]] float2 f1[8], f2[8];
                        if constexpr (kQuant) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                f1[j] = *reinterpret_cast<const float2 *>(&sc.k[b][8 * j + column]);
                                f2[j] = *reinterpret_cast<const float2 *>(&sc.v_log2[b][8 * j + column]);
                            }
                            if (i == 0)
#pragma unroll
                                for (int k = 0; k < 2; ++k)
                                    now[k].factor = sc.q[seg & 3][first_row + 16 * h + 8 * k + lane / 4];
                        }
                        tmem_wait_load(x);
                        auto pair = [&](int e) {  // elements 2e and 2e + 1, of row e % 2
                            return make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
                        };
                        if constexpr (kQuant) {
                            // scores to base 2, plus log2 of the value's scale
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
#pragma unroll
                                for (int k = 0; k < 2; ++k) {
                                    const float f = now[k].factor;
                                    const float2 y = fma2(mul2(pair(2 * j + k), make_float2(f, f)), f1[j], f2[j]);
                                    x[4 * j + 2 * k] = __float_as_uint(y.x);
                                    x[4 * j + 2 * k + 1] = __float_as_uint(y.y);
                                }
                            }
                        } else if (negative) {
#pragma unroll
                            for (int j = 0; j < 32; ++j) x[j] ^= 0x80000000u;
                        }
                        if (!prefix_only) {
                            // prefix positions, then the row's ancestors in the window
                            const int pre = max(s.q.P - p0, 0), skip = max(p0 - s.q.P, 0);
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const unsigned long long w = skip < 32 ? (unsigned long long)(now[k].seen >> skip) : 0;
                                const unsigned long long sees = (w << pre | ((1ull << pre) - 1)) >> column;
#pragma unroll
                                for (int j = 0; j < 8; ++j)
#pragma unroll
                                    for (int e = 0; e < 2; ++e)
                                        if (!(sees >> (8 * j + e) & 1)) x[4 * j + 2 * k + e] = 0xFF800000u;
                            }
                        }
                        // The maximum moves only when it grows by 2^kLazy: until then the
                        // weights may pass 1, and sum and output stay as they are.
                        float top[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            top[k] = fmaxf(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1]));
#pragma unroll
                            for (int j = 1; j < 8; ++j)
                                top[k] = fmaxf(top[k], fmaxf(__uint_as_float(x[4 * j + 2 * k]),
                                                             __uint_as_float(x[4 * j + 2 * k + 1])));
                            if (kQuant) top[k] -= kHalfRoom;
                            else top[k] *= c;
                        }
                        auto grows = [&](int k) {
                            return top[k] > now[k].mx + kLazy || (now[k].mx == -INFINITY && top[k] > now[k].mx);
                        };
                        if (__any_sync(kFullMask, grows(0) || grows(1))) {
                            float f[2];
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                top[k] = fmaxf(top[k], __shfl_xor_sync(kFullMask, top[k], 1));
                                top[k] = fmaxf(top[k], __shfl_xor_sync(kFullMask, top[k], 2));
                                const bool grow = grows(k);
                                f[k] = grow ? exp2_approx(now[k].mx - top[k]) : 1.0f;
                                if (grow) now[k].mx = top[k];
                                now[k].l *= f[k];
                            }
                            if (i > 0) {
                                if (!wait(&ctl.o_done[(tile - 1) & 1], (tile - 1) >> 1)) break;
                                tmem_fence_after();
#pragma unroll 1
                                for (int d = 0; d < D; d += 64) {
                                    uint32_t o[32];
                                    tmem_load_rows16(at + 2 * kTile + d, o);
                                    tmem_wait_load(o);
#pragma unroll
                                    for (int j = 0; j < 32; ++j)
                                        o[j] = __float_as_uint(__uint_as_float(o[j]) * f[j >> 1 & 1]);
                                    tmem_store_rows16(at + 2 * kTile + d, o);
                                }
                            }
                        }
                        uint32_t w[16];
                        if constexpr (kQuant) {
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                f1[j] = *reinterpret_cast<const float2 *>(&sc.v_inv[b][8 * j + column]);
                        }
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float shift = now[k].mx == -INFINITY ? 0.0f : now[k].mx;
                            float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                if constexpr (kQuant) {
                                    const float2 y = add2(pair(2 * j + k), make_float2(-shift, -shift));
                                    const float2 u = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                                    sum = fma2(u, f1[j], sum);
                                    // (half, 11 digits: exact codes times it, and eight times
                                    // finer than the output)
                                    const __half2 two = __floats2half2_rn(u.x, u.y);
                                    w[2 * j + k] = *reinterpret_cast<const uint32_t *>(&two);
                                } else {
                                    const float2 y = fma2(pair(2 * j + k), make_float2(c, c), make_float2(-shift, -shift));
                                    const float2 u = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                                    sum = add2(u, sum);
                                    // (bfloat16, 8 digits, as the values are: a product takes
                                    // operands of one type.  The sum keeps all digits, for
                                    // lse.  The output's error against 64 bits is 0.0023 of
                                    // it, 0.0017 with weights of 32 bits)
                                    const __nv_bfloat162 two = __floats2bfloat162_rn(u.x, u.y);
                                    w[2 * j + k] = *reinterpret_cast<const uint32_t *>(&two);
                                }
                            }
                            now[k].l += sum.x + sum.y;
                        }
                        // the weights over the scores, which have been read
                        tmem_store_pairs16(at + b * kTile, w);
                        if (halves == 2)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const Row r = now[k];
                                now[k] = other[k];
                                other[k] = r;
                            }
                    }
                    tmem_wait_store();  // before giving up too: the columns are about to be freed
                    if (!ok) break;
                }
                if (!kQuant && p0 + kTile > s.q.P) {
                    // Values past the request's end become zeros, and so do NaN
                    // and infinities of the window (0 x NaN would reach rows that
                    // do not see them); the rows that do get them at the end.
                    // (loads come K0, K1, V0, K2, V1, ..., V(n-1))
                    const unsigned load = loads + (i + 1 < s.count ? 2 * i + 2 : 2 * i + 1);
                    const unsigned slot = load % S::kBufs;
                    if (!wait(&ctl.full[slot], load / S::kBufs)) break;
                    unsigned char *buf = smem + S::kQBytes + slot * S::kBufBytes;
                    for (int j = tid; j < kTile * kChunks; j += 128) {
                        const int tok = j / kChunks, ch = j % kChunks, pos = p0 + tok;
                        if (pos < s.q.P) continue;
                        uint4 *at = reinterpret_cast<uint4 *>(buf + (ch / 8) * kHalfBytes + tok * 128 +
                                                              ((ch % 8 ^ (tok & 7)) << 4));
                        uint4 v = make_uint4(0, 0, 0, 0);
                        if (pos < n) {
                            v = *at;
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
                            atomicOr(&ctl.nonfinite[seg & 3], 1u << (pos - s.q.P));
                        }
                        *at = v;
                    }
                    fence_async_proxy();
                }
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&ctl.p_ready[b]));
            }
            const unsigned last = done + s.count - 1;
            if (!wait(&ctl.o_done[last & 1], last >> 1)) continue;
            done += s.count;
            loads += 2 * s.count;
            tmem_fence_after();

            const bool whole = s.count == s.q.tiles;
            // from here on a lane is a row
            float row_mx = 0.0f, row_l = 0.0f;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float sum = h ? other[k].l : now[k].l;
                    sum += __shfl_xor_sync(kFullMask, sum, 1);
                    sum += __shfl_xor_sync(kFullMask, sum, 2);
                    const float u = __shfl_sync(kFullMask, h ? other[k].mx : now[k].mx, lane % 8 * 4);
                    const float v = __shfl_sync(kFullMask, sum, lane % 8 * 4);
                    if (lane / 8 == 2 * h + k) row_mx = u, row_l = v;
                }
            const float shift = row_mx == -INFINITY ? 0.0f : row_mx;
            const unsigned extra = *(volatile unsigned *)&ctl.nonfinite[seg & 3] & bits;
            const int slot = 2 * cta + (seg > 0);
            if (active) {
                const float inv = row_l == 0.0f ? 0.0f : 1.0f / row_l;
                __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + packed * a.ld_out +
                                     (long long)head * D;
#pragma unroll 1
                for (int h = 0; h < D / 32; ++h) {
                    uint32_t o[32];
                    tmem_load32(lanes + 2 * kTile + h * 32, o);
                    tmem_wait_load(o);
                    for (unsigned e = extra; e; e &= e - 1) {
                        int tok;
                        const int page = kv_page(a.cache, s.r, (long long)s.q.P + __ffs(e) - 1, &tok);
                        if (page < 0) continue;
                        using E = typename std::conditional<kQuant, e4m3, __nv_bfloat16>::type;
                        const E *v = reinterpret_cast<const E *>(a.cache.v) +
                                     kv_offset(a.cache, page, tok, s.head) + h * 32;
                        float f = 1.0f;
                        if constexpr (kQuant)
                            f = __ldg(a.cache.v_scale + kv_scale_offset(a.cache, page, tok, s.head));
#pragma unroll
                        for (int j = 0; j < 32; ++j) {
                            const float y = elem_value(v[j]) * f;
                            if (!(y - y == 0.0f)) o[j] = __float_as_uint(__uint_as_float(o[j]) + y);
                        }
                    }
                    if (!whole) {
                        float4 *part = reinterpret_cast<float4 *>(t.part_o) +
                                       ((long long)slot * (D / 4) + h * 8) * kRowsPerTile + m;
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (own) part[j * kRowsPerTile] =
                                make_float4(__uint_as_float(o[4 * j]), __uint_as_float(o[4 * j + 1]),
                                            __uint_as_float(o[4 * j + 2]), __uint_as_float(o[4 * j + 3]));
                    } else if (valid) {
                        uint32_t w[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            float u = __uint_as_float(o[2 * j]) * inv, v = __uint_as_float(o[2 * j + 1]) * inv;
                            if (row_l == 0.0f) u = v = 0.0f;
                            const __nv_bfloat162 two = __floats2bfloat162_rn(u, v);
                            w[j] = *reinterpret_cast<const uint32_t *>(&two);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            reinterpret_cast<uint4 *>(out + h * 32)[j] =
                                make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
                    }
                }
                if (!whole && own) {
                    t.part_ml[(long long)slot * 2 * kRowsPerTile + m] = row_mx;
                    t.part_ml[((long long)slot * 2 + 1) * kRowsPerTile + m] = row_l;
                } else if (whole && valid && a.lse) {
                    a.lse[(long long)packed * a.n_q_heads + head] =
                        row_l == 0.0f ? -INFINITY : shift * kLn2 + logf(row_l);
                }
            }
            tmem_fence_before();
            ++seg;
            if (tid == 0 && walk.left <= 0 && !whole) note_split(t, s, deal, lo, hi, seg - 1, token0, rows);
        }
    }
    __syncthreads();
    if (warp == S::kScoreWarp) tmem_free(tmem, kTmemCols);
}

// Joins the parts of the jobs that several CTAs share, in the CTAs' order: a block for
// each of these CTAs but the last takes its share of the columns, four of them a warp, and
// 32 rows, a lane each; warps to spare deal the parts among them.  Each block does little,
// and most do nothing (a CTA whose jobs are whole), so that the launch is what it costs;
// with one block a job instead, a call of a single token over 131040 takes 94 us, not 76.
constexpr int kJoinWarps = 16;

template <int D>
__global__ void __launch_bounds__(kJoinWarps * 32, 2) attend_join_kernel(const TensorArgs t) {
    constexpr int kFours = D / 4;
    __shared__ float4 part[kJoinWarps][32];
    __shared__ float part_l[kJoinWarps][32];
    pdl_wait();
    pdl_trigger();
    int c0 = blockIdx.x;
    auto job = [&](int i) { return __ldcg(reinterpret_cast<const int4 *>(t.desc) + c0 * 2 + i); };
    int4 d0 = job(0), d1 = job(1);
    if (!d0.x) {
        if (d1.w < 0) return;
        c0 = d1.w;
        d0 = job(0);
        d1 = job(1);
    }
    const int base = blockIdx.y * 32;
    const int c1 = d0.y, kv_head = d1.x, token0 = d1.y, rows = d1.z;
    const int share = blockIdx.x - c0, shares = min(max(c1 - c0, 1), kFours);
    if (base >= rows || share >= shares) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, m = base + lane;
    auto slot = [&](int c) { return (long long)(c == c0 ? d0.z : 2 * c); };
    auto ml = [&](int c, int which) {
        return __ldcg(t.part_ml + (slot(c) * 2 + which) * kRowsPerTile + m);
    };
    const int head = kv_head * t.group + m % t.group;
    const long long packed = d0.w + token0 + m / t.group;
    auto from = [&](int c, int four) {
        return __ldcg(reinterpret_cast<const float4 *>(t.part_o) + (slot(c) * kFours + four) * kRowsPerTile + m);
    };
    auto add = [](float4 &x, float f, float4 y) {
        x.x = fmaf(f, y.x, x.x), x.y = fmaf(f, y.y, x.y), x.z = fmaf(f, y.z, x.z), x.w = fmaf(f, y.w, x.w);
    };
    auto put = [&](int four, float4 x, float shift, float l) {
        if (m >= rows) return;
        const float inv = 1.0f / l;
        if (l == 0.0f) x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        else x.x *= inv, x.y *= inv, x.z *= inv, x.w *= inv;
        const __nv_bfloat162 u = __floats2bfloat162_rn(x.x, x.y), v = __floats2bfloat162_rn(x.z, x.w);
        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(t.a.out) + packed * t.a.ld_out +
                                   (long long)head * D + four * 4) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&u), *reinterpret_cast<const uint32_t *>(&v));
        if (t.a.lse && four == 0)
            t.a.lse[packed * t.a.n_q_heads + head] = l == 0.0f ? -INFINITY : shift * kLn2 + logf(l);
    };
    const int begin = share * kFours / shares, end = (share + 1) * kFours / shares;
    float top = -INFINITY;
    if (end - begin > kJoinWarps) {
        // then there are two parts: all loads before the first use
        constexpr int kOwn = kFours / kJoinWarps, kParts = 2;
        float pm[kParts], pl[kParts], l = 0.0f;
        float4 po[kParts][kOwn], x[kOwn] = {};
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            pm[i] = c0 + i <= c1 ? ml(c0 + i, 0) : -INFINITY;
            pl[i] = c0 + i <= c1 ? ml(c0 + i, 1) : 0.0f;
#pragma unroll
            for (int j = 0; j < kOwn; ++j) {
                const int four = begin + warp + j * kJoinWarps;
                if (c0 + i <= c1 && four < end) po[i][j] = from(c0 + i, four);
            }
        }
#pragma unroll
        for (int i = 0; i < kParts; ++i) top = fmaxf(top, pm[i]);
        const float shift = top == -INFINITY ? 0.0f : top;
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
            if (c0 + i > c1) continue;
            const float f = exp2_approx(pm[i] - shift);
            l = fmaf(f, pl[i], l);
#pragma unroll
            for (int j = 0; j < kOwn; ++j)
                if (begin + warp + j * kJoinWarps < end) add(x[j], f, po[i][j]);
        }
#pragma unroll
        for (int j = 0; j < kOwn; ++j)
            if (begin + warp + j * kJoinWarps < end) put(begin + warp + j * kJoinWarps, x[j], shift, l);
        return;
    }
    // a four of columns a warp; warps to spare deal the parts among them
    const int n = end - begin, deals = kJoinWarps / n, deal = warp / n, four = begin + warp % n;
#pragma unroll 4
    for (int c = c0 + warp; c <= c1; c += kJoinWarps) top = fmaxf(top, ml(c, 0));
    part_l[warp][lane] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, part_l[w][lane]);
    const float shift = top == -INFINITY ? 0.0f : top;
    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    float l = 0.0f;
    if (deal < deals) {
#pragma unroll 4
        for (int c = c0 + deal; c <= c1; c += deals) {
            const float f = exp2_approx(ml(c, 0) - shift);
            l = fmaf(f, ml(c, 1), l);
            add(x, f, from(c, four));
        }
    }
    __syncthreads();
    part[warp][lane] = x;
    part_l[warp][lane] = l;
    __syncthreads();
    if (deal > 0) return;
    for (int w = warp + n; w < n * deals; w += n) {
        add(x, 1.0f, part[w][lane]);
        l += part_l[w][lane];
    }
    put(four, x, shift, l);
}

namespace {

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *,
                              CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                              CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, looked up once.
EncodeFn encoder() {
    static std::atomic<EncodeFn> kept{nullptr};
    EncodeFn f = kept.load(std::memory_order_acquire);
    if (f) return f;
    void *p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
        return nullptr;
    f = reinterpret_cast<EncodeFn>(p);
    kept.store(f, std::memory_order_release);
    return f;
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

// A 4-D tensor map of bfloat16 or bytes; boxes of `width` elements a row, with the
// swizzle of that many bytes or none.  (L2 promotion: a head's codes are 128 bytes beside
// the next head's, which 256 bytes fetch as well.  Two long contexts' trees then read 956
// MB, with 128 bytes 618, in the same 264 us: HBM does not bound them.)
bool encode(CUtensorMap *map, const void *p, int elem_bytes, int width, bool swizzle, const int64_t (&dims)[4],
            const int64_t (&strides)[3], int box1, int box3) {
    const EncodeFn f = encoder();
    if (!f) return false;
    cuuint64_t d[4], s[3];
    for (int i = 0; i < 4; ++i) d[i] = (cuuint64_t)dims[i];
    for (int i = 0; i < 3; ++i) s[i] = (cuuint64_t)(strides[i] * elem_bytes);
    const cuuint32_t box[4] = {(cuuint32_t)width, (cuuint32_t)box1, 1, (cuuint32_t)box3};
    const cuuint32_t ones[4] = {1, 1, 1, 1};
    const bool codes = elem_bytes == 1;
    return f(map, codes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
             const_cast<void *>(p), d, s, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
             !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE
             : width * elem_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether any of `rows` rows of `bytes` at a, ld_a bytes apart, shares a byte with one
// of those at b (no stride is below `bytes`).  Slices of one buffer, side by side or
// one after the other, do not.
bool rows_overlap(const void *a, int64_t ld_a, const void *b, int64_t ld_b, int64_t rows, int64_t bytes) {
    const int64_t x = (int64_t)reinterpret_cast<uintptr_t>(a), y = (int64_t)reinterpret_cast<uintptr_t>(b);
    if (y >= x + (rows - 1) * ld_a + bytes || x >= y + (rows - 1) * ld_b + bytes) return false;
    // the rows of b that begin last before, and first after, the begin of a row of a
    // (with equal strides one row of a stands for all)
    for (int64_t i = 0; i < (ld_a == ld_b ? 1 : rows); ++i) {
        const int64_t from = x + i * ld_a - y;
        const int64_t first = from / ld_b - (from % ld_b < 0);
        for (int64_t j = first; j <= first + 1; ++j) {
            const bool there = ld_a == ld_b ? j > -rows && j < rows : j >= 0 && j < rows;
            const int64_t off = j * ld_b - from;
            if (there && off < bytes && off > -bytes) return true;
        }
    }
    return false;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

size_t part_o_bytes(int D) { return (size_t)2 * kMaxCtas * kRowsPerTile * D * 4; }
size_t part_ml_bytes() { return (size_t)2 * kMaxCtas * kRowsPerTile * 2 * 4; }
size_t desc_bytes() { return (size_t)kMaxCtas * kDescInts * 4; }

// Whether a call runs on the tensor cores: 16-bit rows, head sizes whose
// output and two score tiles fit half of tensor memory, boxes of whole 8-row
// swizzle groups inside a page, and the strides and bases that TMA and the
// 16-byte accesses take.
bool tensor_fits(const AttendArgs &a, int dtype, const dspark_kv_cache &c) {
    if (dtype != DSPARK_DTYPE_BF16 || c.dtype == DSPARK_DTYPE_F32) return false;
    if ((c.head_dim != 64 && c.head_dim != 128) || c.page_size % 16) return false;
    if (a.n_q_heads / c.n_kv_heads > kRowsPerTile) return false;
    const int e = kv_elem_bytes(c.dtype);
    const int64_t strides[3] = {c.token_stride, c.head_stride, c.page_stride};
    for (int64_t s : strides)
        if (s * e % 16 || s < 1 || s * e >= (1ll << 40)) return false;
    return aligned(c.k, 16) && aligned(c.v, 16) && aligned(a.q, 16) && aligned(a.out, 16) &&
           a.ld_q % 8 == 0 && a.ld_out % 8 == 0 && a.ld_q < (1ll << 39);
}

// Whether fewrows.cuh takes a call's heads and layouts.
bool few_fits(const AttendArgs &a, const dspark_kv_cache &c) {
    return c.dtype == DSPARK_DTYPE_E4M3 && a.n_q_heads / c.n_kv_heads <= kFewRows &&
           aligned(c.k_scale, 16) && aligned(c.v_scale, 16);
}

TensorArgs tensor_args(const AttendArgs &a, const dspark_kv_cache &c, void *workspace, int rows) {
    TensorArgs t;
    t.a = a;
    t.group = a.n_q_heads / c.n_kv_heads;
    t.tokens = min(rows / t.group, DSPARK_MAX_WINDOW);
    t.few = min(rows / 2 / t.group, DSPARK_MAX_WINDOW);
    t.box = gcd(c.page_size, kTile);
    unsigned char *w = static_cast<unsigned char *>(workspace);
    const size_t o = part_o_bytes(c.head_dim);
    t.part_o = reinterpret_cast<float *>(w);
    t.part_ml = reinterpret_cast<float *>(w + o);
    t.desc = reinterpret_cast<int *>(w + o + part_ml_bytes());
    // A split job's parts are joined by a second launch.  Where no request can have more
    // than kWholeTiles tiles, a job stays whole and that launch is not made.
    t.whole = (long long)c.table_width * c.page_size <= kWholeTiles * kTile;
    t.choose = 0;
    return t;
}

template <int D>
cudaError_t launch_join(const TensorArgs &t, int grid, int rows, cudaStream_t stream) {
    if (t.whole) return cudaSuccess;
    return launch_pdl(attend_join_kernel<D>, dim3(grid, (rows + 31) / 32), dim3(kJoinWarps * 32), 0, stream, t);
}

template <int D>
cudaError_t launch_few(const AttendArgs &a, const dspark_kv_cache &c, void *workspace, bool choose,
                       cudaStream_t stream) {
    constexpr int kSmem = FewShape<D>::kRing + (int)sizeof(FewControl);
    TensorArgs t = tensor_args(a, c, workspace, kFewRows);
    t.choose = choose;
    cudaError_t e = ensure_smem(reinterpret_cast<const void *>(attend_few_kernel<D>), kSmem, 24 + (D == 128));
    if (e != cudaSuccess) return e;
    const int grid = min(2 * sm_count(), kMaxCtas);
    e = launch_pdl(attend_few_kernel<D>, dim3(grid), dim3(kFewWarps * 32), kSmem, stream, t);
    return e != cudaSuccess || choose ? e : launch_join<D>(t, grid, kFewRows, stream);
}

template <int D, bool kQuant>
cudaError_t launch_tensor(const AttendArgs &a, const dspark_kv_cache &c, void *workspace, bool choose,
                          cudaStream_t stream) {
    using S = TensorShape<D, kQuant>;
    constexpr int kSmemSlot = 20 + (D == 128) + 2 * kQuant;  // of ensure_smem
    TensorArgs t = tensor_args(a, c, workspace, kRowsPerTile);
    t.choose = choose;
    // the cache as [page][head][token][element], the queries as [row][kv head]
    // [head of it][element]
    const int64_t dims[4] = {D, c.page_size, c.n_kv_heads, c.n_pages};
    const int64_t strides[3] = {c.token_stride, c.head_stride, c.page_stride};
    const int64_t q_dims[4] = {D, t.group, c.n_kv_heads, a.max_rows};
    const int64_t q_strides[3] = {D, (int64_t)t.group * D, a.ld_q};
    const int e_bytes = kv_elem_bytes(c.dtype), width = kQuant ? D : 64;
    CUtensorMap map_k, map_v, map_q, map_few;
    if (!encode(&map_k, c.k, e_bytes, width, true, dims, strides, t.box, 1) ||
        !encode(&map_v, c.v, e_bytes, width, !kQuant, dims, strides, t.box, 1) ||
        !encode(&map_q, a.q, 2, 64, true, q_dims, q_strides, t.group, t.tokens) ||
        !encode(&map_few, a.q, 2, 64, true, q_dims, q_strides, t.group, max(t.few, 1)))
        return cudaErrorUnknown;
    cudaError_t e = ensure_smem(reinterpret_cast<const void *>(attend_tensor_kernel<D, kQuant>),
                                S::kTotal, kSmemSlot);
    if (e != cudaSuccess) return e;
    const int grid = min(2 * sm_count(), kMaxCtas);
    e = launch_pdl(attend_tensor_kernel<D, kQuant>, dim3(grid), dim3(S::kThreads), S::kTotal, stream,
                   map_k, map_v, map_q, map_few, t);
    return e != cudaSuccess ? e : launch_join<D>(t, grid, min(t.tokens, a.max_rows) * t.group, stream);
}

}  // namespace

}  // namespace dspark

using namespace dspark;

extern "C" size_t dspark_tree_attention_workspace_bytes(int32_t n_q_heads, int32_t head_dim) {
    if (n_q_heads < 1 || head_dim < 2 || head_dim > DSPARK_MAX_HEAD_DIM) return 0;
    return round256(part_o_bytes(head_dim) + part_ml_bytes() + desc_bytes());
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
    // (a split job reads its queries again after another CTA has written its outputs)
    const int64_t e_bytes = kv_elem_bytes(dtype);
    if (rows_overlap(q, ld_q * e_bytes, out, ld_out * e_bytes, max_rows, width * e_bytes))
        return DSPARK_ERR_INVALID_ARG;
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
    cudaError_t e;
    const bool quant = cache->dtype == DSPARK_DTYPE_E4M3, small = cache->head_dim == 64;
    if (tensor_fits(a, dtype, *cache)) {
        // Few rows over E4M3: where the rows that the call has room for are not few in any
        // one request, both kernels are launched, and the requests' lengths tell which of
        // them works and which leaves at once (1 to 4 us).
        const bool few = quant && few_fits(a, *cache);
        const bool always = few && a.max_rows * (a.n_q_heads / cache->n_kv_heads) <= kFewRows;
        e = cudaSuccess;
        if (few) e = small ? launch_few<64>(a, *cache, workspace, !always, st)
                           : launch_few<128>(a, *cache, workspace, !always, st);
        if (e == cudaSuccess && !always)
            e = quant ? small ? launch_tensor<64, true>(a, *cache, workspace, few, st)
                              : launch_tensor<128, true>(a, *cache, workspace, few, st)
                : small ? launch_tensor<64, false>(a, *cache, workspace, false, st)
                        : launch_tensor<128, false>(a, *cache, workspace, false, st);
    } else {
        e = dtype == DSPARK_DTYPE_BF16 ? launch_any<__nv_bfloat16>(a, cache->dtype, st)
                                       : launch_any<float>(a, cache->dtype, st);
    }
    return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
