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
//
// latent_tensor_kernel   bfloat16 over a bfloat16 cache with 512 + 64 elements a token, on
//   the tensor cores.  A job is a request and 64 of its (token, head) rows, taken as they
//   come, so that a tile may end inside a token; a step is 64 positions, whose entries are
//   fetched once for both products:  S = Q [C | R]^T into tensor memory, then
//     y = S c   m' = max(m, max y)   w = 2^(y - m')   l = l 2^(m - m') + sum w
//     O = O 2^(m - m') + W C
//   m moves only when a row's maximum grows by 2^kLazy (until then w may pass 1, and O is
//   not touched).  64 rows, not 128, since O alone is 512 columns of 32 bits a row and
//   tensor memory has 512 columns for 128 lanes: with 64 rows O takes half of it, two
//   score tiles an eighth, and two thirds of the queries the rest, which leaves shared
//   memory for two and a half tiles of entries.
//   One warp copies (TMA), one issues both products, four do the softmax, a thread half a
//   row's positions, and four bring the next job's queries.  One CTA an SM.  CTAs work in
//   teams of two where requests have more rows than a tile: the two take neighbouring row
//   tiles over the same positions at the same time, so that the entries come from HBM once
//   and from L2 the second time.  The tiles of all jobs are dealt evenly to the teams, so
//   jobs are split along the positions where there are few, and latent_join_kernel adds
//   the parts in a fixed order.

#include "latentcache.cuh"
#include "schedule.cuh"
#include "tensor.cuh"
#include "tensormap.cuh"

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

// --------------------------------------------------- tensor-core kernel

constexpr int kLatent = 512, kEntry = 576;  // of an entry, its latent part
constexpr int kRows = 64;                   // (token, head) rows of a job
constexpr int kLatentCtas = 160;            // at most
constexpr int kChunkBytes = kTile * 128;    // 64 elements of 64 tokens, or of 64 rows
constexpr int kUnitBytes = 4 * kChunkBytes; // half of a tile's latent parts
constexpr int kUnits = 5, kKeyParts = 3;    // buffers: 2.5 tiles
constexpr int kQChunks = 6;                 // 64-element parts of the queries in tensor memory
constexpr int kQAt = 0;                     // the other three, in shared memory
constexpr int kUnitAt = kQAt + 3 * kChunkBytes;
constexpr int kKeyAt = kUnitAt + kUnits * kUnitBytes;
constexpr int kWeightsAt = kKeyAt + kKeyParts * kChunkBytes;
constexpr int kControlAt = kWeightsAt + 2 * kChunkBytes;
constexpr int kLatentSmem = kControlAt + 2816;
constexpr int kOutCol = 0, kScoreCol = 256, kQueryCol = 320;  // columns of tensor memory
constexpr int kLatentThreads = 320, kCopyWarp = 8, kMatrixWarp = 9;
constexpr int kLookAhead = 4;  // tiles whose pages are known, and asked for, ahead of their copy
constexpr int kLatentJobCost = 2;  // of a job's begin and end, in tiles
constexpr int kLatentDesc = 8;     // words about a split job, for the join

struct LatentTensorArgs {
    AttendArgs a;
    int box;    // cache tokens a TMA box
    int whole;  // no job is split
    float *part_o;   // [2 kLatentCtas][128][64] float4
    float *part_ml;  // [2 kLatentCtas][2][64]
    int *desc;       // [kLatentCtas][kLatentDesc]
};

struct LatentRequest {
    int row0, len, P, tiles, row_tiles;
};

__device__ __forceinline__ bool to_latent(const LatentTensorArgs &t, const Window &w, LatentRequest *q, bool report) {
    if (!usable(t.a, w, report)) return false;
    q->row0 = w.lo;
    q->len = w.hi - w.lo;
    q->P = w.P;
    q->tiles = (q->P + q->len + kTile - 1) / kTile;
    q->row_tiles = (q->len * t.a.n_q_heads + kRows - 1) / kRows;
    return true;
}

// Consecutive tiles of one job that a CTA works through.
struct LatentSegment {
    LatentRequest q = {};
    int r, row_tile, first, count;
    unsigned k;  // how many the team had before it
};

// Where a team's share begins: the request, which team's worth of its row tiles, and the
// unit of that.
struct LatentBegin {
    int r, group, unit, left;
    LatentRequest q;
};

// Walks a team's units: requests in order, in each the row tiles, a team's worth at a
// time, in each the positions.  Every warp role walks on its own and sees the same.
struct LatentWalk {
    int left, r, group, unit, team, member;
    unsigned k;
    LatentRequest q = {};
    Window ahead;

    __device__ __forceinline__ void begin(const LatentTensorArgs &t, const LatentBegin &b, int team_size, int of) {
        left = b.left;
        r = b.r;
        group = b.group;
        unit = b.unit;
        q = b.q;
        team = team_size;
        member = of;
        k = 0;
        ahead = load_window(t.a, min(r + 1, t.a.B - 1));
    }
    __device__ __forceinline__ bool next(const LatentTensorArgs &t, LatentSegment *s) {
        while (left > 0) {
            const int take = t.whole ? 1 : min(q.tiles + kLatentJobCost - unit, left);
            s->q = q;
            s->r = r;
            s->row_tile = group * team + member;
            s->first = max(unit - kLatentJobCost, 0);
            s->count = t.whole ? q.tiles : max(unit + take - kLatentJobCost, 0) - s->first;
            s->k = k;
            left -= take;
            unit = 0;
            if (++group * team >= q.row_tiles) {
                group = 0;
                while (left > 0) {
                    const bool has = to_latent(t, ahead, &q, false);
                    ++r;
                    ahead = load_window(t.a, min(r + 1, t.a.B - 1));
                    if (has) break;
                }
            }
            if (s->count > 0) {
                ++k;
                if (s->row_tile < s->q.row_tiles) return true;  // (else the other member's alone)
            }
        }
        return false;
    }
};

// The size of teams, this CTA's team's share and where it begins (for all after the next
// barrier); false where none are left for it.
//   Teams of one do row_tiles x tiles steps on each CTA, each of whose entries may come from
// HBM; teams of two do half as many, a step of which takes 0.92 of the time of two (an idle
// member where the row tiles are odd; the entries come from HBM once).
__device__ __forceinline__ bool latent_share(const LatentTensorArgs &t, LatentBegin *begin, long long *scan,
                                             Deal *deal, int *team_size) {
    const AttendArgs &a = t.a;
    const int tid = threadIdx.x, cta = blockIdx.x;
    const int per = (a.B + kLatentThreads - 1) / kLatentThreads;
    long long alone = 0, paired = 0;
    LatentRequest q = {};
    for (int i = 0, r = tid * per; i < per && r < a.B; ++i, ++r)
        if (to_latent(t, load_window(a, r), &q, cta == 0)) {
            const int job = t.whole ? 1 : q.tiles + kLatentJobCost;
            alone += (long long)job * q.row_tiles;
            paired += (long long)job * ((q.row_tiles + 1) / 2);
        }
    const long long sum_alone = block_sum<long long>(alone, scan), sum_paired = block_sum<long long>(paired, scan);
    const int team = t.whole || 12 * sum_alone <= 13 * sum_paired ? 1 : 2;
    const long long mine = team == 1 ? alone : paired, T = team == 1 ? sum_alone : sum_paired;
    long long total;
    const long long before = block_exclusive_scan<long long>(mine, scan, &total);
    const int n = (int)min((long long)((int)gridDim.x / team),
                           t.whole ? T : (T + kLatentJobCost + 1) / (kLatentJobCost + 2));
    if (tid == 0 && !t.whole) {
        t.desc[cta * kLatentDesc] = 0;
        t.desc[cta * kLatentDesc + 7] = -1;
    }
    const int at = cta / team;
    if (at >= n) return false;
    deal->n = n;
    deal->each = div_nonneg(T, n);
    deal->rest = (int)(T - deal->each * n);
    *team_size = team;
    const long long lo = deal->first(at), hi = deal->first(at + 1);
    if (lo >= before && lo < before + mine) {
        long long from = before;
        for (int r = tid * per;; ++r) {
            if (per > 1 && !to_latent(t, load_window(a, r), &q, false)) continue;
            const int job = t.whole ? 1 : q.tiles + kLatentJobCost;
            const long long units = (long long)job * ((q.row_tiles + team - 1) / team);
            if (lo >= from + units) {
                from += units;
                continue;
            }
            begin->r = r;
            begin->group = (int)div_nonneg(lo - from, job);
            begin->unit = (int)(lo - from - (long long)begin->group * job);
            begin->left = (int)(hi - lo);
            begin->q = q;
            break;
        }
    }
    return true;
}

struct alignas(16) LatentControl {
    unsigned long long unit_full[kUnits], unit_empty[kUnits], key_full[kKeyParts], key_empty[kKeyParts];
    unsigned long long s_full[2], p_ready[2], o_done[2], q_full, q_empty, o_free, drain;
    unsigned tmem;
    unsigned nonfinite[4];  // window tokens whose values were zeroed, by segment
    int abort;
    LatentBegin begin;
    long long scan[40];
    float top[2][2][kRows];  // [tile's parity][half of the positions]
    float sum[2][kRows];
};
static_assert(sizeof(LatentControl) <= 2816 && kLatentSmem <= 227 * 1024, "shared memory");

// Where the entries of 64 rows x 64 elements lie: 16-byte piece c of row r.
__device__ __forceinline__ int chunk_piece(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

__global__ void __launch_bounds__(kLatentThreads, 1)
latent_tensor_kernel(const __grid_constant__ CUtensorMap map, const LatentTensorArgs t) {
    extern __shared__ __align__(1024) unsigned char smem[];
    LatentControl &ctl = *reinterpret_cast<LatentControl *>(smem + kControlAt);
    const AttendArgs &a = t.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = smem_addr(smem);
    if (tid == 0) {
        for (int i = 0; i < kUnits; ++i) {
            mbar_init(smem_addr(&ctl.unit_full[i]), 1);
            mbar_init(smem_addr(&ctl.unit_empty[i]), 1);
        }
        for (int i = 0; i < kKeyParts; ++i) {
            mbar_init(smem_addr(&ctl.key_full[i]), 1);
            mbar_init(smem_addr(&ctl.key_empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&ctl.s_full[i]), 1);
            mbar_init(smem_addr(&ctl.p_ready[i]), 4);
            mbar_init(smem_addr(&ctl.o_done[i]), 1);
        }
        mbar_init(smem_addr(&ctl.q_full), 4);
        mbar_init(smem_addr(&ctl.q_empty), 1);
        mbar_init(smem_addr(&ctl.o_free), 4);
        mbar_init(smem_addr(&ctl.drain), 1);
        ctl.abort = 0;
        for (int i = 0; i < 4; ++i) ctl.nonfinite[i] = 0;
        fence_mbar_init();
        prefetch_map(&map);
    }
    if (warp == kMatrixWarp) tmem_alloc(smem_addr(&ctl.tmem), 512);
    pdl_wait();
    pdl_trigger();

    Deal deal;
    int team;
    const int cta = blockIdx.x;
    if (!latent_share(t, &ctl.begin, ctl.scan, &deal, &team)) {
        if (warp == kMatrixWarp) {
            __syncwarp();
            tmem_free(*(volatile unsigned *)&ctl.tmem, 512);
        }
        return;
    }
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = ctl.tmem;
    volatile int *abort = &ctl.abort;
    LatentWalk walk;
    walk.begin(t, ctl.begin, team, cta % team);
    LatentSegment s = {};
    bool ok = true;
    auto wait = [&](unsigned long long *bar, unsigned parity) {
        return ok = warp_wait(ok, smem_addr(bar), parity, abort, a.status);
    };
    const int hq = a.n_q_heads;
    unsigned done = 0, seg = 0;  // tiles and segments so far

    if (warp == kCopyWarp) {
        // ------------------------------------------------ copy warp
        const int boxes = kTile / t.box;
        const int box = lane >> 2, chunk = lane & 3;  // of a unit; lane b < boxes looks up box b
        unsigned unit = 0, unit_parity = 0, part = 0, part_parity = 0;
        while (ok && walk.next(t, &s)) {
            const int n = s.q.P + s.q.len, from = s.first * kTile + lane * t.box;
            // what each of the team's two asks L2 for, if both are there: the latent part's
            // first half, with the key part, or its second half
            const bool both = team == 2 && (s.row_tile ^ 1) < s.q.row_tiles;
            const bool first_half = !both || cta % 2 == 0, second_half = !both || cta % 2 == 1;
            Place at;
            at.begin(a.cache, lane < boxes ? from : 0);
            // tile i's page and token of this lane's box, kLookAhead tiles ahead
            int pages[kLookAhead + 1], tokens[kLookAhead + 1];
            auto look_up = [&](int i) {
                tokens[kLookAhead] = at.token;
                pages[kLookAhead] = at.entry(a.cache, s.r, lane < boxes && i < s.count && from + i * kTile < n);
                at.step(a.cache);
            };
            auto shift = [&]() {
#pragma unroll
                for (int j = 0; j < kLookAhead; ++j) pages[j] = pages[j + 1], tokens[j] = tokens[j + 1];
            };
            auto fetch = [&](int i) {  // to L2, the tile looked up before the last
                const int page = pages[kLookAhead - 1], token = tokens[kLookAhead - 1];
                if (i >= s.count) return;
                const int my_page = __shfl_sync(kFullMask, page, box), my_token = __shfl_sync(kFullMask, token, box);
                if (box >= boxes || (unsigned)my_page >= (unsigned)a.cache.n_pages) return;
                if (first_half) {
                    if (chunk == 0) tma_prefetch_4d(&map, kLatent, my_token, 0, my_page);
                    tma_prefetch_4d(&map, chunk * 64, my_token, 0, my_page);
                }
                if (second_half) tma_prefetch_4d(&map, (4 + chunk) * 64, my_token, 0, my_page);
            };
#pragma unroll
            for (int j = 0; j < kLookAhead; ++j) {
                look_up(j);
                shift();
            }
            for (int i = 0; i < s.count; ++i) {
                look_up(i + kLookAhead);
                int page = pages[0];
                const int token = tokens[0];
                // a page outside the pool, as past the request's end, arrives as zeros
                if (lane < boxes && from + i * kTile < n && (unsigned)page >= (unsigned)a.cache.n_pages) {
                    flag(a.status, DSPARK_STATUS_BAD_INDEX);
                    page = a.cache.n_pages;
                }
                const int my_page = __shfl_sync(kFullMask, page, box), my_token = __shfl_sync(kFullMask, token, box);
                fetch(i + kLookAhead - 1);
                shift();
                if (!wait(&ctl.key_empty[part], part_parity ^ 1)) break;
                const uint32_t key_bar = smem_addr(&ctl.key_full[part]);
                if (lane == 0) mbar_expect(key_bar, kChunkBytes);
                __syncwarp();
                if (lane < boxes)
                    tma_load_4d(base + kKeyAt + part * kChunkBytes + lane * t.box * 128, &map, kLatent, token, 0, page,
                                key_bar);
                if (++part == kKeyParts) part = 0, part_parity ^= 1;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    if (!wait(&ctl.unit_empty[unit], unit_parity ^ 1)) break;
                    const uint32_t bar = smem_addr(&ctl.unit_full[unit]);
                    if (lane == 0) mbar_expect(bar, kUnitBytes);
                    __syncwarp();
                    if (box < boxes)
                        tma_load_4d(base + kUnitAt + unit * kUnitBytes + chunk * kChunkBytes + box * t.box * 128, &map,
                                    (4 * h + chunk) * 64, my_token, 0, my_page, bar);
                    if (++unit == kUnits) unit = 0, unit_parity ^= 1;
                }
                if (!ok) break;
            }
        }
        if (!ok && lane == 0) {
            // copies still under way write this block's buffers: the last load of each
            // slot, complete or never begun
            for (int i = 0; i < kUnits; ++i)
                mbar_wait(smem_addr(&ctl.unit_full[i]), i < (int)unit ? unit_parity : unit_parity ^ 1);
            for (int i = 0; i < kKeyParts; ++i)
                mbar_wait(smem_addr(&ctl.key_full[i]), i < (int)part ? part_parity : part_parity ^ 1);
        }
    } else if (warp == kMatrixWarp) {
        // ---------------------------------------------- matrix warp
        // Keeps step as a whole, so that addresses stay in uniform registers; one lane
        // issues.  Scores of tile i, then the output of tile i - 1, whose weights are
        // computed meanwhile.
        constexpr uint32_t score_word = mma_word(true, kTile, false) - kHalfRows;
        constexpr uint32_t value_word = mma_word(true, 256, true) - kHalfRows;
        const uint32_t ubase = __shfl_sync(kFullMask, base, 0), utmem = __shfl_sync(kFullMask, tmem, 0);
        const bool leader = elect_one();
        const uint64_t desc_q = smem_operand(ubase + kQAt, 16, 128);
        const uint64_t desc_unit = smem_operand(ubase + kUnitAt, 16, 128);
        const uint64_t desc_value = smem_operand(ubase + kUnitAt, kChunkBytes, 128);
        const uint64_t desc_key = smem_operand(ubase + kKeyAt, 16, 128);
        const uint64_t desc_w = smem_operand(ubase + kWeightsAt, 16, 128);
        unsigned unit = 0, unit_parity = 0, value_unit = 0, part = 0, part_parity = 0;
        // O += W C of the segment's tile i
        auto values = [&](int i, unsigned tile) {
            if (i == 0 && seg > 0 && !wait(&ctl.o_free, seg - 1)) return;
            if (!wait(&ctl.p_ready[tile & 1], tile >> 1)) return;
            tmem_fence_after();
            const uint64_t w = desc_w + (tile & 1) * (kChunkBytes >> 4);
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                const uint64_t v = desc_value + value_unit * (kUnitBytes >> 4);
                if (leader) {
#pragma unroll
                    for (int k = 0; k < kTile / 16; ++k)
                        mma_ws_ss(utmem + kOutCol + 128 * h, w + (k * 32 >> 4), v + (k * 16 * 128 >> 4), value_word,
                                  i > 0 || k > 0);
                    mma_commit(smem_addr(&ctl.unit_empty[value_unit]));
                    if (h == 1) mma_commit(smem_addr(&ctl.o_done[tile & 1]));
                }
                __syncwarp();
                if (++value_unit == kUnits) value_unit = 0;
            }
        };
        while (ok && walk.next(t, &s)) {
            if (!wait(&ctl.q_full, seg)) break;
            const int count = __shfl_sync(kFullMask, s.count, 0);
            for (int i = 0; i < count; ++i) {
                // (the scores of tile - 2 have been read, and its weights multiplied)
                const unsigned tile = done + i;
                const uint32_t d = utmem + kScoreCol + (tile & 1) * 32;
                if (!wait(&ctl.key_full[part], part_parity)) break;
                tmem_fence_after();
                if (leader) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_ws_ss(d, desc_q + (2 * kChunkBytes + k * 32 >> 4),
                                  desc_key + (part * kChunkBytes + k * 32 >> 4), score_word, k > 0);
                    mma_commit(smem_addr(&ctl.key_empty[part]));
                }
                __syncwarp();
                if (++part == kKeyParts) part = 0, part_parity ^= 1;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (!wait(&ctl.unit_full[unit], unit_parity)) break;
                    tmem_fence_after();
                    if (leader) {
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const int c = 4 * h + k / 4;  // the 64-element part
                            const uint64_t b = desc_unit + (unit * kUnitBytes + k / 4 * kChunkBytes + k % 4 * 32 >> 4);
                            if (c < kQChunks)
                                mma_ws_ts(d, utmem + kQueryCol + c * 32 + k % 4 * 8, b, score_word, true);
                            else
                                mma_ws_ss(d, desc_q + ((c - kQChunks) * kChunkBytes + k % 4 * 32 >> 4), b, score_word,
                                          true);
                        }
                        if (h == 1) {
                            mma_commit(smem_addr(&ctl.s_full[tile & 1]));
                            if (i + 1 == count) mma_commit(smem_addr(&ctl.q_empty));
                        }
                    }
                    __syncwarp();
                    if (++unit == kUnits) unit = 0, unit_parity ^= 1;
                }
                if (!ok) break;
                if (i > 0) values(i - 1, tile - 1);
                if (!ok) break;
            }
            if (!ok) break;
            values(count - 1, done + count - 1);
            done += count;
            ++seg;
        }
        // after a timeout: products still under way write tensor memory and barriers of
        // this block
        if (!ok && leader) {
            mma_commit(smem_addr(&ctl.drain));
            mbar_wait(smem_addr(&ctl.drain), 0);
        }
        __syncwarp();
    } else if (warp >= 4) {
        // --------------------------------------------- query warps
        // A lane of tensor memory a thread: row m's first six parts into lanes m and 64 + m;
        // of the other three, which go to shared memory, each of the two takes half.
        const int lane_at = tid - 128, m = lane_at & 63, half = lane_at >> 6;
        const uint32_t lanes = tmem + ((uint32_t)(lane_at & ~31) << 16);
        while (ok && walk.next(t, &s)) {
            const int row = s.row_tile * kRows + m;
            const bool there = row < s.q.len * hq;
            const int token = there ? row / hq : 0, head = there ? row % hq : 0;
            const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) +
                                                             (s.q.row0 + token) * a.ld_q + (long long)head * kEntry);
            auto piece = [&](int i) { return there ? __ldg(q + i) : make_uint4(0, 0, 0, 0); };
            uint4 rest[12];
#pragma unroll
            for (int i = 0; i < 12; ++i) rest[i] = piece(8 * kQChunks + 12 * half + i);
            if (seg > 0 && !wait(&ctl.q_empty, seg - 1)) break;
#pragma unroll
            for (int i = 0; i < 12; ++i) {
                const int p = 12 * half + i;
                *reinterpret_cast<uint4 *>(smem + kQAt + p / 8 * kChunkBytes + chunk_piece(m, p % 8)) = rest[i];
            }
            tmem_fence_after();
#pragma unroll 2
            for (int c = 0; c < kQChunks; ++c) {
                uint32_t x[32];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint4 v = piece(8 * c + i);
                    x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
                }
                tmem_store32(lanes + kQueryCol + 32 * c, x);
            }
            tmem_wait_store();
            tmem_fence_before();
            fence_async_proxy();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&ctl.q_full));
            ++seg;
        }
    } else {
        // --------------------------------------------- softmax warps
        const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
        const float c = fmaxf(fabsf(a.scale) * kLog2e, 0x1p-100f);  // 0 would turn -inf into NaN
        const bool negative = a.scale < 0.0f;
        const int m = tid & 63, half = tid >> 6;  // a row, and which 32 of a tile's positions
        // The four warps meet once a tile and once behind the last: a warp that gave up comes
        // to the next such barrier, and all leave there.
        bool met = true;
        while (walk.next(t, &s)) {
            const int n = s.q.P + s.q.len, rows = min(s.q.len * hq - s.row_tile * kRows, kRows);
            const bool valid = m < rows;
            const int row = s.row_tile * kRows + min(m, rows - 1);
            const int token = row / hq, head = row % hq, packed = s.q.row0 + token;
            const unsigned bits = ancestors_of(a, packed, token, s.q.len);
            if (tid == 0) ctl.nonfinite[(seg + 2) & 3] = 0;  // the one's before the last
            float mx = -INFINITY, l = 0.0f;  // running maximum (to base 2); this half's sum
            for (int i = 0; i < s.count; ++i) {
                const unsigned tile = done + i, b = tile & 1;
                const int p0 = (s.first + i) * kTile;
                wait(&ctl.s_full[b], tile >> 1);
                tmem_fence_after();
                uint32_t x[32];
                tmem_load32(lanes + kScoreCol + 32 * b, x);
                tmem_wait_load(x);
                if (negative) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) x[j] ^= 0x80000000u;
                }
                if (p0 + kTile > s.q.P) {
                    // prefix positions, then the row's ancestors in the window
                    const int pre = max(s.q.P - p0, 0), skip = max(p0 - s.q.P, 0);
                    const unsigned long long w = skip < 32 ? (unsigned long long)(bits >> skip) : 0;
                    const unsigned sees = (unsigned)((w << pre | ((1ull << pre) - 1)) >> (32 * half));
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (!(sees >> j & 1)) x[j] = 0xFF800000u;
                }
                float part[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    part[j] = fmaxf(__uint_as_float(x[j]), __uint_as_float(x[j + 4]));
#pragma unroll
                    for (int k = 8 + j; k < 32; k += 4) part[j] = fmaxf(part[j], __uint_as_float(x[k]));
                }
                float top = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3])) * c;
                ctl.top[b][half][m] = top;
                if (!(met = named_all(1, 128, ok))) break;
                top = fmaxf(top, ctl.top[b][half ^ 1][m]);
                // The maximum moves only when it grows by 2^kLazy: until then the weights may
                // pass 1, and sum and output stay as they are.
                const bool grow = top > mx + kLazy || (mx == -INFINITY && top > mx);
                if (__any_sync(kFullMask, grow)) {
                    const float f = grow ? exp2_approx(mx - top) : 1.0f;
                    if (grow) mx = top;
                    l *= f;
                    if (i > 0) {
                        if (!wait(&ctl.o_done[(tile - 1) & 1], (tile - 1) >> 1)) continue;
                        tmem_fence_after();
#pragma unroll 1
                        for (int d = 0; d < 256; d += 32) {
                            uint32_t o[32];
                            tmem_load32(lanes + kOutCol + d, o);
                            tmem_wait_load(o);
#pragma unroll
                            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                            tmem_store32(lanes + kOutCol + d, o);
                        }
                        tmem_wait_store();
                    }
                }
                const float shift = mx == -INFINITY ? 0.0f : mx;
                float2 sum[2] = {};
                unsigned char *weights = smem + kWeightsAt + b * kChunkBytes;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t w[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int e = 8 * j + 2 * k;
                        const float2 y = fma2(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])),
                                              make_float2(c, c), make_float2(-shift, -shift));
                        const float2 u = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                        sum[k & 1] = add2(sum[k & 1], u);
                        // (bfloat16, 8 digits, as the latent vectors are: a product takes
                        // operands of one type.  The sum keeps all digits, for lse)
                        const __nv_bfloat162 two = __floats2bfloat162_rn(u.x, u.y);
                        w[k] = *reinterpret_cast<const uint32_t *>(&two);
                    }
                    *reinterpret_cast<uint4 *>(weights + chunk_piece(m, 4 * half + j)) =
                        make_uint4(w[0], w[1], w[2], w[3]);
                }
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                if (p0 + kTile > s.q.P) {
                    // Latent vectors past the request's end become zeros, and so do NaN and
                    // infinities of the window (0 x NaN would reach rows that do not see
                    // them); the rows that do get them at the end.  The scores have been
                    // computed.
                    const int from = max(s.q.P, p0);
                    for (int j = tid; j < (p0 + kTile - from) * 64; j += 128) {
                        const int pos = from + j / 64, piece = j % 64;  // of the latent part
                        const unsigned u = (2 * tile + piece / 32) % kUnits;
                        uint4 *at = reinterpret_cast<uint4 *>(smem + kUnitAt + u * kUnitBytes +
                                                              piece / 8 % 4 * kChunkBytes +
                                                              chunk_piece(pos - p0, piece % 8));
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
                }
                fence_async_proxy();
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_addr(&ctl.p_ready[b]));
            }
            if (!met) break;
            const unsigned last = done + s.count - 1;
            wait(&ctl.o_done[last & 1], last >> 1);
            done += s.count;
            tmem_fence_after();
            // the row's sum: both halves'
            ctl.sum[half][m] = l;
            if (!named_all(1, 128, ok)) break;
            l = ctl.sum[0][m] + ctl.sum[1][m];
            const bool whole = s.count == s.q.tiles;
            const unsigned extra = *(volatile unsigned *)&ctl.nonfinite[seg & 3] & bits;
            const int slot = 2 * cta + (s.k > 0);
            const float shift = mx == -INFINITY ? 0.0f : mx, inv = l == 0.0f ? 0.0f : 1.0f / l;
            __nv_bfloat16 *out =
                static_cast<__nv_bfloat16 *>(a.out) + packed * a.ld_out + (long long)head * kLatent;
#pragma unroll 1
            for (int d = 0; d < 256; d += 32) {
                // columns 0..127 are elements 0..255, a lane half 128 of them; the others
                // 256..511
                const int e = (d & 128) * 2 + 128 * half + (d & 127);
                uint32_t o[32];
                tmem_load32(lanes + kOutCol + d, o);
                tmem_wait_load(o);
                for (unsigned x = extra; x; x &= x - 1) {
                    int tok;
                    const int page = kv_page(a.cache, s.r, (long long)s.q.P + __ffs(x) - 1, &tok);
                    if (page < 0) continue;
                    const __nv_bfloat16 *v =
                        reinterpret_cast<const __nv_bfloat16 *>(a.cache.k) + kv_offset(a.cache, page, tok, 0) + e;
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const float y = elem_value(v[j]);
                        if (!(y - y == 0.0f)) o[j] = __float_as_uint(__uint_as_float(o[j]) + y);
                    }
                }
                if (!whole) {
                    float4 *part = reinterpret_cast<float4 *>(t.part_o) + ((long long)slot * 128 + e / 4) * kRows + m;
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        part[j * kRows] = make_float4(__uint_as_float(o[4 * j]), __uint_as_float(o[4 * j + 1]),
                                                      __uint_as_float(o[4 * j + 2]), __uint_as_float(o[4 * j + 3]));
                } else if (valid) {
                    uint32_t w[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float u = __uint_as_float(o[2 * j]) * inv, v = __uint_as_float(o[2 * j + 1]) * inv;
                        if (l == 0.0f) u = v = 0.0f;
                        const __nv_bfloat162 two = __floats2bfloat162_rn(u, v);
                        w[j] = *reinterpret_cast<const uint32_t *>(&two);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        reinterpret_cast<uint4 *>(out + e)[j] =
                            make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
                }
            }
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_addr(&ctl.o_free));
            if (half == 0) {
                if (!whole) {
                    t.part_ml[(long long)slot * 2 * kRows + m] = mx;
                    t.part_ml[((long long)slot * 2 + 1) * kRows + m] = l;
                } else if (valid && a.lse) {
                    a.lse[(long long)packed * hq + head] = l == 0.0f ? -INFINITY : shift * kLn2 + logf(l);
                }
            }
            ++seg;
            if (tid == 0 && !whole) {
                // what the join is told: of a job that begins here and ends in a later CTA, or
                // of the one that the whole of this CTA lies in
                const int at = cta / team;
                int *d = t.desc + cta * kLatentDesc;
                if (s.first == 0) {
                    const long long hi = deal.first(at + 1);
                    d[1] = deal.cta_of(hi - 1 + s.q.tiles - s.count, at) * team + cta % team;
                    d[2] = slot;
                    d[3] = s.q.row0;
                    d[4] = s.row_tile;
                    d[5] = rows;
                    d[6] = team;
                    d[0] = 1;
                } else if (s.k == 0 && s.first + s.count < s.q.tiles) {
                    // (where its first tile is)
                    d[7] = deal.cta_of(deal.first(at) - s.first, 0) * team + cta % team;
                }
            }
        }
    }
    __syncthreads();
    if (warp == kMatrixWarp) tmem_free(tmem, 512);
}

// Joins the parts of the jobs that several CTAs share, in the CTAs' order: a block for
// each of these CTAs but the last takes its share of the rows' fours of elements; threads to
// spare deal the parts among them.
constexpr int kLatentJoinThreads = 256, kLatentJoinPieces = 16;

__global__ void __launch_bounds__(kLatentJoinThreads) latent_join_kernel(const LatentTensorArgs t) {
    __shared__ float4 sum[kLatentJoinThreads];
    __shared__ float sum_l[kLatentJoinThreads];
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
    const int team = d1.z, rows = d1.y, n = (d0.y - c0) / team + 1;  // parts
    const int share = (blockIdx.x - c0) / team, shares = max(n - 1, 1);
    const long long fours = 128ll * rows, pieces = (long long)shares * gridDim.y;
    const long long piece = (long long)share * gridDim.y + blockIdx.y;
    const int begin = (int)(piece * fours / pieces), end = (int)((piece + 1) * fours / pieces);
    const int tid = threadIdx.x, hq = t.a.n_q_heads;
    auto slot = [&](int i) { return (long long)(i == 0 ? d0.z : 2 * (c0 + i * team)); };
    for (int base = begin; base < end; base += kLatentJoinThreads) {
        const int items = min(end - base, kLatentJoinThreads), deals = kLatentJoinThreads / items;
        const int deal = tid / items, item = base + tid % items, four = item / rows, m = item % rows;
        auto ml = [&](int i, int which) { return __ldcg(t.part_ml + (slot(i) * 2 + which) * kRows + m); };
        float top = -INFINITY;
        if (deal < deals)
#pragma unroll 4
            for (int i = deal; i < n; i += deals) top = fmaxf(top, ml(i, 0));
        sum_l[tid] = top;
        __syncthreads();
        for (int i = 0; i < deals; ++i) top = fmaxf(top, sum_l[i * items + tid % items]);
        const float shift = top == -INFINITY ? 0.0f : top;
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float l = 0.0f;
        if (deal < deals)
#pragma unroll 4
            for (int i = deal; i < n; i += deals) {
                const float f = exp2_approx(ml(i, 0) - shift);
                const float4 y =
                    __ldcg(reinterpret_cast<const float4 *>(t.part_o) + (slot(i) * 128 + four) * kRows + m);
                l = fmaf(f, ml(i, 1), l);
                x.x = fmaf(f, y.x, x.x), x.y = fmaf(f, y.y, x.y), x.z = fmaf(f, y.z, x.z), x.w = fmaf(f, y.w, x.w);
            }
        __syncthreads();
        sum[tid] = x;
        sum_l[tid] = l;
        __syncthreads();
        if (deal == 0) {
            for (int i = 1; i < deals; ++i) {
                const float4 y = sum[i * items + tid];
                x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
                l += sum_l[i * items + tid];
            }
            const float inv = 1.0f / l;
            if (l == 0.0f) x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            else x.x *= inv, x.y *= inv, x.z *= inv, x.w *= inv;
            const int row = d1.x * kRows + m, head = row % hq;
            const long long packed = d0.w + row / hq;
            const __nv_bfloat162 u = __floats2bfloat162_rn(x.x, x.y), v = __floats2bfloat162_rn(x.z, x.w);
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(t.a.out) + packed * t.a.ld_out +
                                       (long long)head * kLatent + four * 4) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&u), *reinterpret_cast<const uint32_t *>(&v));
            if (t.a.lse && four == 0)
                t.a.lse[packed * hq + head] = l == 0.0f ? -INFINITY : shift * kLn2 + logf(l);
        }
        __syncthreads();
    }
}

namespace {

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

size_t latent_part_o_bytes() { return (size_t)2 * kLatentCtas * kRows * kLatent * 4; }
size_t latent_part_ml_bytes() { return (size_t)2 * kLatentCtas * kRows * 2 * 4; }
size_t latent_desc_bytes() { return (size_t)kLatentCtas * kLatentDesc * 4; }

// Whether a call runs on the tensor cores: the dimensions that the kernel is laid out for,
// boxes of whole 8-row swizzle groups inside a page, and the strides and bases that TMA
// and the 16-byte accesses take.
bool latent_tensor_fits(const AttendArgs &a, int dtype, const dspark_latent_cache &c) {
    if (dtype != DSPARK_DTYPE_BF16 || c.dtype != DSPARK_DTYPE_BF16) return false;
    if (c.latent_dim != kLatent || c.latent_dim + c.rope_dim != kEntry || c.page_size % 16) return false;
    for (int64_t s : {c.token_stride, c.page_stride})
        if (s % 8 || s < 1 || s * 2 >= (1ll << 40)) return false;
    return aligned(c.data, 16) && aligned(a.q, 16) && aligned(a.out, 16) && a.ld_q % 8 == 0 && a.ld_out % 8 == 0 &&
           a.n_q_heads <= (1 << 20);
}

cudaError_t launch_latent_tensor(const AttendArgs &a, const dspark_latent_cache &c, void *workspace,
                                 cudaStream_t stream) {
    LatentTensorArgs t;
    t.a = a;
    t.box = gcd(c.page_size, kTile);
    // A split job's parts are joined by a second launch.  Where no request can have more
    // than kWholeTiles tiles, a job stays whole and that launch is not made.
    t.whole = (long long)c.table_width * c.page_size <= kWholeTiles * kTile;
    unsigned char *w = static_cast<unsigned char *>(workspace);
    t.part_o = reinterpret_cast<float *>(w);
    t.part_ml = reinterpret_cast<float *>(w + latent_part_o_bytes());
    t.desc = reinterpret_cast<int *>(w + latent_part_o_bytes() + latent_part_ml_bytes());
    const int64_t dims[4] = {kEntry, c.page_size, 1, c.n_pages};
    const int64_t strides[3] = {c.token_stride, c.page_stride, c.page_stride};
    CUtensorMap map;
    if (!encode(&map, c.data, 2, 64, true, dims, strides, t.box, 1)) return cudaErrorUnknown;
    cudaError_t e = ensure_smem(reinterpret_cast<const void *>(latent_tensor_kernel), kLatentSmem, 26);
    if (e != cudaSuccess) return e;
    const int grid = min(sm_count(), kLatentCtas);
    e = launch_pdl(latent_tensor_kernel, dim3(grid), dim3(kLatentThreads), kLatentSmem, stream, map, t);
    if (e != cudaSuccess || t.whole) return e;
    return launch_pdl(latent_join_kernel, dim3(grid, kLatentJoinPieces), dim3(kLatentJoinThreads), 0, stream, t);
}

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
    return round256(latent_part_o_bytes() + latent_part_ml_bytes() + latent_desc_bytes());
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
    const cudaError_t e = latent_tensor_fits(a, dtype, *cache) ? launch_latent_tensor(a, *cache, workspace, st)
                          : dtype == DSPARK_DTYPE_BF16         ? launch_any<__nv_bfloat16>(t, cache->dtype, st)
                                                               : launch_any<float>(t, cache->dtype, st);
    return e == cudaSuccess ? DSPARK_OK : DSPARK_ERR_CUDA;
}
