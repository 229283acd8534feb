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
//   position, each with a running maximum and sum, joined at the end.  It reads the cache
//   for each of them again: single tokens of 4 short chats 64 us (the next 17), of 32
//   requests of up to 8192 with 128 heads 9924 us (58.6).
//
// latent_tensor_kernel   bfloat16 over a bfloat16 cache with 512 + 64 elements a token, on
//   the tensor cores of two CTAs at a time.  A job is a request and 128 of its (token,
//   head) rows, taken as they come, so that a tile may end inside a token; a step is 128
//   positions:  S = Q [C | R]^T into tensor memory, then
//     y = S c   m' = max(m, max y)   w = 2^(y - m')   l = l 2^(m - m') + sum w
//     O = O 2^(m - m') + W C
//   m moves only when a row's maximum grows by 2^kLazy (until then w may pass 1, and O is
//   not touched).
//   A CTA has 64 of the rows: O alone is 512 columns of 32 bits a row, and for 128 rows
//   that is all of an SM's tensor memory.  With products over a pair of CTAs 64 rows run at
//   the full rate (alone they take half of it, or with .ws 0.6 to 0.8), and each CTA
//   holds half of either product's right operand: the keys of 64 of the positions, and 256
//   of the elements of all 128 as values.  (With 64 positions a step the scores take as long
//   as with 128.)  An entry comes once for each product, a third of the keys, or half of the
//   values, at a time, into buffers that the products of the tile before are just done with.
//   Four warps copy (TMA: a box is 64 elements of up to 64 tokens of a page, and issuing
//   one takes a warp a hundred cycles), one of the first CTA issues both products, four do
//   the softmax, a thread half a row's positions, and three bring the next job's queries.
//   The tiles of all jobs are dealt evenly to the pairs, so jobs are split along the
//   positions where there are few, and latent_join_kernel adds the parts in a fixed order.
//   What bounds it: with many rows the products (trees of 32 tokens of 64 heads over two
//   contexts of up to 131040, 841 GFLOP: 510 to 594 us by GPU, 1.42 to 1.65 PFLOP/s).  With
//   few, HBM and what comes before and after (single tokens of 128 heads, 32 requests of up
//   to 8192, 156 MB of entries: 59 us, of which 11 pass until the first scores, 4 with the
//   last output and 11 in the join).  While steps follow one another entries come at 6.4
//   TB/s, 0.95 of a copy (76 requests of 4096, 8192 and 16384, a job a pair: 76, 132 and 245
//   us), which would be 24 of the 59; uneven lengths and jobs' ends are the other 9.  On the way the trees took 938 us with one CTA
//   a job of 64 rows, 860 with pairs and 64 positions a step, 713 with 128, 654 without
//   prefetches into L2.

#include "latentcache.cuh"
#include "schedule.cuh"
#include "tensor.cuh"
#include "tensormap.cuh"

#include <atomic>

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

constexpr int kLatent = 512, kEntry = 576;   // of an entry, its latent part
constexpr int kChunks = kEntry / 64;         // parts of 64 elements
constexpr int kRows = 64;                    // (token, head) rows of a CTA
constexpr int kPairRows = 2 * kRows;         // of a job
constexpr int kLatentCtas = 160;             // at most
constexpr int kStep = 128;                   // positions a tile
constexpr int kChunkBytes = kRows * 128;     // 64 elements of 64 rows, or of 64 tokens
constexpr int kKeyParts = 3, kKeyBytes = 3 * kChunkBytes;      // a third of a CTA's keys of a tile
constexpr int kValueParts = 2, kValueBytes = 4 * kChunkBytes;  // half of its values: 128 elements
constexpr int kKeyAt = kChunks * kChunkBytes;  // behind the queries
constexpr int kValueAt = kKeyAt + kKeyParts * kKeyBytes;
constexpr int kWeightsAt = kValueAt + kValueParts * kValueBytes;
constexpr int kControlAt = kWeightsAt + 2 * kChunkBytes;
constexpr int kControlBytes = 3 * 1024;
constexpr int kLatentSmem = kControlAt + kControlBytes;
constexpr int kOutCol = 0, kScoreCol = 256;  // columns of tensor memory
constexpr int kLatentThreads = 384, kQueryWarp = 4, kMatrixWarp = 7, kCopyWarp = 8;
constexpr int kQueryWarps = kMatrixWarp - kQueryWarp, kCopyWarps = 4;  // of these two for keys, two for values
static_assert(kLatentThreads == 32 * (kCopyWarp + kCopyWarps), "roles");
// Of a job's begin and end, in tiles.  Single tokens of 32 requests with 0, 1, 2, 4: 63.5,
// 62.0, 58.6, 57.7 us; windows with 16 heads 63.4, 59.0, 56.6, 57.1.
constexpr int kLatentJobCost = 2;
// A split job's parts are joined by a second launch.  Where no request can have more than
// so many tiles, a job stays whole and that launch is not made.  Whole and split, us: 4
// requests of up to 256 tokens 17.3 and 23.8, of 500 17.3 and 22.8, of 1000 23.9 and 22.8;
// 64 of 256 18.1 and 26.2.
constexpr int kLatentWholeTiles = 4;
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
    q->tiles = (q->P + q->len + kStep - 1) / kStep;
    q->row_tiles = (q->len * t.a.n_q_heads + kPairRows - 1) / kPairRows;
    return true;
}

// Consecutive tiles of one job that a pair works through.
struct LatentSegment {
    LatentRequest q = {};
    int r, row_tile, first, count;
    unsigned k;  // how many the team had before it
};

// Where a team's share begins, and how many units it has.
struct LatentBegin {
    int r, group, unit, left;
    LatentRequest q;
};

// Pairs of CTAs work in teams, whose members take neighbouring row tiles over the same
// positions at the same time, so that the entries come from HBM once and from L2 to the
// others.  `size` pairs a team; this pair is the `member`-th of team `at`.
struct Team {
    int size, member, at;
};

// Walks a team's units: requests in order, in each the row tiles, a team's worth at a
// time, in each the positions.  Every warp role of both CTAs walks on its own and sees the
// same.  (What comes behind a segment is found when it is asked for, so that the first does
// not wait for the second's window.)
struct LatentWalk {
    int left, r, group, unit;
    Team team;
    unsigned k;
    bool behind;
    LatentRequest q = {};
    Window ahead;

    __device__ __forceinline__ void begin(const LatentTensorArgs &t, const LatentBegin &b, const Team &of) {
        left = b.left;
        r = b.r;
        group = b.group;
        unit = b.unit;
        q = b.q;
        team = of;
        k = 0;
        behind = false;
        ahead = load_window(t.a, min(r + 1, t.a.B - 1));
    }
    __device__ __forceinline__ bool next(const LatentTensorArgs &t, LatentSegment *s) {
        while (left > 0) {
            if (behind && ++group * team.size >= q.row_tiles) {
                group = 0;
                for (bool has = false; !has;) {  // (there are units left, so a request)
                    if (++r >= t.a.B) return false;
                    has = to_latent(t, ahead, &q, false);
                    ahead = load_window(t.a, min(r + 1, t.a.B - 1));
                }
            }
            behind = true;
            const int take = t.whole ? 1 : min(q.tiles + kLatentJobCost - unit, left);
            s->q = q;
            s->r = r;
            s->row_tile = group * team.size + team.member;
            s->k = k;
            s->first = max(unit - kLatentJobCost, 0);
            s->count = t.whole ? q.tiles : max(unit + take - kLatentJobCost, 0) - s->first;
            left -= take;
            unit = 0;
            if (s->count > 0) {
                ++k;
                if (s->row_tile < s->q.row_tiles) return true;  // (else other members' alone)
            }
        }
        return false;
    }
};

// The size of teams, and this CTA's team's share and where it begins (for all after the
// next barrier); false where none are left for it.
//   Larger teams read less from HBM and leave members idle where the row tiles are no
// multiple of them: the largest is taken whose members' steps are at most an eighth more
// than those of pairs alone.  Trees of 16 row tiles over two long contexts, pairs alone and
// in teams of four: 600 and 514 us; single tokens of one row tile stay alone (59 us).
//   (Loops are rolled up: code that runs once is fetched as slowly as it is long.)
__device__ __forceinline__ bool latent_share(const LatentTensorArgs &t, LatentBegin *begin, int4 *of_warp,
                                             Deal *deal, Team *team) {
    const AttendArgs &a = t.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x, pairs = gridDim.x / 2;
    const int per = (a.B + kLatentThreads - 1) / kLatentThreads;
    LatentRequest q = {};
    auto job = [&]() { return t.whole ? 1 : q.tiles + kLatentJobCost; };
    // units (a call has fewer than 2^31) for teams of 1, 2 and 4: a thread's, with those before
    // it in its warp, and the warps'
    int mine[3] = {}, before[3], all[3] = {};
#pragma unroll 1
    for (int i = 0, r = tid * per; i < per && r < a.B; ++i, ++r)
        if (to_latent(t, load_window(a, r), &q, cta == 0))
#pragma unroll
            for (int g = 0; g < 3; ++g) mine[g] += job() * (q.row_tiles + (1 << g) - 1 >> g);
#pragma unroll
    for (int g = 0; g < 3; ++g) before[g] = mine[g];
#pragma unroll 1
    for (int d = 1; d < 32; d <<= 1)
#pragma unroll
        for (int g = 0; g < 3; ++g) {
            const int x = __shfl_up_sync(kFullMask, before[g], d);
            if (lane >= d) before[g] += x;
        }
    if (lane == 31) of_warp[warp] = make_int4(before[0], before[1], before[2], 0);
    __syncthreads();
#pragma unroll 1
    for (int w = 0; w < kLatentThreads / 32; ++w) {
        const int4 v = of_warp[w];
        const int x[3] = {v.x, v.y, v.z};
#pragma unroll
        for (int g = 0; g < 3; ++g) {
            all[g] += x[g];
            if (w < warp) before[g] += x[g];
        }
    }
    int shift = 0, own = mine[0], to = before[0], T = all[0];
#pragma unroll
    for (int g = 1; g < 3; ++g)
        if (!t.whole && pairs >> g > 0 && all[g] * (8ll * pairs) <= all[0] * (9ll * (pairs >> g)))
            shift = g, own = mine[g], to = before[g], T = all[g];
    const int size = 1 << shift, from = to - own;
    const int n = min(pairs >> shift, t.whole ? T : (T + kLatentJobCost + 1) / (kLatentJobCost + 2));
    if (tid == 0 && !t.whole) {
        t.desc[cta * kLatentDesc] = 0;
        t.desc[cta * kLatentDesc + 7] = -1;
    }
    *team = {size, cta / 2 & size - 1, cta / 2 >> shift};
    if (team->at >= n) return false;
    const unsigned each = (unsigned)T / (unsigned)n;
    deal->n = n;
    deal->each = each;
    deal->rest = T - (int)each * n;
    const int lo = (int)deal->first(team->at), hi = (int)deal->first(team->at + 1);
    if (lo >= from && lo < to) {
        int left = lo - from;
#pragma unroll 1
        for (int r = tid * per; r < a.B; ++r) {
            if (per > 1 && !to_latent(t, load_window(a, r), &q, false)) continue;
            const int units = job() * (q.row_tiles + size - 1 >> shift);
            if (left >= units) {
                left -= units;
                continue;
            }
            begin->r = r;
            begin->group = left / job();
            begin->unit = left - begin->group * job();
            begin->left = hi - lo;
            begin->q = q;
            break;
        }
    }
    return true;
}

// Barriers that the issuing warp waits on are the first CTA's (the same place in the other
// is not used); those that it commits to are each CTA's own.
struct alignas(16) LatentControl {
    unsigned long long key_full[kKeyParts], value_full[kValueParts], p_ready[2], q_full, o_free;  // the first's
    unsigned long long key_empty[kKeyParts], value_empty[kValueParts], s_full[2], o_done[2], value_seen[2], q_empty,
        drain;
    unsigned tmem;
    unsigned nonfinite[4];  // window tokens whose values were zeroed in either CTA, by segment
    int abort;
    LatentBegin begin;
    int4 of_warp[kLatentThreads / 32];
    float top[2][2][kRows];  // [tile's parity][half of the positions]
    float sum[2][kRows];
};
static_assert(sizeof(LatentControl) <= kControlBytes && kLatentSmem <= 227 * 1024, "shared memory");

// Where the entries of rows of 64 elements lie: 16-byte piece c of row r.
__device__ __forceinline__ int chunk_piece(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kLatentThreads, 1)
latent_tensor_kernel(const __grid_constant__ CUtensorMap map, const LatentTensorArgs t) {
    extern __shared__ __align__(1024) unsigned char smem[];
    LatentControl &ctl = *reinterpret_cast<LatentControl *>(smem + kControlAt);
    const AttendArgs &a = t.a;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
    const int rank = (int)cluster_rank();
    const uint32_t base = smem_addr(smem);
    if (tid == 0) {
        for (int i = 0; i < kKeyParts; ++i) {
            mbar_init(smem_addr(&ctl.key_full[i]), 1);
            mbar_init(smem_addr(&ctl.key_empty[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_addr(&ctl.value_full[i]), 1);
            mbar_init(smem_addr(&ctl.value_empty[i]), 1);
            mbar_init(smem_addr(&ctl.p_ready[i]), 8);
            mbar_init(smem_addr(&ctl.s_full[i]), 1);
            mbar_init(smem_addr(&ctl.o_done[i]), 1);
            mbar_init(smem_addr(&ctl.value_seen[i]), 1);
        }
        mbar_init(smem_addr(&ctl.q_full), 2 * kQueryWarps);
        mbar_init(smem_addr(&ctl.o_free), 8);
        mbar_init(smem_addr(&ctl.q_empty), 1);
        mbar_init(smem_addr(&ctl.drain), 1);
        ctl.abort = 0;
        for (int i = 0; i < 4; ++i) ctl.nonfinite[i] = 0;
        fence_mbar_init();
        prefetch_map(&map);
    }
    __syncwarp();
    cluster_arrive_all();  // the barriers are there
    if (warp == kMatrixWarp) tmem_alloc_pair(smem_addr(&ctl.tmem), 512);
    pdl_wait();
    pdl_trigger();

    Deal deal;
    Team team;
    if (!latent_share(t, &ctl.begin, ctl.of_warp, &deal, &team)) {  // (neither CTA of the pair)
        if (warp == kMatrixWarp) {
            __syncwarp();
            tmem_free_pair(*(volatile unsigned *)&ctl.tmem, 512);
        }
        cluster_wait_all();
        cluster_sync();
        return;
    }
    __syncthreads();
    cluster_wait_all();
    tmem_fence_after();
    const uint32_t tmem = ctl.tmem;
    volatile int *abort = &ctl.abort;
    LatentWalk walk;
    walk.begin(t, ctl.begin, team);
    LatentSegment s = {};
    bool ok = true;
    auto wait = [&](unsigned long long *bar, unsigned parity) {
        return ok = warp_wait(ok, smem_addr(bar), parity, abort, a.status);
    };
    auto first_cta = [&](unsigned long long *bar) { return cluster_addr(smem_addr(bar), 0); };
    const int hq = a.n_q_heads;
    unsigned done = 0, seg = 0;  // tiles and segments so far

    if (warp >= kCopyWarp) {
        // ----------------------------------------------- copy warps
        // Of a tile's boxes a CTA copies half as keys and all, of its elements, as values:
        // two warps every other box of nine parts each of the keys', two one half each of
        // the values'.  The table's entries of `per` tiles are looked up at a time, a box a
        // lane, one such batch ahead.
        const int which = warp - kCopyWarp, half = which & 1;
        const bool keys = which < 2;
        const int boxes = kStep / t.box, key_boxes = boxes / 2, per = 32 / boxes;
        // boxes that this lane copies from: of keys every other one, in parts of three (one
        // box: the first warp two of the three, the second the other)
        const int split = key_boxes > 1 ? 3 : 2 - half, chunk = key_boxes > 1 ? lane % 3 : 2 * half + lane;
        const int place = key_boxes > 1 ? 2 * (lane / 3) + half : 0;
        const int box = keys ? rank * key_boxes + place : lane >> 1;
        const bool mine = keys ? key_boxes > 1 ? place < key_boxes : lane < split : box < boxes;
        const uint32_t dst = keys ? base + kKeyAt + chunk * kChunkBytes + place * t.box * 128
                                  : base + kValueAt + half * kValueBytes + (lane & 1) * 2 * kChunkBytes +
                                        box * t.box * 128;
        while (ok && walk.next(t, &s)) {
            const int n = s.q.P + s.q.len, from = s.first * kStep;
            struct Batch {
                int page, token;
            } now, next;
            auto look_up = [&](int tile) -> Batch {
                const int pos = from + tile * kStep + lane * t.box;
                const unsigned col = (unsigned)pos / (unsigned)a.cache.page_size;
                return {tile + lane / boxes < s.count && pos < n
                            ? __ldg(a.cache.table + (long long)s.r * a.cache.table_width + col)
                            : a.cache.n_pages,
                        (int)(pos - col * a.cache.page_size)};
            };
            now = look_up(0);
            next = look_up(per);
            for (int i = 0; i < s.count; ++i) {
                const int j = i % per;
                if (j == 0 && i > 0) {
                    now = next;
                    next = look_up(i + per);
                }
                int page = __shfl_sync(kFullMask, now.page, (j * boxes + box) % 32);
                const int token = __shfl_sync(kFullMask, now.token, (j * boxes + box) % 32);
                // a page outside the pool, as past the request's end, arrives as zeros
                if ((unsigned)page >= (unsigned)a.cache.n_pages) {
                    if (mine && from + i * kStep + box * t.box < n) flag(a.status, DSPARK_STATUS_BAD_INDEX);
                    page = a.cache.n_pages;
                }
                if (keys) {
#pragma unroll 1
                    for (int part = 0; part < kKeyParts; ++part) {
                        if (!wait(&ctl.key_empty[part], done + i + 1)) break;
                        if (rank == 0 && half == 0 && lane == 0)
                            mbar_expect(smem_addr(&ctl.key_full[part]), 2 * kKeyBytes);
                        __syncwarp();
                        if (mine)
                            tma_load_4d_pair(dst + part * kKeyBytes, &map, (3 * part + chunk) * 64, token, 0, page,
                                             first_cta(&ctl.key_full[part]));
                    }
                } else {
                    if (!wait(&ctl.value_empty[half], done + i + 1)) break;
                    if (rank == 0 && lane == 0) mbar_expect(smem_addr(&ctl.value_full[half]), 2 * kValueBytes);
                    __syncwarp();
                    if (mine)
                        tma_load_4d_pair(dst, &map, (4 * rank + 2 * half + (lane & 1)) * 64, token, 0, page,
                                         first_cta(&ctl.value_full[half]));
                }
                if (!ok) break;
            }
            done += s.count;
        }
        if (!ok && rank == 0 && which == 0 && lane == 0) {
            // copies still under way write the pair's buffers (each wait ends by itself; the
            // CTAs leave together)
            for (int p = 0; p < 2; ++p) {
                for (int i = 0; i < kKeyParts; ++i) mbar_wait(smem_addr(&ctl.key_full[i]), p, kWaitLimitNs / 4);
                for (int i = 0; i < kValueParts; ++i) mbar_wait(smem_addr(&ctl.value_full[i]), p, kWaitLimitNs / 4);
            }
        }
    } else if (warp == kMatrixWarp) {
        // ---------------------------------------------- matrix warp
        // Keeps step as a whole, so that addresses stay in uniform registers; one lane
        // issues.  Scores of tile i, then the output of tile i - 1, whose weights are
        // computed meanwhile.
        if (rank == 0) {
            constexpr uint32_t score_word = mma_word(true, kStep, false), value_word = mma_word(true, 256, true);
            const uint32_t ubase = __shfl_sync(kFullMask, base, 0), utmem = __shfl_sync(kFullMask, tmem, 0);
            const bool leader = elect_one();
            const uint64_t desc_q = smem_operand(ubase, 16, 128);
            const uint64_t desc_key = smem_operand(ubase + kKeyAt, 16, 128);
            const uint64_t desc_value = smem_operand(ubase + kValueAt, 2 * kChunkBytes, 128);
            const uint64_t desc_w = smem_operand(ubase + kWeightsAt, 16, 128);
            // O += W C of the segment's tile i
            auto values = [&](int i, unsigned tile) {
                const unsigned b = tile & 1;
                if (i == 0 && seg > 0 && !wait(&ctl.o_free, seg - 1)) return;
                if (!wait(&ctl.value_full[0], tile) || !wait(&ctl.value_full[1], tile)) return;
                if (lane < 2) cluster_arrive(cluster_addr(smem_addr(&ctl.value_seen[b]), lane));
                if (!wait(&ctl.p_ready[b], tile >> 1)) return;
                tmem_fence_after();
                if (leader) {
#pragma unroll 1
                    for (int h = 0; h < kValueParts; ++h) {
#pragma unroll
                        for (int k = 0; k < kStep / 16; ++k)
                            mma_pair_ss(utmem + kOutCol + 128 * h, desc_w + (k / 4 * kChunkBytes + k % 4 * 32 >> 4),
                                        desc_value + (h * kValueBytes + k * 16 * 128 >> 4), value_word, i > 0 || k > 0);
                        mma_pair_commit(smem_addr(&ctl.value_empty[h]));
                    }
                    mma_pair_commit(smem_addr(&ctl.o_done[b]));
                }
                __syncwarp();
            };
            while (ok && walk.next(t, &s)) {
                if (!wait(&ctl.q_full, seg)) break;
                const int count = __shfl_sync(kFullMask, s.count, 0);
                for (int i = 0; i < count; ++i) {
                    // (the scores of tile - 2 have been read)
                    const unsigned tile = done + i, b = tile & 1;
#pragma unroll 1
                    for (int part = 0; part < kKeyParts; ++part) {
                        if (!wait(&ctl.key_full[part], tile)) break;
                        tmem_fence_after();
                        if (leader) {
#pragma unroll
                            for (int k = 0; k < 12; ++k) {
                                const int at = 3 * part * kChunkBytes + (k / 4 * kChunkBytes + k % 4 * 32);
                                mma_pair_ss(utmem + kScoreCol + b * 64, desc_q + (at >> 4), desc_key + (at >> 4),
                                            score_word, part > 0 || k > 0);
                            }
                            mma_pair_commit(smem_addr(&ctl.key_empty[part]));
                            if (part + 1 == kKeyParts) {
                                mma_pair_commit(smem_addr(&ctl.s_full[b]));
                                if (i + 1 == count) mma_pair_commit(smem_addr(&ctl.q_empty));
                            }
                        }
                        __syncwarp();
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
            // the pair
            if (!ok && leader) {
                mma_pair_commit(smem_addr(&ctl.drain));
                mbar_wait(smem_addr(&ctl.drain), 0);
            }
            __syncwarp();
        }
    } else if (warp >= kQueryWarp) {
        // --------------------------------------------- query warps
        // A warp a row at a time, 16 bytes a lane.
        while (ok && walk.next(t, &s)) {
            if (seg > 0 && !wait(&ctl.q_empty, seg - 1)) break;
            const int rows = s.q.len * hq, first = s.row_tile * kPairRows + rank * kRows;
            int row = first + warp - kQueryWarp, token = row / hq, head = row - token * hq;
            const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + s.q.row0 * a.ld_q + 8 * lane;
            uint32_t dst = base + lane / 8 * kChunkBytes + (warp - kQueryWarp) * 128;
#pragma unroll 4
            for (int m = warp - kQueryWarp; m < kRows; m += kQueryWarps) {
                const bool there = row < rows;
                const __nv_bfloat16 *from = q + (there ? token * a.ld_q + (long long)head * kEntry : 0);
                const uint32_t at = dst + ((lane % 8 ^ (m & 7)) << 4);
                copy16(at, from, there);
                copy16(at + 4 * kChunkBytes, from + 256, there);
                if (lane < 8) copy16(at + 8 * kChunkBytes, from + 512, there);
                dst += kQueryWarps * 128;
                row += kQueryWarps;
                for (head += kQueryWarps; head >= hq; head -= hq) ++token;
            }
            copy16_wait();
            fence_async_proxy();
            __syncwarp();
            if (lane == 0) cluster_arrive(first_cta(&ctl.q_full));
            ++seg;
        }
    } else {
        // --------------------------------------------- softmax warps
        const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
        const float c = fmaxf(fabsf(a.scale) * kLog2e, 0x1p-100f);  // 0 would turn -inf into NaN
        const bool negative = a.scale < 0.0f;
        const int m = tid & 63, half = tid >> 6;  // a row, and which 64 of a tile's positions
        // The four warps meet once a tile and once behind the last: a warp that gave up comes
        // to the next such barrier, and all leave there.
        bool met = true;
        while (walk.next(t, &s)) {
            const int n = s.q.P + s.q.len, all = s.q.len * hq;
            const int row = s.row_tile * kPairRows + rank * kRows + m, safe = min(row, all - 1);
            const bool valid = row < all;
            const int token = safe / hq, head = safe % hq, packed = s.q.row0 + token;
            const unsigned bits = ancestors_of(a, packed, token, s.q.len);
            if (tid == 0) ctl.nonfinite[(seg + 2) & 3] = 0;  // the one's before the last
            float mx = -INFINITY, l = 0.0f;  // running maximum (to base 2); this half's sum
            for (int i = 0; i < s.count; ++i) {
                const unsigned tile = done + i, b = tile & 1;
                const int p0 = (s.first + i) * kStep;
                wait(&ctl.s_full[b], tile >> 1);
                tmem_fence_after();
                uint32_t x[64];
                tmem_load32(lanes + kScoreCol + 64 * b, x);
                tmem_load32(lanes + kScoreCol + 64 * b + 32, x + 32);
                tmem_wait_load(x);
                tmem_wait_load(x + 32);
                if (negative) {
#pragma unroll
                    for (int j = 0; j < 64; ++j) x[j] ^= 0x80000000u;
                }
                if (p0 + kStep > s.q.P) {
                    // prefix positions, then the row's ancestors in the window
                    const int pre = s.q.P - (p0 + 64 * half);
                    const unsigned long long w = pre >= 0 ? bits : pre > -32 ? bits >> -pre : 0;
                    const unsigned long long sees = pre >= 64 ? ~0ull : pre > 0 ? w << pre | ((1ull << pre) - 1) : w;
#pragma unroll
                    for (int j = 0; j < 64; ++j)
                        if (!(sees >> j & 1)) x[j] = 0xFF800000u;
                }
                float part[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    part[j] = fmaxf(__uint_as_float(x[j]), __uint_as_float(x[j + 4]));
#pragma unroll
                    for (int k = 8 + j; k < 64; k += 4) part[j] = fmaxf(part[j], __uint_as_float(x[k]));
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
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    const float2 y = fma2(make_float2(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])),
                                          make_float2(c, c), make_float2(-shift, -shift));
                    const float2 u = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                    sum[j & 1] = add2(sum[j & 1], u);
                    // (bfloat16, 8 digits, as the latent vectors are: a product takes operands
                    // of one type.  The sum keeps all digits, for lse)
                    const __nv_bfloat162 two = __floats2bfloat162_rn(u.x, u.y);
                    x[j] = *reinterpret_cast<const uint32_t *>(&two);
                }
                // in the place of the last tile's, once they are multiplied
                if (i > 0 && !wait(&ctl.o_done[(tile - 1) & 1], (tile - 1) >> 1)) continue;
                unsigned char *weights = smem + kWeightsAt + half * kChunkBytes;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<uint4 *>(weights + chunk_piece(m, j)) =
                        make_uint4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
                l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
                if (p0 + kStep > s.q.P) {
                    // Latent vectors past the request's end become zeros, and so do NaN and
                    // infinities of the window (0 x NaN would reach rows that do not see
                    // them); the rows that do get NaN at the end.  Each CTA does so for the
                    // elements that it holds as values.
                    if (!wait(&ctl.value_seen[b], tile >> 1)) continue;
                    const int from = max(s.q.P, p0);
                    for (int j = tid; j < (p0 + kStep - from) * 32; j += 128) {
                        const int pos = from + j / 32, piece = j % 32;
                        uint4 *at = reinterpret_cast<uint4 *>(smem + kValueAt + piece / 8 * 2 * kChunkBytes +
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
                            for (int k = 0; k < 2; ++k)
                                cluster_or(cluster_addr(smem_addr(&ctl.nonfinite[seg & 3]), k),
                                           1u << (pos - s.q.P));
                        }
                        *at = v;
                    }
                    cluster_fence();  // (the noted tokens)
                }
                fence_async_proxy();
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) cluster_arrive(first_cta(&ctl.p_ready[b]));
            }
            if (!met) break;
            const unsigned last = done + s.count - 1;
            wait(&ctl.o_done[last & 1], last >> 1);
            done += s.count;
            tmem_fence_after();
            if ((s.first + s.count) * kStep > s.q.P) cluster_fence();
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
                const int e = 256 * half + d;  // the upper lanes hold the second CTA's elements
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
                        // (an infinite element is a part of the key too, so that the score is
                        // infinite or NaN and the weight 0 or NaN: either makes the product NaN)
                        const float y = elem_value(v[j]);
                        if (!(y - y == 0.0f)) o[j] = __float_as_uint(NAN);
                    }
                }
                if (!whole) {
                    float4 *part = reinterpret_cast<float4 *>(t.part_o) + ((long long)slot * 128 + e / 4) * kRows + m;
                    if (valid)
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
            if (lane == 0) cluster_arrive(first_cta(&ctl.o_free));
            if (half == 0 && valid) {
                if (!whole) {
                    t.part_ml[(long long)slot * 2 * kRows + m] = mx;
                    t.part_ml[((long long)slot * 2 + 1) * kRows + m] = l;
                } else if (a.lse) {
                    a.lse[(long long)packed * hq + head] = l == 0.0f ? -INFINITY : shift * kLn2 + logf(l);
                }
            }
            if (tid == 0 && !whole) {
                // what the join is told: of a job that begins here and ends in a later team, or
                // of the one that the whole of this team's share lies in
                auto same = [&](int at) { return (at * team.size + team.member) * 2 + rank; };  // in a team
                int *d = t.desc + cta * kLatentDesc;
                if (s.first == 0) {
                    const long long hi = deal.first(team.at + 1);
                    d[1] = same(deal.cta_of(hi - 1 + s.q.tiles - s.count, team.at));
                    d[2] = slot;
                    d[3] = s.q.row0;
                    d[4] = s.row_tile * kPairRows + rank * kRows;
                    d[5] = min(all - d[4], kRows);
                    d[6] = 31 - __clz(2 * team.size);
                    d[0] = 1;
                } else if (s.k == 0 && s.first + s.count < s.q.tiles) {
                    // (where its first tile is)
                    d[7] = same(deal.cta_of(deal.first(team.at) - s.first, 0));
                }
            }
            ++seg;
        }
    }
    __syncthreads();
    cluster_sync();  // the other CTA may arrive on, or multiply from, what is here
    if (warp == kMatrixWarp) tmem_free_pair(tmem, 512);
}

// Joins the parts of the jobs that several CTAs share, in the CTAs' order: a block for
// each of these CTAs but the last takes its share of the rows' fours of elements.  A thread
// keeps to a row, and a block's groups of kRows threads take fours in turn, or where there
// are many parts one four and the parts in turn.  Instructions that run once and L2 bound
// it: of the 11 us that it adds to single tokens of 32 requests (107 parts of 256 KB) 4 are
// the launch's, 3.5 the code's without parts.  Blocks a CTA, 4, 8 and 16: 65, 61 and 64 us.
constexpr int kJoinThreads = 256, kJoinGroups = kJoinThreads / kRows, kJoinPieces = 8;
constexpr int kJoinFew = 8;  // parts that a thread adds alone

__global__ void __launch_bounds__(kJoinThreads) latent_join_kernel(const LatentTensorArgs t) {
    __shared__ float factor[kLatentCtas / 2][kRows];  // of a part (a pair has one of a job)
    __shared__ float2 of_group[kJoinGroups][kRows];
    __shared__ float4 sum[kJoinThreads];
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
    const int rows = d1.y, by = d1.z, n = (d0.y - c0 >> by) + 1;  // parts, of every 2^by-th CTA
    if (rows <= 0) return;
    constexpr int kFours = kLatent / 4;
    const int pieces = max(n - 1, 1) * kJoinPieces, piece = ((int)blockIdx.x - c0 >> by) * kJoinPieces + blockIdx.y;
    const int each = (kFours + pieces - 1) / pieces, begin = piece * each, end = min(begin + each, kFours);
    if (begin >= end) return;
    const int tid = threadIdx.x, m = tid % kRows, group = tid / kRows;
    const int deals = n > kJoinFew ? kJoinGroups : 1, deal = group % deals, step = kJoinGroups / deals;
    auto slot = [&](int i) { return (long long)(i == 0 ? d0.z : 2 * (c0 + (i << by))); };
    auto part = [&](int i, int four) {
        return __ldcg(reinterpret_cast<const float4 *>(t.part_o) + (slot(i) * kFours + four) * kRows + m);
    };
    auto add = [](float4 &x, float f, float4 y) {
        x.x = fmaf(f, y.x, x.x), x.y = fmaf(f, y.y, x.y), x.z = fmaf(f, y.z, x.z), x.w = fmaf(f, y.w, x.w);
    };
    auto in = [&](int four) { return four < end && m < rows; };
    // the row's maximum and sum, and each part's factor
    float top = -INFINITY, l = 0.0f;
    if (m < rows)
        for (int i = group; i < n; i += kJoinGroups) {
            const float *ml = t.part_ml + slot(i) * 2 * kRows + m;
            const float pm = __ldcg(ml), pl = __ldcg(ml + kRows), higher = fmaxf(top, pm);
            const float base = higher == -INFINITY ? 0.0f : higher;
            l = l * exp2_approx(top - base) + pl * exp2_approx(pm - base);
            top = higher;
            factor[i][m] = pm;
        }
    of_group[group][m] = make_float2(top, l);
    __syncthreads();
    top = -INFINITY, l = 0.0f;
#pragma unroll
    for (int i = 0; i < kJoinGroups; ++i) top = fmaxf(top, of_group[i][m].x);
    const float shift = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int i = 0; i < kJoinGroups; ++i) l = fmaf(exp2_approx(of_group[i][m].x - shift), of_group[i][m].y, l);
    if (m < rows)
        for (int i = group; i < n; i += kJoinGroups) factor[i][m] = exp2_approx(factor[i][m] - shift);
    __syncthreads();
    const int hq = t.a.n_q_heads, row = d1.x + m, head = row % hq;
    const long long packed = d0.w + row / hq;
    __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(t.a.out) + packed * t.a.ld_out + (long long)head * kLatent;
    const float inv = 1.0f / l;
    for (int four = begin + group / deals, at = begin; at < end; at += step, four += step) {
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (in(four))
#pragma unroll 4
            for (int i = deal; i < n; i += deals) add(x, factor[i][m], part(i, four));
        if (deals > 1) {
            sum[tid] = x;
            __syncthreads();
            if (deal == 0)
#pragma unroll
                for (int i = 1; i < kJoinGroups; ++i) add(x, 1.0f, sum[tid + i * kRows]);
            __syncthreads();
        }
        if (deal > 0 || !in(four)) continue;
        if (l == 0.0f) x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        else x.x *= inv, x.y *= inv, x.z *= inv, x.w *= inv;
        const __nv_bfloat162 u = __floats2bfloat162_rn(x.x, x.y), v = __floats2bfloat162_rn(x.z, x.w);
        *reinterpret_cast<uint2 *>(out + four * 4) =
            make_uint2(*reinterpret_cast<const uint32_t *>(&u), *reinterpret_cast<const uint32_t *>(&v));
        if (t.a.lse && four == 0) t.a.lse[packed * hq + head] = l == 0.0f ? -INFINITY : shift * kLn2 + logf(l);
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
           // (the dealing counts tiles of 128 positions and 128 rows in 31 bits)
           ((long long)c.table_width * c.page_size / kStep + kLatentJobCost + 1) *
                   ((long long)DSPARK_MAX_WINDOW * a.n_q_heads / kPairRows + 1) * a.B < (1ll << 31);
}

// How many pairs of CTAs run at a time on the current device (they sit in one cluster of
// SMs each, so an odd SM of those is left), looked up once.
int pair_count() {
    static std::atomic<int> kept[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
    if ((n = kept[dev].load(std::memory_order_relaxed)) > 0) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kLatentCtas);
    cfg.blockDim = dim3(kLatentThreads);
    cfg.dynamicSmemBytes = kLatentSmem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {2, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&n, latent_tensor_kernel, &cfg) != cudaSuccess || n < 1) return 1;
    n = min(n, kLatentCtas / 2);
    kept[dev].store(n, std::memory_order_relaxed);
    return n;
}

cudaError_t launch_latent_tensor(const AttendArgs &a, const dspark_latent_cache &c, void *workspace,
                                 cudaStream_t stream) {
    LatentTensorArgs t;
    t.a = a;
    t.box = gcd(c.page_size, kStep / 2);
    t.whole = (long long)c.table_width * c.page_size <= kLatentWholeTiles * kStep;
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
    const int grid = 2 * pair_count();
    e = launch_pdl(latent_tensor_kernel, dim3(grid), dim3(kLatentThreads), kLatentSmem, stream, map, t);
    if (e != cudaSuccess || t.whole) return e;
    return launch_pdl(latent_join_kernel, dim3(grid, kJoinPieces), dim3(kJoinThreads), 0, stream, t);
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
    if (rows_overlap(q, ld_q * e_bytes, width * e_bytes, max_rows, out, ld_out * e_bytes, width_out * e_bytes,
                     max_rows))
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
