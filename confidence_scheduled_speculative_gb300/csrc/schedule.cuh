// schedule.cuh -- how attend.cu and fewrows.cuh share a call's work: the window as
// the device finds it, and its jobs dealt to the CTAs in tiles of positions.
#pragma once

#include "kvcache.cuh"

namespace dspark {

struct AttendArgs {
    const void *q;
    long long ld_q;
    void *out;
    long long ld_out;
    float *lse;
    const int32_t *cu, *prefix;
    const uint32_t *ancestors;
    int B, n_q_heads, max_rows;
    float scale;
    KvView cache;
    int32_t *status;
};

// A request's entries as they are: rows [lo, hi) and the prefix length.
struct Window {
    int lo, hi, P;
};

__device__ __forceinline__ Window load_window(const AttendArgs &a, int r) {
    return {__ldg(a.cu + r), __ldg(a.cu + r + 1), __ldg(a.prefix + r)};
}

// A request's last position is below this: the kernels count positions in 32 bits and
// step past the end, by at most 32 steps of 128 (the few-row kernel's look ahead).
constexpr long long kMaxPositions = (1ll << 31) - 8192;

// Whether a window has rows and can be used; with `report`, flags why not.
__device__ __forceinline__ bool usable(const AttendArgs &a, const Window &w, bool report) {
    if (w.hi == w.lo) return false;
    int bad = 0;
    if (w.lo < 0 || w.hi < w.lo || w.hi - w.lo > DSPARK_MAX_WINDOW || w.hi > a.max_rows)
        bad = DSPARK_STATUS_BAD_LEN;
    else if (w.P < 0 || (long long)w.P + (w.hi - w.lo) >
                            min((long long)a.cache.table_width * a.cache.page_size, kMaxPositions))
        bad = DSPARK_STATUS_BAD_INDEX;
    if (bad && report) flag(a.status, bad);
    return !bad;
}

constexpr int kFewRows = 8;  // query rows of a kv head that fewrows.cuh multiplies at once

// The window tokens that token i of a window sees, as bits.
__device__ __forceinline__ unsigned ancestors_of(const AttendArgs &a, int row, int i, int len) {
    const unsigned all = 0xFFFFFFFFu >> (32 - len);
    return (a.ancestors ? __ldg(a.ancestors + row) : 0xFFFFFFFFu >> (31 - i)) & all;
}

constexpr int kTile = 64;           // positions a step
constexpr int kRowsPerTile = 128;   // (token, query head) rows of one kv head
constexpr int kMaxCtas = 320;       // two for each of up to 160 SMs
constexpr int kTmemCols = 256;      // two score tiles of 64, the output's up to 128
constexpr float kLazy = 8.0f;       // log2 of how far weights may grow past 1
// Weights as halves (over E4M3) are taken 2^kHalfRoom times larger, so that those far
// below the largest keep their digits: with 2^kLazy in front a half still holds them.
constexpr float kHalfRoom = 6.0f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kDescInts = 8;  // of a split job, for the join
// The most tiles of a request for which jobs stay whole and the joining launch is not
// made.  Whole and split: 8 requests of up to 300 tokens 13 and 21 us, of 440 15 and 21,
// of 900 21 and 23, of 1900 32 and 25; 200 requests of 300 52 and 49, of 900 92 and 74.
constexpr int kWholeTiles = 8;

struct TensorArgs {
    AttendArgs a;
    int group;   // query heads a kv head
    int tokens;  // window tokens a row tile: all their heads in 128 rows
    int few;     // window tokens whose heads fit in 64 rows
    int box;     // cache tokens a TMA box
    int whole;   // no job is split
    int choose;  // both kernels are launched: either finds out which of them works (few_dearer)
    float *part_o;   // [2 kMaxCtas][D / 4][128] float4
    float *part_ml;  // [2 kMaxCtas][2][128]
    int *desc;       // [kMaxCtas][kDescInts]: the split job that begins in a CTA
};

// A request's jobs: every (kv head, 128 rows) pair reads all its tiles.
struct Request {
    int row0, len, P, tiles, row_tiles;
};

__device__ __forceinline__ bool to_request(const TensorArgs &t, const Window &w, Request *q, bool report) {
    if (!usable(t.a, w, report)) return false;
    q->row0 = w.lo;
    q->len = w.hi - w.lo;
    q->P = w.P;
    q->tiles = (q->P + q->len + kTile - 1) / kTile;
    q->row_tiles = (q->len + t.tokens - 1) / t.tokens;
    return true;
}

// How much dearer, over E4M3, a request is to fewrows.cuh's kernel than to the one of 128
// rows; the kernel for which the requests' sum is less does the call.  It goes by each
// request's own length and rows, so that neither empty windows nor short requests beside
// a long one count for more than they take.  A pass of eight rows takes 4/7 of one of 128,
// and a job's begin and end cost the latter some tiles more.  There and in the kernel of
// 128 rows a tile, each launched alone, us (4 heads a kv head, 8 kv heads of 128):
//   32 requests of up to 8192 tokens, 1 to 2 tokens each 74 and 113, 3 or 4 (two passes)
//   119 and 113, 5 172 and 116, 1 to 5 108 and 113, 1 to 6 117 and 114;  of 800, 3 or 4
//   tokens 41 and 45, 6 55 and 46;  of 300, 4 tokens 21 and 18;  2 of 8192, 4 tokens 29
//   and 27, 6 35 and 27;  256 of 1000, 2 tokens 137 and 240, 4 255 and 242, 6 374 and 249
//   one token over 131040 72 and 79;  8 of 32 with 8 tokens, the others without, 116 and
//   56;  8 heads a kv head: 2 of 64 with 32 tokens, the others without, 206 and 52; one of
//   32 tokens over 100000 beside 63 single tokens 1129 and 199
//   2 kv heads, 32 requests, 1 token 31 and 43, 4 44 and 43;  heads of 64, 1 token 48 and
//   81, 4 82 and 81, 6 117 and 86
// Finding out costs the one that does the call 1 to 4 us.
__device__ __forceinline__ long long few_dearer(const TensorArgs &t, const Request &q) {
    const int few = kFewRows / t.group, all = kRowsPerTile / t.group;  // window tokens a pass
    return 4ll * q.tiles * ((q.len + few - 1) / few) - (7ll * q.tiles + 24) * ((q.len + all - 1) / all);
}

// Where a CTA's share begins.
struct Begin {
    int r, head, row_tile, unit;
    Request q;
};

// T units dealt to n CTAs in order, each T / n of them or one more.  A job counts
// its tiles and, before them, some units for its beginning and end, so that CTAs
// with many short jobs get fewer tiles; where no job is split it is one unit.
struct Deal {
    int n, rest;  // below 1024
    long long each;
    __device__ __forceinline__ long long first(int c) const { return c * each + c * rest / n; }
    // the CTA, c or later, that a unit falls to
    __device__ __forceinline__ int cta_of(long long unit, int c) const {
        int hi = n - 1;
        while (c < hi) {
            const int mid = (c + hi + 1) >> 1;
            if (first(mid) <= unit) c = mid;
            else hi = mid - 1;
        }
        return c;
    }
};

// Consecutive tiles of one job that a CTA works through.
struct Segment {
    Request q = {};
    int r, head, row_tile, first, count;
};

// Walks a CTA's units job by job: requests in order, in each the kv heads, in
// each the row tiles (which read the same keys and values at about the same time: of
// 276 MB that the second tiles of a long tree read, L2 had two thirds).  Every warp role walks on its own and sees the same; the
// next request is loaded while the present one is worked on.
template <int kJobCost>
struct Walk {
    int left, r, head, row_tile, unit;
    Request q = {};
    Window ahead;

    __device__ __forceinline__ void begin(const TensorArgs &t, const Begin &b, int n) {
        left = n;
        r = b.r;
        head = b.head;
        row_tile = b.row_tile;
        unit = b.unit;
        q = b.q;
        ahead = load_window(t.a, min(r + 1, t.a.B - 1));
    }
    __device__ __forceinline__ bool next(const TensorArgs &t, Segment *s) {
        while (left > 0) {
            const int take = t.whole ? 1 : min(q.tiles + kJobCost - unit, left);
            s->q = q;
            s->r = r;
            s->head = head;
            s->row_tile = row_tile;
            s->first = max(unit - kJobCost, 0);
            s->count = t.whole ? q.tiles : max(unit + take - kJobCost, 0) - s->first;
            left -= take;
            unit = 0;
            if (++row_tile == q.row_tiles) {
                row_tile = 0;
                if (++head == t.a.cache.n_kv_heads) {
                    head = 0;
                    while (left > 0) {
                        const bool has = to_request(t, ahead, &q, false);
                        ++r;
                        ahead = load_window(t.a, min(r + 1, t.a.B - 1));
                        if (has) break;
                    }
                }
            }
            if (s->count > 0) return true;
        }
        return false;
    }
};

// This CTA's units [lo, hi) of all of them, and where they begin (for all after the
// next barrier); false where none are left for it.  Each thread sums a run of
// requests, and a scan over the threads finds the request that holds the first.
// kFew: of fewrows.cuh, which has none if the other kernel does the call.
template <int kThreads, int kJobCost, bool kFew>
__device__ __forceinline__ bool share_of(const TensorArgs &t, Begin *begin, long long *scan, Deal *deal,
                                         long long *lo, long long *hi) {
    const AttendArgs &a = t.a;
    const int tid = threadIdx.x, cta = blockIdx.x;
    const int per = (a.B + kThreads - 1) / kThreads;
    long long mine = 0, dearer = 0;
    Request q = {};
    auto job_units = [&]() { return t.whole ? 1 : q.tiles + kJobCost; };
    auto units = [&]() { return (long long)job_units() * (q.row_tiles * a.cache.n_kv_heads); };
    for (int i = 0, r = tid * per; i < per && r < a.B; ++i, ++r)
        if (to_request(t, load_window(a, r), &q, cta == 0)) {
            mine += units();
            if (kFew) dearer += few_dearer(t, q);
        }
    if (kFew && t.choose && block_sum<long long>(dearer, scan) > 0) return false;
    long long T;
    const long long before = block_exclusive_scan<long long>(mine, scan, &T);
    // (a CTA with less than two tiles to do would cost more than it brings)
    const int n_ctas =
        (int)min((long long)gridDim.x, t.whole ? T : (T + kJobCost + 1) / (kJobCost + 2));
    if (tid == 0 && !t.whole) {
        t.desc[cta * kDescInts] = 0;
        t.desc[cta * kDescInts + 7] = -1;
    }
    if (cta >= n_ctas) return false;
    deal->n = n_ctas;
    deal->each = div_nonneg(T, n_ctas);
    deal->rest = (int)(T - deal->each * n_ctas);
    *lo = deal->first(cta);
    *hi = deal->first(cta + 1);
    if (*lo >= before && *lo < before + mine) {
        long long at = before;
        for (int r = tid * per;; ++r) {
            // (with one request a thread it is the one just loaded)
            if (per > 1 && !to_request(t, load_window(a, r), &q, false)) continue;
            if (*lo >= at + units()) {
                at += units();
                continue;
            }
            const int job = (int)div_nonneg(*lo - at, job_units());
            begin->r = r;
            begin->unit = (int)(*lo - at - (long long)job * job_units());
            begin->head = job / q.row_tiles;
            begin->row_tile = job % q.row_tiles;
            begin->q = q;
            break;
        }
    }
    return true;
}

// Tells the join, after a CTA's last segment s (its k-th) that is not a whole job, of
// the job that begins here and ends in a later CTA, or of the one that the whole of
// this CTA lies in.
__device__ __forceinline__ void note_split(const TensorArgs &t, const Segment &s, const Deal &deal,
                                           long long lo, long long hi, unsigned k, int token0, int rows) {
    const int cta = blockIdx.x;
    int *d = t.desc + cta * kDescInts;
    if (s.first == 0) {
        // (its last tile comes q.tiles - count units after the CTA's last)
        d[1] = deal.cta_of(hi - 1 + s.q.tiles - s.count, cta);
        d[2] = 2 * cta + (k > 0);
        d[3] = s.q.row0;
        d[4] = s.head;
        d[5] = token0;
        d[6] = rows;
        d[0] = 1;
    } else if (k == 0 && s.first + s.count < s.q.tiles) {
        d[7] = deal.cta_of(lo - s.first, 0);  // where its first tile is
    }
}

}  // namespace dspark
