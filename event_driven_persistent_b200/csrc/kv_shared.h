// Paged key-value cache: parameter blocks and the index arithmetic that the
// kernels and the host (and a host-side test) share.
#pragma once
#include <stdint.h>

#ifdef __CUDACC__
#define KV_HD __host__ __device__ __forceinline__
#else
#define KV_HD inline
struct float2;
#endif

namespace et {

enum { KV_BF16 = 0, KV_FP16 = 1, KV_E4M3 = 2 };

constexpr int kKvMaxB = 1024;      // requests a run (their tile counts are scanned in shared memory)
constexpr int kKvMaxSplits = 2;    // partial results a team can leave: of its first and its last segment
constexpr int kKvAttnWarps = 4;
constexpr int kKvJoin = 16;        // parts that are joined at a time
constexpr int kKvShareLog = 2;     // log2 of the tiles that a team takes at least
constexpr int kKvWarpParts = 3;    // teams are warps while no segment has more than this many of their shares
constexpr int kKvWarpExtra = 1;    // numbers before a segment's tiles: for teams of a warp, and of a CTA,
KV_HD constexpr int kv_cta_extra(int row_bytes) { return row_bytes >= 512 ? 6 : 12; }  // about 2 us of its share of the bandwidth (tiles of 16 KB, else 8)
// Query heads of one unit: two n = 8 tensor-core tiles.  Over 256 dims in e4m3 one: two need more registers than a warp
// has (340 bytes spilled), and to read a KV head twice is faster where there are many ends or joins, slower over long rows.
// 64 / 4 heads, units of 16 and of 8: 32 x 512..4096 82 and 60 us, 128 x 2048 229 and 197, 1 x 60000 76 and 63, 8 x 30000
// 152 and 157 (held for seconds, at the power limit's clocks, 152 and 180).  With twice the bytes to read again, in bf16, it
// is slower: 8 x 30000 245 and 304.
KV_HD constexpr int kv_unit_heads(int hd, bool e4m3) { return hd == 256 && e4m3 ? 8 : 16; }

// Where the error of a run is kept; the first one stays until it is collected.
struct KvCtl {
    int status;
    int diag[8];
    int* host_status;        // mapped host word the status is mirrored into
    unsigned evict_run;      // number of the current eviction (tags the page owners)
    unsigned evict_done;     // CTAs of the eviction's selection that are done
};
// diag[0] of a KvCtl: what was out of range
enum { KV_BAD_LEN = 1, KV_BAD_PAGE = 2, KV_BAD_REQ = 3, KV_BAD_SLOT = 4, KV_BAD_DST = 5, KV_BAD_WEIGHT = 6 };

// The pages: element (page, head, slot, d) of K and V lies at
// page * page_stride + head * head_stride + slot * slot_stride + d (elements).
struct KvPool {
    void* K;
    void* V;
    const float* k_scale;
    const float* v_scale;
    float* acc;              // fp32 [n_pages, n_kv, page_size]
    long long page_stride, head_stride, slot_stride;
    int n_pages, page_size, n_kv;
};

struct KvTable {
    const int* pages;        // int32 [B, ld]
    long long ld;
    int max_len;             // min(max_ctx, ld * page_size): the longest a request can be
};

// ------------------------------------------------- split of the attention ----
// The tiles of all (request, unit) segments are numbered request-major, then
// unit, then tile, a few numbers left out before each segment's first; a unit is
// a KV head (or 16 or 8 query heads of one).  Team c of C (a warp or a CTA) takes numbers [floor(c N / C), floor((c + 1) N / C)): equal shares
// whatever the lengths, at most two segments of which are shared with others.
KV_HD long long kv_share_div(long long a, long long b) {  // 32 bits where they do: a 64-bit division is a long call
    return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}
// q = N / C, r = N % C: floor(c N / C) = c q + floor(c r / C)
KV_HD long long kv_share_begin(int c, long long N, int C, long long q) { return c * q + kv_share_div(c * (N - q * C), C); }
KV_HD long long kv_share_begin(long long c, long long N, long long C) { return kv_share_begin((int)c, N, (int)C, kv_share_div(N, C)); }
// the team that owns tile t
KV_HD long long kv_share_owner(long long t, long long N, long long C) { return kv_share_div((t + 1) * C - 1, N); }
// teams that share N tiles: none gets less than 2^share_log unless there is only one
KV_HD int kv_share_teams(long long N, int most, int share_log) {
    const long long c = N >> share_log;
    return (int)(c < 1 ? 1 : (c < most ? c : most));
}
// Which of its two partial slots team c uses for the segment whose tiles begin
// at number s0: the first segment of a team's run uses slot 0, another one slot 1.
KV_HD int kv_share_slot(long long c, long long s0, long long N, long long C) {
    return s0 <= kv_share_begin(c, N, C) ? 0 : 1;
}

// How a run's tiles are shared out: teams of one warp each (solo) or of a CTA each, C of them, that share N numbers, of
// which `extra` before each segment's tiles stand for what its end costs (its join and the next one's start).
struct KvTeams {
    bool solo;
    int extra, C;
    long long N;
};
// tiles: of the n_live requests that have any, one KV head each; longest: the most of one
KV_HD KvTeams kv_choose_teams(int tiles, int n_live, int longest, int units, int grid, int warps, int warp_share_log, int cta_share_log,
                              int warp_extra, int cta_extra, int warp_parts) {
    KvTeams t;
    const long long n1 = (long long)(tiles + n_live * warp_extra) * units;
    const int C1 = kv_share_teams(n1, grid * warps, warp_share_log);
    t.solo = (long long)(longest + warp_extra) * C1 <= (long long)warp_parts * n1;
    t.extra = t.solo ? warp_extra : cta_extra;
    t.N = t.solo ? n1 : (long long)(tiles + n_live * t.extra) * units;
    t.C = t.solo ? C1 : kv_share_teams(t.N, grid, cta_share_log);
    // requests of one length: whole teams a segment, if few idle for it (a team with two segments takes twice as
    // long in a small run: 1 x 517 11 -> 8 us)
    const int segs = n_live * units;
    if (t.N == (long long)(longest + t.extra) * segs && t.C >= segs && t.C % segs * 8 <= t.C) t.C -= t.C % segs;
    return t;
}

// An upper bound of the numbers that one team takes, for a handle's longest possible run: a team counts its own in 32 bits.
KV_HD long long kv_longest_run(int max_B, int max_ctx, int units, int n_sm) {
    const long long N = (long long)max_B * ((max_ctx + 15) / 16 + 12) * units;  // tiles have 16 keys or more
    return N / n_sm / 7 * 8 + 8;  // one CTA an SM at least, of which an eighth may idle
}

// largest i < live with (pre[i] + i extra) units <= t: the request of numbered tile t
KV_HD int kv_find_request(const int* pre, int live, int extra, int units, long long t) {
    int lo = 0, hi = live;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((long long)(pre[mid] + mid * extra) * units <= t) lo = mid; else hi = mid;
    }
    return lo;
}
// A segment, and its tiles counted from the first number of the team's run.
struct KvWalk {
    int i, u, nt;         // request (in the list of those that have tiles), unit, tiles of the segment
    int s0, s1;           // [s0, s1): the segment's tiles
};
// the segment whose tiles, or the `extra` numbers before them, hold number t0
KV_HD void kv_walk_to(KvWalk& w, const int* pre, int live, int extra, int units, long long t0) {
    w.i = kv_find_request(pre, live, extra, units, t0);
    w.nt = pre[w.i + 1] - pre[w.i];
    const int r = (int)(t0 - (long long)(pre[w.i] + w.i * extra) * units);
    w.u = r / (w.nt + extra);
    w.s0 = w.u * (w.nt + extra) + extra - r;
    w.s1 = w.s0 + w.nt;
}
// the next one; past the last segment it lies beyond every run
KV_HD void kv_walk_next(KvWalk& w, const int* pre, int live, int extra, int units) {
    w.s0 = w.s1 + extra;
    if (++w.u == units) {
        w.u = 0;
        if (++w.i == live) {
            w.s0 = 0x7FFFFFF0;
            w.nt = 0;
        } else {
            w.nt = pre[w.i + 1] - pre[w.i];
        }
    }
    w.s1 = w.s0 + w.nt;
}

// The parts of a shared segment: who leaves them, and where.
struct KvParts {
    int c0, n;            // the first team, how many
    int first;            // which of its slots the first one uses; the others use slot 0
};
KV_HD KvParts kv_parts(long long s0, long long s1, long long N, int C) {  // [s0, s1): the segment's tiles, by number
    KvParts p;
    p.c0 = (int)kv_share_owner(s0, N, C);
    p.n = (int)kv_share_owner(s1 - 1, N, C) - p.c0 + 1;
    p.first = kv_share_slot(p.c0, s0, N, C);
    return p;
}
KV_HD long long kv_part_slot(const KvParts& p, int k) { return (long long)(p.c0 + k) * kKvMaxSplits + (k == 0 ? p.first : 0); }
// The join of a group of kKvJoin parts lies past the slots of the grid's CTAs, by the slot of the team that made it (a CTA may
// do so for two segments).
KV_HD long long kv_group_slot(int grid, long long slot) { return (long long)grid * kKvMaxSplits + slot; }
KV_HD int kv_join_groups(int n_parts) { return (n_parts + kKvJoin - 1) / kKvJoin; }
// what a handle allocates: slots, and events a segment (its own, then its groups')
KV_HD long long kv_part_slots(int n_sm) { return 2ll * n_sm * kKvAttnWarps * kKvMaxSplits; }  // two CTAs an SM at most
KV_HD int kv_arrivals(int n_sm) { return 1 + kv_join_groups(2 * n_sm); }

// A length that can be used, or -1.
KV_HD int kv_checked_len(int len, int max_len) { return len >= 0 && len <= max_len ? len : -1; }
// Element offset of a slot's row (head 0) in the pools, or -1 for a page
// number outside the pool.
KV_HD long long kv_row_offset(int page, int in_page, const KvPool& p) {
    if (page < 0 || page >= p.n_pages) return -1;
    return (long long)page * p.page_stride + (long long)in_page * p.slot_stride;
}

// Order of accumulated weights: larger key = larger weight; -0 equals +0, a
// NaN counts as the largest.
KV_HD uint32_t kv_weight_key(uint32_t bits) {
    if ((bits & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
    if (bits == 0x80000000u) bits = 0;
    return (bits & 0x80000000u) ? ~bits : bits | 0x80000000u;
}

// The search of an eviction's border key: a pass counts the keys of [lo, hi] in at most 2^log_bins bins of 2^shift keys,
// the first one from lo on, and the next pass takes the bin that the border lies in.
KV_HD int kv_border_shift(uint32_t range, int log_bins) {  // range: hi - lo
    int bits = 0;
#ifdef __CUDA_ARCH__
    bits = 32 - __clz((int)range);
#else
    while (bits < 32 && range >> bits) ++bits;
#endif
    return bits > log_bins ? bits - log_bins : 0;
}
// passes that a search takes at most: each leaves log_bins bits fewer
KV_HD constexpr int kv_border_passes(int log_bins) { return (32 + log_bins - 1) / log_bins; }
// the last key of the bin that begins at lo, of [lo, hi]: bins begin at any key, so the top one may pass 32 bits (a NaN's
// key is the last there is), and only the distance from lo can be compared
KV_HD uint32_t kv_border_end(uint32_t lo, uint32_t hi, int shift) {
    const uint32_t step = (1u << shift) - 1;
    return lo + (hi - lo < step ? hi - lo : step);
}

struct KvAppendParams {
    KvPool pool;
    KvTable table;
    KvCtl* ctl;
    const double* turns;     // [hd / 2] rotary frequency / (2 pi)
    const void *q, *k, *v;
    void* q_out;
    long long ldq, ldk, ldv, ldqo;  // elements from one token to the next
    const void *gq, *gk;
    const int *req, *slots, *pos;
    float eps;
    int N, B, n_q, n_kv;
};

struct KvAttnParams {
    KvPool pool;
    KvTable table;
    KvCtl* ctl;
    const int* lens;
    const void* q;
    void* out;
    float* lse;
    long long ldq, ldo;
    float scale_log2;        // softmax scale * log2(e)
    int B, n_q, n_kv, group, n_qt;  // n_qt: units a KV head
    unsigned page_groups;    // groups of eight rows a page holds, 0 if page_size is no multiple of 8
    unsigned page_magic;     // i / page_groups = (i * page_magic) >> 32 for the groups that a request can have
    int warp_share_log, cta_share_log;  // log2 of the tiles that a team of one warp, of one CTA takes at least
    int warp_extra, cta_extra;  // numbers before a segment's tiles, for each kind of team
    int warp_parts;          // teams are warps while no segment has more than this many of their shares
    float* part;             // [grid * warps * 2][n_col][hd] partial sums of the teams (and of groups of CTAs)
    float2* part_ml;         // [grid * warps * 2][n_col] their (max, sum)
    int* arrivals;           // [B * n_kv * n_qt][arrivals_ld], zero between runs: of the segment, then of its groups
    int* group_slots;        // [B * n_kv * n_qt][arrivals_ld] where a group's join lies
    int arrivals_ld;
    float* scores;           // [B * n_q][ctx_pad] log2-domain scores, or null
    float2* row_ml;          // [B * n_q] (max, 1 / sum)
    int ctx_pad;
};

struct KvWeightParams {
    KvPool pool;
    KvTable table;
    const int* lens;
    const float* scores;
    const float2* row_ml;
    int B, n_q, n_kv, group, ctx_pad;
};

struct KvEvictParams {
    KvPool pool;
    KvTable src, dst;
    KvCtl* ctl;
    const int* lens;
    int* new_lens;
    int* kept;               // [B, n_kv, budget]
    int* new_count;          // [B] slots that stay (workspace: new_lens may be the lens it is made from)
    unsigned long long* owner;  // [n_pages] (run << 32) | (request * ld + column + 1)
    int B, n_kv, budget, n_recent, n_sink;
    int row_bytes;           // head_dim * bytes an element
    int elem_bytes;
    int in_place;
    int page_shift;          // log2(page_size), or -1
    int fours;               // page_size is a multiple of 4 and acc lies on 16 bytes
};

}  // namespace et
