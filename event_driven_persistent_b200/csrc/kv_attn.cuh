// Attention of one new token a request over the paged cache.
//
//   x_hj = scale q_h . K_j,  m_h = max_j x_hj,  l_h = sum_j exp(x_hj - m_h)
//   o_h  = sum_j exp(x_hj - m_h) V_j / l_h,     lse_h = m_h + log l_h
//
// Bound: every K and V row is read once from HBM (the query heads of a group
// share it), 4 hd flops a row and query head; nothing else is of that size.
//
// Split.  A segment is one request and one unit (a KV head, or 16 query
// heads of one, over 256 dims in e4m3 8).  All segments' tiles are numbered in order and every team takes an
// equal run of them (kv_share_begin), so ragged lengths balance without a
// plan from the host.  A segment that several teams share is joined by the
// team that arrives last: an event with a data-dependent wait count, as the
// decode layer's attention uses, but nobody waits on it.  A team is a warp
// while no segment is shared by more than a few of them, else a CTA, whose
// warps take its tiles in turn and join in shared memory first.
//
// Each warp has a ring of its own in shared memory, filled by cp.async, 16
// bytes a lane: no barrier between warps until a segment ends, rows of any
// page size and stride, and rows past the end written as zeros (whatever the
// page holds there, NaN included, never meets a product).  The ring runs
// across segment ends.  TMA boxes in their place (a page's slots in one copy,
// 10 % fewer instructions) were slower on every case, by 4 to 24 %: pages lie all over
// the pool, and a copy that waits for its address translation holds up
// every other copy of the SM.
//
// Products run on mma.sync m16n8k16 with the keys (then the head dims) as the
// 16 rows and the query heads as the 8 columns: a warp needs no exchange
// with another, and the group's few heads fill n = 8 instead of padding
// m = 128.  The tensor pipe is far from its limit either way.
//
// Precision: scores, running maximum, sum and output are fp32.  The
// probabilities enter the second product as two 16-bit terms, high and
// remainder (16 bits or more of p together), so that rounding p adds nothing next to
// the output's own rounding; with up to four heads a group the remainder
// rides in the columns that would be padding.  (One fp16 term, 2^-11 of p, where an e4m3 cache meets bf16
// outputs would show where values cancel.  It saves 1 us of the 112 of the
// 8 x 20000..65000 below, 8 of 132 at the power limit, and 15 of 112 of 8 x 30000 with 16 heads of 128 a group.)  An e4m3 cache is widened to
// fp16 exactly; bf16 queries are then scaled by a power of two into fp16's range.
//
// Measured (32 query and 8 KV heads of 128 in bf16, pages of 16, unless said; a
// copy reaches 6535 GB/s): 1 x 131071 tokens, pages of 32, 88 us (6100 GB/s);
// 8 x 20000..65000, 64 heads, e4m3, pages of 64, 112 us (6200; held for a
// second the GPU meets its power limit, and at 1.8 GHz it is 132 us); 16 x 512..4096
// 31 us (4870); 128 x 1..900, 16 / 16 heads of 64 in fp16, pages of 24, 47 us
// (5030); 1 x 517 8 us, a chain of latencies.  Long or many tokens are bound
// by HBM; what a run adds to that is about 5 us before its first tile and
// 2 us for a segment that several teams share.
#pragma once
#include <cuda_runtime.h>

#include <type_traits>

#include "kv_device.cuh"

namespace et {
namespace kv {

// How the query heads of a unit map to the tensor-core columns.
enum { kCols4 = 0, kCols8 = 1, kCols16 = 2 };

template <int HD, int CACHE, int MODE>
struct AttnShape {
    static constexpr int kWarps = kKvAttnWarps;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kElem = CACHE == KV_E4M3 ? 1 : 2;
    static constexpr int kRow = HD * kElem;                 // bytes of a cache row
    static constexpr int kCpr = kRow / 16;                  // 16-byte pieces of a row
    static constexpr int kKeys = kRow >= 256 ? 16 : 4096 / kRow;  // keys a tile: 4 KB of K (8 KB with 512-byte rows)
    static constexpr int kMt = kKeys / 16;
    static constexpr int kTile = 2 * kKeys * kRow;          // K and V
    static constexpr int kNt = MODE == kCols16 ? 2 : 1;
    static constexpr int kHeads = MODE == kCols4 ? 4 : (MODE == kCols8 ? 8 : 16);
    static constexpr int kRounds = kHeads * HD > 512 ? kHeads * HD / 512 : 1;  // passes of the join of the warps (about 8 KB each)
    static constexpr int kJoinDims = HD / kRounds;
    static constexpr int kJoinPitch = kJoinDims + 4;        // floats; + 4: the lanes of a store meet no bank twice
    static constexpr int kJoin = kWarps * kHeads * kJoinPitch * 4;
    // Two CTAs an SM (one with 512-byte rows, whose tiles are 16 KB)
    static constexpr int kPerSm = kRow >= 512 ? 1 : 2;
    static constexpr int kStages = 3;
    static constexpr int kRing = kWarps * kStages * kTile;
    static constexpr int kMl = 2 * kWarps * 16 * 4;         // each warp's (max, sum) a column
    static int smem(int B) { return kRing + kJoin + kMl + 64 + 4 * (B + 1) + 2 * B; }
};

// Byte offset of 16-byte piece c of row r inside the K or V half of a tile: the
// pieces of eight consecutive rows meet every bank once, for the copies and
// for ldmatrix.
template <int ROW>
__device__ __forceinline__ uint32_t piece(int r, int c) {
    if constexpr (ROW == 64) return (uint32_t)(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
    return (uint32_t)(r * ROW + ((c ^ (r & 7)) << 4));
}

template <int HD, class T, int CACHE, int MODE>
__global__ void __launch_bounds__(kKvAttnWarps * 32, (AttnShape<HD, CACHE, MODE>::kPerSm))
attn_kernel(const __grid_constant__ KvAttnParams p) {
    using S = AttnShape<HD, CACHE, MODE>;
    using M = typename std::conditional<CACHE == KV_E4M3, Fp16, T>::type;  // operand type of the products
    constexpr int W = S::kWarps, KT = S::kKeys, NT = S::kNt, NH = S::kHeads, ST = S::kStages;
    constexpr int ROW = S::kRow, CPR = S::kCpr, MT = S::kMt, KK = HD / 16;
    constexpr bool E4 = CACHE == KV_E4M3;
    // Probabilities are held as 2^up exp(x - m): fp16 operands keep their steps down to 2^(-24 - up), so that a long
    // tail of tiny ones is not lost next to one that is near 1 (bf16 has fp32's range).
    constexpr float UP = std::is_same<M, Fp16>::value ? 12.f : 0.f;
    constexpr float SLACK = std::is_same<M, Fp16>::value ? 3.f : 8.f;  // 2^(UP + SLACK) is inside fp16
    extern __shared__ __align__(128) unsigned char smem[];
    float* join = reinterpret_cast<float*>(smem + S::kRing);
    float* sm_m = reinterpret_cast<float*>(smem + S::kRing + S::kJoin);
    float* sm_l = sm_m + W * 16;
    int* tmp = reinterpret_cast<int*>(sm_l + W * 16);
    int* pre = tmp + 16;
    uint16_t* id = reinterpret_cast<uint16_t*>(pre + p.B + 1);
    const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const int units = p.n_kv * p.n_qt;

    grid_wait();
    // (the weights kernel, if any, counts on the release below lying behind this wait)
    const Live live = scan_tiles<W * 32>(pre, id, tmp, p.lens, p.B, KT, p.table.max_len, p.ctl);
    grid_launch();

    // rows of empty requests: zeros, log-sum-exp of nothing
    if (live.n < p.B)
        for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
            if (kv_checked_len(p.lens[b], p.table.max_len) > 0) continue;
            uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + (long long)b * p.ldo);
            for (int i = tid; i < p.n_q * HD / 2; i += W * 32) o[i] = 0;
            if (p.lse)
                for (int i = tid; i < p.n_q; i += W * 32) p.lse[(long long)b * p.n_q + i] = -INFINITY;
        }
    if (live.n == 0) return;

    // ---- teams: a warp each, or a CTA each
    const KvTeams teams = kv_choose_teams(pre[live.n], live.n, live.longest, units, gridDim.x, W, p.warp_share_log, p.cta_share_log,
                                          p.warp_extra, p.cta_extra, p.warp_parts);
    const bool solo = teams.solo;
    const int team = solo ? 1 : W, tw = solo ? 0 : w, tt = solo ? lane : tid;
    const int extra = teams.extra, C = teams.C;
    const long long N = teams.N;
    const int c = solo ? w * gridDim.x + blockIdx.x : blockIdx.x;
    if (c >= C) return;
    auto team_sync = [&]() {
        if (solo) __syncwarp(); else __syncthreads();
    };
    const long long share = kv_share_div(N, C), t0 = kv_share_begin(c, N, C, share), t1 = kv_share_begin(c + 1, N, C, share);
    const int run = (int)(t1 - t0);

    // ---- the warp's loads: tiles tw, tw + team, ... of the team's run.  Two
    // ways: eight rows of a page at a time (page_size a multiple of 8, every
    // key there), where a copy's address is the one before plus a step; else row by row.
    const uint32_t ring = smem_addr(smem) + w * (ST * S::kTile);
    const long long row_step = p.pool.slot_stride * S::kElem, page_step = p.pool.page_stride * S::kElem;
    const char* const k_lane = static_cast<const char*>(p.pool.K) + (lane / CPR) * row_step + (lane % CPR) * 16;
    const long long v_off = static_cast<const char*>(p.pool.V) - static_cast<const char*>(p.pool.K);
    const bool wide = (p.page_groups & 1) == 0;  // pages of 16 rows or more: every other group lies behind the one before
    KvWalk lw;
    kv_walk_to(lw, pre, live.n, extra, units, t0);
    KvWalk seg = lw;                         // the segment in use; the loads run ahead of it
    int lt = tw;                           // next tile to load
    int lb = 0, l_len = -1;                // its request, its length, page numbers, KV head's byte offset
    const int* l_pages = nullptr;
    long long l_head = 0;
    bool l_fast = false;
    int l_page[2 * MT];                    // pages of its groups of eight rows
    constexpr int RPL = KT > 32 ? KT / 32 : 1;  // rows whose offsets a lane works out
    long long l_off[RPL];                  // their byte offsets, -1: zeros
    auto page_of = [&](unsigned g8) { return p.page_groups == 1 ? g8 : __umulhi(g8, p.page_magic); };
    auto locate = [&]() {                  // where tile lt lies; its page numbers are on their way when this returns
        for (;;) {                         // over the extra numbers, and segments with no tile of this warp's
            if (lt < lw.s0) lt = lw.s0 + ((tw - lw.s0) & (team - 1));
            if (lt >= run) return;
            if (lt < lw.s1) break;
            kv_walk_next(lw, pre, live.n, extra, units);
            l_len = -1;
        }
        if (l_len < 0) {
            lb = id[lw.i];
            l_len = p.lens[lb];
            l_pages = p.table.pages + (long long)lb * p.table.ld;
            l_head = (long long)(p.n_qt == 1 ? lw.u : lw.u / p.n_qt) * p.pool.head_stride * S::kElem;
        }
        const int i = lt - lw.s0;
        l_fast = p.page_groups && (i + 1) * KT <= l_len;
        if (l_fast) {
#pragma unroll
            for (int g8 = 0; g8 < 2 * MT; ++g8)
                if (!(g8 & 1) || !wide) l_page[g8] = l_pages[page_of(i * 2 * MT + g8)];
        } else {
#pragma unroll
            for (int r = 0; r < RPL; ++r) {
                const int key = i * KT + ((lane + 32 * r) & (KT - 1));
                l_off[r] = -1;
                if (key < l_len) {
                    const unsigned pg = (unsigned)key / (unsigned)p.pool.page_size;
                    const int page = l_pages[pg];
                    const long long o = kv_row_offset(page, key - (int)pg * p.pool.page_size, p.pool);
                    if (o < 0) fail(p.ctl, KV_BAD_PAGE, lb, key, page);
                    else l_off[r] = o * S::kElem + l_head;
                }
            }
        }
    };
    constexpr int PER8 = 8 * CPR / 32, RPI = CPR >= 32 ? 1 : 32 / CPR;  // copies for eight rows, rows a copy
    auto load = [&](uint32_t dst) {        // tile lt into the ring, then on to the next one
        if (lt < run) {
            if (l_fast) {
                const int i = lt - lw.s0;
                const char* a = nullptr;
                uint32_t bytes = 0;
#pragma unroll
                for (int g8 = 0; g8 < 2 * MT; ++g8) {
                    if (!(g8 & 1) || !wide) {
                        const unsigned gi = i * 2 * MT + g8;
                        const bool in = (unsigned)l_page[g8] < (unsigned)p.pool.n_pages;
                        if (!in) fail(p.ctl, KV_BAD_PAGE, lb, gi * 8, l_page[g8]);
                        bytes = in ? 16u : 0u;
                        a = k_lane + l_head + (long long)((gi - page_of(gi) * p.page_groups) * 8) * row_step +
                            (in ? (long long)l_page[g8] * page_step : 0);
                    }
#pragma unroll
                    for (int k = 0; k < PER8; ++k) {
                        const uint32_t d = dst + piece<ROW>(g8 * 8 + k * RPI + lane / CPR, lane % CPR);
                        cp16(d, a, bytes);
                        cp16(d + KT * ROW, a + v_off, bytes);
                        a += RPI * row_step;
                    }
                }
            } else {
                const char* const kb = static_cast<const char*>(p.pool.K) + (lane % CPR) * 16;
#pragma unroll
                for (int k = 0; k < KT * CPR / 32; ++k) {
                    const int r = k * RPI + lane / CPR;
                    const long long o = __shfl_sync(0xFFFFFFFFu, l_off[(RPL > 1) ? r / 32 : 0], r & 31);
                    const uint32_t d = dst + piece<ROW>(r, lane % CPR), bytes = o >= 0 ? 16u : 0u;
                    const char* a = kb + (o >= 0 ? o : 0);
                    cp16(d, a, bytes);
                    cp16(d + KT * ROW, a + v_off, bytes);
                }
            }
            lt += team;
            locate();
        }
        cp_commit();
    };
    locate();
#pragma unroll 1
    for (int i = 0; i < ST - 1; ++i) load(ring + i * S::kTile);

    // ---- the team's segments, in order
    int ct = tw;                           // next tile to use
    uint32_t kb = ring, refill = ring + (ST - 1) * S::kTile;
    // the segment's request, KV head, first query head and how many; its queries as the B operand: lane (g, t4) holds
    // dims of column g (with e4m3 the dims of a 16-piece as the widened pairs fall)
    int b, len, kvh, h0, nh;
    uint32_t qf[KK][NT][2];
    auto take = [&]() {                    // issues the loads of segment `seg`
        b = id[seg.i];
        len = p.lens[b];
        kvh = p.n_qt == 1 ? seg.u : seg.u / p.n_qt;
        h0 = kvh * p.group + (p.n_qt == 1 ? 0 : (seg.u - kvh * p.n_qt) * kv_unit_heads(HD, E4));
        nh = min(p.group - (h0 - kvh * p.group), NH);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int hl = MODE == kCols4 ? (g & 3) : n * 8 + g;
            const uint16_t* qrow = static_cast<const uint16_t*>(p.q) + (long long)b * p.ldq + (long long)(h0 + hl) * HD;
#pragma unroll
            for (int k = 0; k < KK; ++k) {
                if constexpr (E4) {
                    uint2 v = make_uint2(0, 0);
                    if (hl < nh) v = *reinterpret_cast<const uint2*>(qrow + k * 16 + t4 * 4);
                    qf[k][n][0] = v.x;
                    qf[k][n][1] = v.y;
                } else {
                    qf[k][n][0] = hl < nh ? *reinterpret_cast<const uint32_t*>(qrow + k * 16 + t4 * 2) : 0u;
                    qf[k][n][1] = hl < nh ? *reinterpret_cast<const uint32_t*>(qrow + k * 16 + 8 + t4 * 2) : 0u;
                }
            }
        }
    };
    if (seg.s0 < run) take();
    while (seg.s0 < run) {
        const int s = seg.s0 > 0 ? seg.s0 : 0, e = seg.s1 < run ? seg.s1 : run;
        if (ct < s) ct = s + ((tw - s) & (team - 1));
        float qs[NT][2];                   // log2-domain scale of the lane's two columns
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            float sc = p.scale_log2;
            if constexpr (E4) {
                sc *= p.pool.k_scale[kvh];
                if constexpr (std::is_same<T, Bf16>::value) {
                    // bf16 -> fp16 through a power of two that brings the row's largest element to [1, 2): exact
                    // down to 2^-24 of that element
                    float mx = 0.f;
#pragma unroll
                    for (int k = 0; k < KK; ++k)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            mx = fmaxf(mx, fmaxf(fabsf(Bf16::lo(qf[k][n][i])), fabsf(Bf16::hi(qf[k][n][i]))));
                    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, 2));
                    // (2^-ex in two factors: one alone may lie beyond fp32's range)
                    const int ex = mx > 0.f && mx < INFINITY ? ilogbf(mx) : 0, e1 = ex / 2;
                    const float f1 = scalbnf(1.f, -e1), f2 = scalbnf(1.f, e1 - ex);
#pragma unroll
                    for (int k = 0; k < KK; ++k)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            qf[k][n][i] = Fp16::pack(Bf16::lo(qf[k][n][i]) * f1 * f2, Bf16::hi(qf[k][n][i]) * f1 * f2);
                    const float up = scalbnf(1.f, ex);  // of column g: hand it to the lanes whose columns are 2 t4, 2 t4 + 1
                    qs[n][0] = sc * __shfl_sync(0xFFFFFFFFu, up, 8 * t4);
                    qs[n][1] = sc * __shfl_sync(0xFFFFFFFFu, up, 8 * t4 + 4);
                } else {
                    qs[n][0] = qs[n][1] = sc;
                }
            } else {
                qs[n][0] = qs[n][1] = sc;
            }
        }

        // m: a maximum that lags by up to SLACK, so that few tiles need the exchange that finds a new one and the
        // rescaling; mb: what scores are taken from, m - UP (0 while there is no maximum)
        float o[KK][NT][4], m[NT][2], mb[NT][2], l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n][0] = m[n][1] = -INFINITY;
            mb[n][0] = mb[n][1] = 0.f;
            l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int k = 0; k < KK; ++k) o[k][n][0] = o[k][n][1] = o[k][n][2] = o[k][n][3] = 0.f;
        }

        for (; ct < e; ct += team) {
            cp_wait<ST - 2>();
            __syncwarp();
            const uint32_t vb = kb + KT * ROW;
            load(refill);  // the slot used one tile ago is free
            refill = kb;
            const int left = len - (ct - seg.s0) * KT;  // keys from the tile's first one on

            // S = K q^T: rows = keys, columns = heads
            float x[MT][NT][4];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
#pragma unroll
                for (int n = 0; n < NT; ++n) x[i][n][0] = x[i][n][1] = x[i][n][2] = x[i][n][3] = 0.f;
                const int r = i * 16 + (lane & 15);
                if constexpr (E4) {
#pragma unroll
                    for (int k = 0; k < KK; k += 2) {
                        uint32_t f[4];
                        ldsm4(f, kb + piece<ROW>(r, k + (lane >> 4)));
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t a[4] = {e4m3x2_f16x2(f[2 * h]), e4m3x2_f16x2(f[2 * h + 1]),
                                                   e4m3x2_f16x2(f[2 * h] >> 16), e4m3x2_f16x2(f[2 * h + 1] >> 16)};
#pragma unroll
                            for (int n = 0; n < NT; ++n) M::mma(x[i][n], a, qf[k + h][n][0], qf[k + h][n][1]);
                        }
                    }
                } else {
                    // a second chain of sums halves the wait for the products' latency (with two column tiles there are two already)
                    float odd[NT][4] = {};
#pragma unroll
                    for (int k = 0; k < KK; ++k) {
                        uint32_t a[4];
                        ldsm4(a, kb + piece<ROW>(r, 2 * k + (lane >> 4)));
#pragma unroll
                        for (int n = 0; n < NT; ++n) M::mma((k & 1) && NT == 1 ? odd[n] : x[i][n], a, qf[k][n][0], qf[k][n][1]);
                    }
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        if (NT == 1) x[i][0][v] += odd[0][v];
                }
            }
            // scale, mask
            const int key0 = (ct - seg.s0) * KT + g;
            bool grew = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int v = 0; v < 4; ++v) x[i][n][v] *= qs[n][v & 1];
            if (left < KT) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < MT; ++i)
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            if (g + i * 16 + (v >> 1) * 8 >= left) x[i][n][v] = -INFINITY;
            }
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    float top = x[0][n][v];
#pragma unroll
                    for (int i = 0; i < MT; ++i) top = fmaxf(top, fmaxf(x[i][n][v], x[i][n][v + 2]));
                    grew |= top > m[n][v] + SLACK;
                }
            if (p.scores) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const int col = n * 8 + 2 * t4 + (v & 1);
                        if (col >= nh) continue;
                        float* row = p.scores + ((long long)b * p.n_q + h0 + col) * p.ctx_pad;
#pragma unroll
                        for (int i = 0; i < MT; ++i) {
                            const int key = key0 + i * 16 + (v >> 1) * 8;
                            if (key < len) row[key] = x[i][n][v];
                        }
                    }
            }
            if (__any_sync(0xFFFFFFFFu, grew)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        float mn = m[n][v];
#pragma unroll
                        for (int i = 0; i < MT; ++i) mn = fmaxf(mn, fmaxf(x[i][n][v], x[i][n][v + 2]));
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xFFFFFFFFu, mn, d));
                        // no maximum yet (-inf): nothing has been summed, any factor serves
                        const float f = m[n][v] == -INFINITY ? 0.f : exp2a(m[n][v] - mn);
                        m[n][v] = mn;
                        mb[n][v] = mn == -INFINITY ? 0.f : mn - UP;
                        l[n][v] *= f;
#pragma unroll
                        for (int k = 0; k < KK; ++k) {
                            o[k][n][v] *= f;
                            o[k][n][v + 2] *= f;
                        }
                    }
            }
            // P, as the B operand of the second product (keys x heads)
            uint32_t ph[MT][NT][2], pl[MT][NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float a = exp2a(x[i][n][2 * h] - mb[n][0]), c1 = exp2a(x[i][n][2 * h + 1] - mb[n][1]);
                        l[n][0] += a;
                        l[n][1] += c1;
                        const uint32_t hi = M::pack(a, c1);
                        const uint32_t rest = M::pack(a - M::lo(hi), c1 - M::hi(hi));
                        if constexpr (MODE == kCols4) {  // columns 4..7 repeat heads 0..3 and carry the remainders
                            ph[i][n][h] = movm(t4 < 2 ? hi : rest);
                        } else {
                            ph[i][n][h] = movm(hi);
                            pl[i][n][h] = movm(rest);
                        }
                    }
            }
            // O += V^T P: rows = head dims, columns = heads
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                if constexpr (E4) {
                    const int r = i * 16 + (lane & 15);
#pragma unroll
                    for (int k = 0; k < KK; k += 2) {
                        uint32_t f[4];
                        ldsm4t(f, vb + piece<ROW>(r, k + (lane >> 4)));
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            // two dims of two keys: regrouped into two keys of each dim, then widened
                            const uint32_t u = __byte_perm(f[2 * h], 0, 0x3120), v = __byte_perm(f[2 * h + 1], 0, 0x3120);
                            const uint32_t a[4] = {e4m3x2_f16x2(u), e4m3x2_f16x2(u >> 16), e4m3x2_f16x2(v), e4m3x2_f16x2(v >> 16)};
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                M::mma(o[k + h][n], a, ph[i][n][0], ph[i][n][1]);
                                if constexpr (MODE != kCols4) M::mma(o[k + h][n], a, pl[i][n][0], pl[i][n][1]);
                            }
                        }
                    }
                } else {
                    const int r = i * 16 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
                    for (int k = 0; k < KK; ++k) {
                        uint32_t a[4];
                        ldsm4t(a, vb + piece<ROW>(r, 2 * k + ((lane >> 3) & 1)));
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            M::mma(o[k][n], a, ph[i][n][0], ph[i][n][1]);
                            if constexpr (MODE != kCols4) M::mma(o[k][n], a, pl[i][n][0], pl[i][n][1]);
                        }
                    }
                }
            }
            kb += S::kTile;
            if (kb == ring + ST * S::kTile) kb = ring;
            __syncwarp();  // every lane has read the tile before its slot is refilled
        }

        // ---- join the team's warps, the next segment's queries on their way meanwhile
        const KvWalk cur = seg;
        const int cb = b, ckvh = kvh, ch0 = h0, cnh = nh;
        kv_walk_next(seg, pre, live.n, extra, units);
        const bool more = seg.s0 < run;
        if (more) take();
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int v = 0; v < 2; ++v) {
#pragma unroll
                for (int d = 4; d < 32; d <<= 1) l[n][v] += __shfl_xor_sync(0xFFFFFFFFu, l[n][v], d);
                if (g == 0) {
                    sm_m[w * 16 + n * 8 + 2 * t4 + v] = m[n][v];
                    sm_l[w * 16 + n * 8 + 2 * t4 + v] = l[n][v];
                }
            }
        if constexpr (MODE == kCols4) {
#pragma unroll
            for (int k = 0; k < KK; ++k)
#pragma unroll
                for (int v = 0; v < 4; ++v) o[k][0][v] += __shfl_xor_sync(0xFFFFFFFFu, o[k][0][v], 2);
        }
        const bool whole = s == cur.s0 && e == cur.s1;
        const long long slot = (long long)c * kKvMaxSplits + kv_share_slot(c, t0 + cur.s0, N, C);
        const float vs = E4 ? p.pool.v_scale[ckvh] : 1.f;
#pragma unroll
        for (int r = 0; r < S::kRounds; ++r) {
            constexpr int KR = KK / S::kRounds;
#pragma unroll
            for (int kr = 0; kr < KR; ++kr) {
                const int k = r * KR + kr;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        const int col = n * 8 + 2 * t4 + (v & 1);
                        const int dim = kr * 16 + (E4 ? 2 * g + (v >> 1) : g + (v >> 1) * 8);
                        if (col < NH) join[(w * NH + col) * S::kJoinPitch + dim] = o[k][n][v];
                    }
            }
            team_sync();
            for (int i = tt; i < NH * S::kJoinDims / 4; i += team * 32) {
                const int col = i / (S::kJoinDims / 4), d = (i % (S::kJoinDims / 4)) * 4;
                if (col >= cnh) continue;
                float mm = -INFINITY, ll = 0.f;
                for (int j = w - tw; j < w - tw + team; ++j) mm = fmaxf(mm, sm_m[j * 16 + col]);
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int j = w - tw; j < w - tw + team; ++j) {
                    const float mj = sm_m[j * 16 + col];
                    const float f = mj == -INFINITY ? 0.f : exp2a(mj - mm);
                    // a warp without a finite score has summed nothing (or NaN, which stays)
                    const float4 y = *reinterpret_cast<const float4*>(join + (j * NH + col) * S::kJoinPitch + d);
                    a.x += f * y.x;
                    a.y += f * y.y;
                    a.z += f * y.z;
                    a.w += f * y.w;
                    ll += f * sm_l[j * 16 + col];
                }
                const int dim = r * S::kJoinDims + d;
                if (whole) {
                    const float inv = vs / ll;
                    uint2 y;
                    y.x = T::pack(a.x * inv, a.y * inv);
                    y.y = T::pack(a.z * inv, a.w * inv);
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (long long)cb * p.ldo + (long long)(ch0 + col) * HD + dim) = y;
                    if (dim == 0) {
                        const long long row = (long long)cb * p.n_q + ch0 + col;
                        if (p.lse) p.lse[row] = (mm - UP + log2f(ll)) * 0.69314718055994531f;
                        if (p.scores) p.row_ml[row] = make_float2(mm - UP, 1.f / ll);
                    }
                } else {
                    *reinterpret_cast<float4*>(p.part + (slot * NH + col) * HD + dim) = a;
                    if (dim == 0) p.part_ml[slot * NH + col] = make_float2(mm, ll);
                }
            }
            team_sync();
        }

        // ---- a shared segment: the team that arrives last joins the parts
        if (whole) continue;
        const KvParts parts = kv_parts(t0 + cur.s0, t0 + cur.s1, N, C);
        const int n_parts = parts.n;
        auto slot_of = [&](int k) { return kv_part_slot(parts, k); };
        // Joins `count` parts, P at a time, of 8 / P pieces of a row (their loads in flight together), with `many` threads, of
        // which this is number mt: into the output, or, unscaled, into slot `to`.  Part k lies in slot where(k).
        auto join_parts = [&](auto at_a_time, int count, auto where, int mt, int many, long long to) {
            constexpr int P = decltype(at_a_time)::value, R = 8 / P;
            const int total = cnh * HD / 4;
            for (int i0 = mt; i0 < total; i0 += many * R) {
                float mm[R], ll[R];
                float4 a[R];
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    mm[r] = -INFINITY;
                    ll[r] = 0.f;
                    a[r] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
                for (int k0 = 0; k0 < count; k0 += P) {
                    float2 ml[R][P];
                    float4 y[R][P];
#pragma unroll
                    for (int k = 0; k < P; ++k) {
                        const long long at = where(min(k0 + k, count - 1)) * NH;
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            const int i = min(i0 + r * many, total - 1), col = i / (HD / 4);
                            ml[r][k] = __ldcg(p.part_ml + at + col);
                            y[r][k] = __ldcg(reinterpret_cast<const float4*>(p.part + (at + col) * HD + (i % (HD / 4)) * 4));
                        }
                    }
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        float mn = mm[r];
#pragma unroll
                        for (int k = 0; k < P; ++k) mn = fmaxf(mn, ml[r][k].x);
                        const float fa = mm[r] == -INFINITY ? 0.f : exp2a(mm[r] - mn);
                        a[r].x *= fa;
                        a[r].y *= fa;
                        a[r].z *= fa;
                        a[r].w *= fa;
                        ll[r] *= fa;
#pragma unroll
                        for (int k = 0; k < P; ++k) {
                            if (k0 + k >= count) continue;
                            const float f = ml[r][k].x == -INFINITY ? 0.f : exp2a(ml[r][k].x - mn);
                            a[r].x += y[r][k].x * f;
                            a[r].y += y[r][k].y * f;
                            a[r].z += y[r][k].z * f;
                            a[r].w += y[r][k].w * f;
                            ll[r] += ml[r][k].y * f;
                        }
                        mm[r] = mn;
                    }
                }
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int i = i0 + r * many, col = i / (HD / 4), d = (i % (HD / 4)) * 4;
                    if (i >= total) break;
                    if (to >= 0) {
                        *reinterpret_cast<float4*>(p.part + (to * NH + col) * HD + d) = a[r];
                        if (d == 0) p.part_ml[to * NH + col] = make_float2(mm[r], ll[r]);
                        continue;
                    }
                    const float inv = vs / ll[r];
                    uint2 y;
                    y.x = T::pack(a[r].x * inv, a[r].y * inv);
                    y.y = T::pack(a[r].z * inv, a[r].w * inv);
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.out) + (long long)cb * p.ldo + (long long)(ch0 + col) * HD + d) = y;
                    if (d == 0) {
                        const long long row = (long long)cb * p.n_q + ch0 + col;
                        if (p.lse) p.lse[row] = (mm[r] - UP + log2f(ll[r])) * 0.69314718055994531f;
                        if (p.scores) p.row_ml[row] = make_float2(mm[r] - UP, 1.f / ll[r]);
                    }
                }
            }
        };
        using std::integral_constant;
        // One thread arrives for the team (the barrier above puts its writes before the arrival).
        int* const arr = p.arrivals + ((long long)cb * units + cur.u) * p.arrivals_ld;
        auto arrived_last = [&](int* at, int count) {
            const bool last = arrive(at) == count - 1;
            if (last) *at = 0;  // ready for the next run
            return (int)last;
        };
        int mt = tid, many = W * 32;
        if (solo || (more && n_parts <= 8)) {
            // a CTA with more to do leaves it, and joining a few parts, to one warp; its others go on
            if (!solo && w != (cur.u & (W - 1))) continue;
            if (!__shfl_sync(0xFFFFFFFFu, lane == 0 ? arrived_last(arr, n_parts) : 0, 0)) continue;
            __syncwarp();  // what lane 0's arrival made visible to it is so for the others too; a shuffle alone orders no memory
            mt = lane;
            many = 32;
        } else if (n_parts <= kKvJoin) {
            if (!__syncthreads_or(tid == 0 ? arrived_last(arr, n_parts) : 0)) continue;
        } else {
            // Many parts (few segments): by groups of kKvJoin, each joined by its last arrival into a slot past the teams'
            // own, then the groups (1 x 73306, 2 KV heads: 38 -> 24 us).
            const int groups = kv_join_groups(n_parts), gr = (c - parts.c0) / kKvJoin, size = min(kKvJoin, n_parts - gr * kKvJoin);
            if (!__syncthreads_or(tid == 0 ? arrived_last(arr + 1 + gr, size) : 0)) continue;
            const long long mine = kv_group_slot(gridDim.x, slot);
            join_parts(integral_constant<int, 8>(), size, [&](int k) { return slot_of(gr * kKvJoin + k); }, tid, W * 32, mine);
            int* const group_slot = p.group_slots + ((long long)cb * units + cur.u) * p.arrivals_ld;
            if (tid == 0) group_slot[gr] = (int)mine;
            __syncthreads();
            if (__syncthreads_or(tid == 0 ? arrived_last(arr, groups) : 0))
                join_parts(integral_constant<int, 8>(), groups, [&](int k) { return (long long)__ldcg(group_slot + k); }, tid, W * 32, -1);
            continue;
        }
        // Where a unit is large a few parts are joined several pieces at a time (16 heads of 128 dims are 16 pieces a lane: 32 x
        // 512..4096, 128 / 8 heads 68 -> 62 us; with 4 heads no faster, and 1 x 517 slower by the code's size, 7.9 -> 8.2 us).
        constexpr bool kLarge = NH * HD >= 1024;
        if (kLarge && n_parts <= 2) join_parts(integral_constant<int, kLarge ? 2 : 8>(), n_parts, slot_of, mt, many, -1);
        else if (kLarge && n_parts <= 4) join_parts(integral_constant<int, kLarge ? 4 : 8>(), n_parts, slot_of, mt, many, -1);
        else join_parts(integral_constant<int, 8>(), n_parts, slot_of, mt, many, -1);
    }
    cp_wait<0>();
}

template <int HD, class T, int CACHE, int MODE>
cudaError_t attn_launch(const KvAttnParams* p, int n_sm, cudaStream_t s) {
    using S = AttnShape<HD, CACHE, MODE>;
    auto* f = attn_kernel<HD, T, CACHE, MODE>;
    if (!p) return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, S::smem(kKvMaxB));
    return launch_pdl(f, dim3((unsigned)(n_sm * S::kPerSm)), dim3(S::kThreads), S::smem(p->B), s, 1, *p);
}

// The instantiation for a head size: type of q and out, cache type, columns (by the
// query heads of a KV head).  p null: sets the kernel up on the current device.
template <int HD>
cudaError_t attn_dispatch(const KvAttnParams* p, int dtype, int cache, int group, int n_sm, cudaStream_t s) {
#define KV_MODE(T, CACHE)                                                                            \
    {                                                                                                \
        constexpr int kMost = kv_unit_heads(HD, CACHE == KV_E4M3) == 8 ? kCols8 : kCols16;           \
        if (group <= 4) return attn_launch<HD, T, CACHE, kCols4>(p, n_sm, s);                        \
        if (group <= 8) return attn_launch<HD, T, CACHE, kCols8>(p, n_sm, s);                        \
        return attn_launch<HD, T, CACHE, kMost>(p, n_sm, s);                                         \
    }
    if (dtype == KV_BF16) {
        if (cache == KV_BF16) KV_MODE(Bf16, KV_BF16)
        KV_MODE(Bf16, KV_E4M3)
    }
    if (cache == KV_FP16) KV_MODE(Fp16, KV_FP16)
    KV_MODE(Fp16, KV_E4M3)
#undef KV_MODE
}

}  // namespace kv
}  // namespace et
