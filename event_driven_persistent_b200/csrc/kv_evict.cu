// Eviction by accumulated attention weight.
//   n = len[b] <= budget: every slot stays.  Otherwise, per KV head, the first n_sink slots, the last n_recent ones and
//   the budget - n_sink - n_recent heaviest of the rest (equal weights: lower slot first) stay, in order, as slots
//   0 .. budget - 1 of the destination pages.
// Two launches, the selection and the move: no row may move before every
// destination page has been claimed, and in place a row's slot may be written once it has been read.
// Bound: memory; the weights are read once, the kept rows read and written once.
// Measured (8 KV heads of 128), to other pages: 32 requests of 1500..4096 slots to 2048 in bf16 97.5 us, of which the
// selection takes 10 and the move reaches 6000 GB/s; 4 x 65537 to 8192 in e4m3 47 us, 20 of them the
// selection: two passes of counting and five barriers across a cluster of eight CTAs; 1 x 4096 to 1024 10.6 us, latency.
// In place: 91 us, 113 us and 17 us; 1 x 65537 to 8192 in bf16 106 us (to other pages 31): few CTAs walk each row's tiles
// in order, each tile a chain of memory latencies.
#include <cooperative_groups.h>

#include "kv_device.cuh"

namespace et {
namespace kv {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxKeys = 16384;  // keys a CTA holds in shared memory; a longer slice reads the rest again from L2

__device__ __forceinline__ unsigned page_of(const KvEvictParams& p, int i) {
    return p.page_shift >= 0 ? (unsigned)i >> p.page_shift : (unsigned)i / (unsigned)p.pool.page_size;
}
__device__ __forceinline__ uint4 keys_of(float4 w) {
    return make_uint4(kv_weight_key(__float_as_uint(w.x)), kv_weight_key(__float_as_uint(w.y)), kv_weight_key(__float_as_uint(w.z)),
                      kv_weight_key(__float_as_uint(w.w)));
}
// Keys of slots i .. i + 3 (i a multiple of 4); those at n and beyond are not defined.
__device__ __forceinline__ uint4 keys_at(const KvEvictParams& p, int b, int u, int i, int n) {
    const int* pages = p.src.pages + (long long)b * p.src.ld;
    float w[4] = {0.f, 0.f, 0.f, 0.f};
    if (p.fours) {  // pages of 4 m slots, acc on 16 bytes: one page number, one load
        const unsigned pg = page_of(p, i);
        const int page = pages[pg];
        if ((unsigned)page < (unsigned)p.pool.n_pages) {
            const float4 v = *reinterpret_cast<const float4*>(p.pool.acc + ((long long)page * p.n_kv + u) * p.pool.page_size + (i - (int)pg * p.pool.page_size));
            w[0] = v.x;
            w[1] = v.y;
            w[2] = v.z;
            w[3] = v.w;
        } else {
            fail(p.ctl, KV_BAD_PAGE, b, i, page);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (i + k >= n) break;
            const unsigned pg = page_of(p, i + k);
            const int page = pages[pg];
            if ((unsigned)page < (unsigned)p.pool.n_pages)
                w[k] = p.pool.acc[((long long)page * p.n_kv + u) * p.pool.page_size + (i + k - (int)pg * p.pool.page_size)];
            else
                fail(p.ctl, KV_BAD_PAGE, b, i + k, page);
        }
    }
    return make_uint4(kv_weight_key(__float_as_uint(w[0])), kv_weight_key(__float_as_uint(w[1])), kv_weight_key(__float_as_uint(w[2])),
                      kv_weight_key(__float_as_uint(w[3])));
}

// Sums over the CTA of (a, b) below the thread (exclusive); *all gets the totals.
template <int kSel>
__device__ __forceinline__ uint2 cta_scan(uint2 v, uint2* tmp, uint2* all) {
    constexpr int kW = kSel / 32;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    uint2 inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(0xFFFFFFFFu, inc.x, o), z = __shfl_up_sync(0xFFFFFFFFu, inc.y, o);
        if (lane >= o) {
            inc.x += y;
            inc.y += z;
        }
    }
    if (lane == 31) tmp[w] = inc;
    __syncthreads();
    const uint2 t = lane < kW ? tmp[lane] : make_uint2(0, 0);
    all->x = __reduce_add_sync(0xFFFFFFFFu, t.x);
    all->y = __reduce_add_sync(0xFFFFFFFFu, t.y);
    const unsigned bx = __reduce_add_sync(0xFFFFFFFFu, lane < w ? t.x : 0u), by = __reduce_add_sync(0xFFFFFFFFu, lane < w ? t.y : 0u);
    __syncthreads();
    return make_uint2(bx + inc.x - v.x, by + inc.y - v.y);
}

// One cluster of CTAs a request and head, each with a slice of the slots, its
// keys (weights in an order-keeping 32-bit form) in shared memory.  The
// smallest key that stays is found by counting keys in bins (four a thread) of
// the range [lo, lo + bins << shift), first that of all keys (weights lie in few
// binades: fixed top digits would put them into a few dozen bins and queue the
// counting atomics there), then that of the bin the border lies in.  The CTAs
// of a cluster see each other's counts by groups of 32 bins first and then one
// group's bins: all bins of all CTAs would be 64 KB a CTA through the cluster's network (6000 cycles a
// pass against 2200).
template <int kSel>
__global__ void __launch_bounds__(kSel) select_kernel(const __grid_constant__ KvEvictParams p, int cap) {
    constexpr int kBins = 4 * kSel, kLogBins = kSel == 512 ? 11 : 9, kGroups = kBins / 32, kW = kSel / 32;
    constexpr int kPer = kGroups > 32 ? kGroups / 32 : 1;  // groups a lane
    constexpr int kStrip = 28;                             // slots a thread numbers at a time, at most
    static_assert(kBins == 1 << kLogBins && kPer * 32 >= kGroups, "");
    __shared__ __align__(16) unsigned hist[2][kBins];
    __shared__ __align__(16) unsigned sums[2][kGroups];
    __shared__ unsigned tmp[2][32], found[3], share[4];
    __shared__ uint2 tmp2[32];
    extern __shared__ __align__(16) unsigned keys[];
    cg::cluster_group cl = cg::this_cluster();
    const int cs = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    const int u = blockIdx.x / cs, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, wi = tid >> 5;
    auto cluster_sync = [&]() {
        __syncthreads();
        if (cs > 1) cl.sync();
    };
    auto over_cluster = [&](unsigned* a, int i) {  // sum of the CTAs' a[i], all loads in flight together
        unsigned t = a[i];
        if (cs > 1) {
            t = 0;
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (r < cs) t += cl.map_shared_rank(a, r)[i];
        }
        return t;
    };
    reinterpret_cast<uint4*>(hist[0])[tid] = make_uint4(0, 0, 0, 0);
    grid_wait();
    const unsigned run = *reinterpret_cast<volatile unsigned*>(&p.ctl->evict_run);
    const int len = kv_checked_len(p.lens[b], p.src.max_len);
    if (len < 0 && tid == 0) fail(p.ctl, KV_BAD_LEN, b, p.lens[b], p.src.max_len);
    const int n = len > 0 ? len : 0, keep = min(n, p.budget);
    int* kept = p.kept + ((long long)b * p.n_kv + u) * p.budget;
    if (blockIdx.x == 0 && tid == 0) p.new_count[b] = keep;
    // Claims of the destination pages: each may be the destination of one column only, but for columns of requests that
    // stay as they are in place (top bit of the tag), which may share: of two claims of a page the later sees the earlier.
    // A thread's first claim travels while the selection goes on.
    const int n_dst = (keep + p.pool.page_size - 1) / p.pool.page_size, j0 = blockIdx.x * kSel + tid;
    const int* const dst = p.dst.pages + (long long)b * p.dst.ld;
    const unsigned still = p.in_place && n <= p.budget ? 0x80000000u : 0u;
    auto claim = [&](int j, int page) -> unsigned long long {
        const unsigned long long tag = (unsigned long long)run << 32 | still | (unsigned)((unsigned)b * (unsigned)p.dst.ld + j + 1);
        return (unsigned)page < (unsigned)p.pool.n_pages ? atomicExch(p.owner + page, tag) : 0ull;
    };
    auto claimed = [&](int j, int page, unsigned long long own) {
        if ((unsigned)page >= (unsigned)p.pool.n_pages) fail(p.ctl, KV_BAD_PAGE, b, j, page);
        else if ((unsigned)(own >> 32) == run && !((unsigned)own & still)) fail(p.ctl, KV_BAD_DST, b, j, page);
    };
    const int page0 = j0 < n_dst ? dst[j0] : 0;
    unsigned long long own0 = 0;
    for (unsigned j = keep + rank * kSel + tid; j < (unsigned)p.budget; j += cs * kSel) kept[j] = -1;  // (unsigned: a budget near 2^31)
    if (n <= p.budget) {
        for (int j = rank * kSel + tid; j < n; j += cs * kSel) kept[j] = j;
        if (j0 < n_dst) own0 = claim(j0, page0);
        if (!p.in_place) {  // nobody reads the weights of its source pages, which are as many as its destinations: here they are checked
            const int* const pages = p.src.pages + (long long)b * p.src.ld;
            for (int j = j0; j < n_dst; j += gridDim.x * kSel)
                if ((unsigned)pages[j] >= (unsigned)p.pool.n_pages) fail(p.ctl, KV_BAD_PAGE, b, j * p.pool.page_size, pages[j]);
        }
    } else {
        const int c0 = p.n_sink, c1 = n - p.n_recent;  // the slots that compete
        const int per = ((n + cs - 1) / cs + 3) & ~3, s0 = min(n, rank * per), s1 = min(n, s0 + per);
        unsigned need = p.budget - p.n_sink - p.n_recent;
        // keys of slots i .. i + 3 (i - s0 a multiple of 4); 0, which no weight has, where a slot does not compete
        const unsigned width = (unsigned)(c1 - c0);
        auto competing = [&](uint4 v, int i) {
            const unsigned at = (unsigned)(i - c0);
            return make_uint4(at < width ? v.x : 0u, at + 1 < width ? v.y : 0u, at + 2 < width ? v.z : 0u, at + 3 < width ? v.w : 0u);
        };
        auto key4 = [&](int i) {
            return i - s0 < cap ? *reinterpret_cast<const uint4*>(keys + (i - s0)) : competing(keys_at(p, b, u, i, n), i);
        };
        unsigned lo = 0xFFFFFFFFu, hi = 0;  // lo: of key - 1
        auto take = [&](uint4 v, int i) {
            v = competing(v, i);
            if (i - s0 < cap) *reinterpret_cast<uint4*>(keys + (i - s0)) = v;
            lo = min(min(lo, min(v.x - 1, v.y - 1)), min(v.z - 1, v.w - 1));
            hi = max(max(hi, max(v.x, v.y)), max(v.z, v.w));
        };
        if (p.fours) {  // four pages' numbers, then four pages' weights in flight together
            const int* pages = p.src.pages + (long long)b * p.src.ld;
            for (int i = s0 + 4 * tid; i < s1; i += 16 * kSel) {
                int page[4];
                float4 w[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) page[k] = i + 4 * kSel * k < s1 ? pages[page_of(p, i + 4 * kSel * k)] : -1;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int at = i + 4 * kSel * k - (int)page_of(p, i + 4 * kSel * k) * p.pool.page_size;
                    w[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if ((unsigned)page[k] < (unsigned)p.pool.n_pages)
                        w[k] = *reinterpret_cast<const float4*>(p.pool.acc + ((long long)page[k] * p.n_kv + u) * p.pool.page_size + at);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (i + 4 * kSel * k >= s1) break;
                    if ((unsigned)page[k] >= (unsigned)p.pool.n_pages) fail(p.ctl, KV_BAD_PAGE, b, i + 4 * kSel * k, page[k]);
                    take(keys_of(w[k]), i + 4 * kSel * k);
                }
            }
        } else {
            for (int i = s0 + 4 * tid; i < s1; i += 4 * kSel) take(keys_at(p, b, u, i, n), i);
        }
        if (j0 < n_dst) own0 = claim(j0, page0);
        // The extremes of all slices, as is everything else the CTAs of a cluster tell one another: lane r reads rank r's.
        __syncwarp();
        lo = __reduce_min_sync(0xFFFFFFFFu, lo);
        hi = __reduce_max_sync(0xFFFFFFFFu, hi);
        if (lane == 0) {
            tmp[0][wi] = lo;
            tmp[1][wi] = hi;
        }
        __syncthreads();
        lo = __reduce_min_sync(0xFFFFFFFFu, tmp[0][lane & (kW - 1)]);
        hi = __reduce_max_sync(0xFFFFFFFFu, tmp[1][lane & (kW - 1)]);
        if (cs > 1) {
            if (tid == 0) {
                share[0] = lo;
                share[1] = hi;
            }
            cluster_sync();
            const unsigned* o = cl.map_shared_rank(share, lane & (cs - 1));  // cs: a power of two
            lo = __reduce_min_sync(0xFFFFFFFFu, o[0]);
            hi = __reduce_max_sync(0xFFFFFFFFu, o[1]);
        }
        ++lo;
        // [lo, hi]: where the border lies; a key above hi stays, one below lo goes
        const bool none = need == 0;
        bool all_in = false;               // every key >= lo stays
        for (int pass = 0; need && pass < kv_border_passes(kLogBins); ++pass) {
            const unsigned range = hi - lo;
            const int shift = kv_border_shift(range, kLogBins);
            unsigned* const h = hist[pass & 1];
            unsigned* const gs = sums[pass & 1];
            for (int i = s0 + 4 * tid; i < s1; i += 4 * kSel) {
                const uint4 v = key4(i);
                const unsigned k[4] = {v.x - lo, v.y - lo, v.z - lo, v.w - lo};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (k[e] <= range) atomicAdd(&h[k[e] >> shift], 1u);
            }
            __syncthreads();
            const uint4 v = reinterpret_cast<const uint4*>(h)[tid];
            unsigned sum = v.x + v.y + v.z + v.w;
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            if ((tid & 7) == 0) gs[tid >> 3] = sum;
            cluster_sync();
            if (wi == 0) {
                // from the top: the lane, then its group, then the bin that holds the need-th key
                unsigned c[kPer] = {};
                const bool on = (lane + 1) * kPer <= kGroups;
#pragma unroll
                for (int k = 0; k < kPer; ++k)
                    if (on) c[k] = over_cluster(gs, kGroups - 1 - (lane * kPer + k));
                unsigned all = 0;
#pragma unroll
                for (int k = 0; k < kPer; ++k) all += c[k];
                unsigned inc = all;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const unsigned y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                    if (lane >= o) inc += y;
                }
                unsigned above = inc - all, group = lane * kPer;
                const int at = __ffs(__ballot_sync(0xFFFFFFFFu, inc >= need)) - 1;
#pragma unroll
                for (int k = 0; k + 1 < kPer; ++k)
                    if (group == (unsigned)(lane * kPer + k) && above + c[k] < need) {
                        above += c[k];
                        ++group;
                    }
                above = __shfl_sync(0xFFFFFFFFu, above, at & 31);
                const unsigned top = (kGroups - 1 - (__shfl_sync(0xFFFFFFFFu, group, at & 31) & (kGroups - 1))) * 32 + 31;  // its highest bin
                const unsigned d = over_cluster(h, top - lane);
                inc = d;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const unsigned y = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                    if (lane >= o) inc += y;
                }
                const unsigned before = above + inc - d;
                if (lane == 0) {           // were weights written meanwhile, there may be no such bin: the search ends (and is reported below)
                    found[0] = 0;
                    found[1] = found[2] = need;
                }
                __syncwarp();
                if (before < need && before + d >= need) {
                    found[0] = top - lane;
                    found[1] = need - before;
                    found[2] = d;
                }
            } else {
                // the next pass's bins; those that the pass before used have been read by all
                for (int i = tid - 32; i < kBins / 4; i += kSel - 32) reinterpret_cast<uint4*>(hist[~pass & 1])[i] = make_uint4(0, 0, 0, 0);
            }
            __syncthreads();
            const unsigned bin = found[0];
            need = found[1];               // how many of the bin's keys stay
            lo += bin << shift;
            if (found[2] == need) {        // all of them
                all_in = true;
                break;
            }
            if (shift == 0) break;         // equal keys
            hi = kv_border_end(lo, hi, shift);
        }
        // Slots are numbered in strips, one a thread: as many fours as the slice needs, an odd number (no bank twice).
        const int fours = min(kStrip / 4, ((s1 - s0 + 4 * kSel - 1) / (4 * kSel)) | 1), strip = 4 * fours;
        auto below = [](int x) { return x <= 0 ? 0u : (x >= 32 ? 0xFFFFFFFFu : (1u << x) - 1u); };
        // of slots i .. i + strip - 1: those that stay, and those with the border's key, of which the first `need` do
        auto kinds = [&](int i) {
            unsigned more = 0, same = 0;
#pragma unroll
            for (int q = 0; q < kStrip / 4; ++q) {
                if (q >= fours || i + 4 * q >= s1) break;
                const uint4 v = key4(i + 4 * q);
                const unsigned k[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    more |= (k[e] > lo ? 1u : 0u) << (4 * q + e);
                    same |= (k[e] == lo ? 1u : 0u) << (4 * q + e);
                }
            }
            if (none) more = same = 0;
            if (all_in) {
                more |= same;
                same = 0;
            }
            const unsigned in = below(c1 - i) & ~below(c0 - i), valid = below(min(s1 - i, strip));
            return make_uint2(((more & in) | ~in) & valid, same & in & valid);
        };
        auto count = [](uint2 m) { return make_uint2(__popc(m.x), __popc(m.y)); };
        int i = s0 + strip * tid;
        unsigned at = 0, ties = 0;
        uint2 m = kinds(i), all, before = cta_scan<kSel>(count(m), tmp2, &all);
        if (cs > 1) {  // what the slices before this one keep
            uint2 total = all;
            if (s1 - s0 > strip * kSel) {
                uint2 v = make_uint2(0, 0), more;
                for (int j = i + strip * kSel; j < s1; j += strip * kSel) {
                    const uint2 y = count(kinds(j));
                    v.x += y.x;
                    v.y += y.y;
                }
                cta_scan<kSel>(v, tmp2, &more);
                total.x += more.x;
                total.y += more.y;
            }
            if (tid == 0) {
                share[2] = total.x;
                share[3] = total.y;
            }
            cluster_sync();
            const unsigned* o = cl.map_shared_rank(share, lane & (cs - 1));
            at = __reduce_add_sync(0xFFFFFFFFu, lane < rank ? o[2] : 0u);
            ties = __reduce_add_sync(0xFFFFFFFFu, lane < rank ? o[3] : 0u);
        }
        const unsigned at0 = at, ties0 = ties;
        for (int first = s0;;) {
            const unsigned tb = ties + before.y, room = need > tb ? need - tb : 0u;
            while ((unsigned)__popc(m.y) > room) m.y &= ~(1u << (31 - __clz(m.y)));  // the first `room` ties
            int to = at + before.x + min(tb, need);
            for (unsigned stay = m.x | m.y; stay; stay &= stay - 1, ++to)
                if (to < p.budget) kept[to] = i + __ffs(stay) - 1;  // (it always is, unless what is checked below fails)
            at += all.x;
            ties += all.y;
            first += strip * kSel;
            if (first >= s1) break;
            i += strip * kSel;
            m = kinds(i);
            before = cta_scan<kSel>(count(m), tmp2, &all);
        }
        // Keys beyond what the CTA holds are read for each step anew.  Were weights written meanwhile, the steps saw different
        // ones: each slice has to number as many slots as it told the others, and all of them `budget`, or the entries of
        // kept are not all written and the move must not use them.
        if (tid == 0 && ((cs > 1 && (at - at0 != share[2] || ties - ties0 != share[3])) ||
                         (rank == cs - 1 && at + min(ties, need) != (unsigned)p.budget)))
            fail(p.ctl, KV_BAD_WEIGHT, b, u, (int)(at + min(ties, need)));
        if (cs > 1) cluster_sync();        // nobody leaves while another reads its shared memory
    }
    if (j0 < n_dst) claimed(j0, page0, own0);
    for (int j = j0 + gridDim.x * kSel; j < n_dst; j += gridDim.x * kSel) {
        const int page = dst[j];
        claimed(j, page, claim(j, page));
    }
    grid_launch();
    // the last CTA opens the next run's tags; every thread has read this run's
    __syncthreads();
    if (tid == 0 && atomicAdd(&p.ctl->evict_done, 1u) == gridDim.x * gridDim.y - 1) {
        p.ctl->evict_done = 0;
        p.ctl->evict_run = run + 1;
    }
}

constexpr int kMove = 256;
constexpr int kPieces = 1024;  // 16-byte pieces of K (and of V) that a CTA holds at a time: 4 + 4 a thread

// A CTA moves K, V and weight of `kPieces / pieces a row` kept rows at a time:
// their places are worked out once for all of it.  grid.x: tiles of rows, or
// in place `slices` of the row, grid.y: KV head, grid.z: request.  In place a
// CTA walks the rows in order, a whole tile read before any of it is written:
// slot j comes from slot kept[j] >= j, so no later tile reads what this one wrote.
template <bool IN_PLACE>
__global__ void __launch_bounds__(kMove, 4) move_kernel(const __grid_constant__ KvEvictParams p, int slice) {
    __shared__ long long from[2][kPieces / 4], to[2][kPieces / 4];  // element offsets, -1: not moved
    __shared__ int bad;
    const int u = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
    const int lp = 31 - __clz(slice / 16);                    // log2 of the pieces a row
    const int rows = kPieces >> lp, first_piece = IN_PLACE ? blockIdx.x << lp : 0;
    grid_wait();
    // one reading for the whole CTA: the loop below holds barriers
    if (tid == 0) bad = *reinterpret_cast<volatile int*>(&p.ctl->status);
    __syncthreads();
    if (bad) return;
    const int keep = p.new_count[b];
    const int* kept = p.kept + ((long long)b * p.n_kv + u) * p.budget;
    const unsigned run = *reinterpret_cast<volatile unsigned*>(&p.ctl->evict_run) - 1;  // the selection has moved it on
    if (blockIdx.x == 0 && u == 0 && tid == 0) p.new_lens[b] = keep;
    const bool weights = !IN_PLACE || blockIdx.x == 0;
    auto where = [&](const KvTable& t, int i, bool check, long long* acc) -> long long {
        const unsigned pg = page_of(p, i);
        const int page = t.pages[(long long)b * t.ld + pg], in = i - (int)pg * p.pool.page_size;
        const long long o = kv_row_offset(page, in, p.pool);
        if (o < 0) return -1;  // reported by the selection
        if (check) {           // a source page that is the destination of another place, unless nothing moves there
            const unsigned long long own = p.owner[page];
            if ((unsigned)(own >> 32) == run && !((unsigned)own >> 31) &&
                (!IN_PLACE || (unsigned)own != (unsigned)b * (unsigned)t.ld + pg + 1)) {
                fail(p.ctl, KV_BAD_DST, b, (int)pg, page);
                return -1;
            }
        }
        *acc = ((long long)page * p.n_kv + u) * p.pool.page_size + in;
        return o + u * p.pool.head_stride;
    };
    int half = 0;
    for (int j0 = IN_PLACE ? 0 : blockIdx.x * rows; j0 < keep; j0 += IN_PLACE ? rows : gridDim.x * rows, half ^= 1) {
        float w = 0.f;
        long long wt = -1;
        if (tid < rows) {  // rows <= kMove
            const int j = j0 + tid;
            long long f = -1, t = -1, wf = 0;
            if (j < keep) {
                const int i = kept[j];
                // (the selection has written every entry, in ascending order, or reported that it has not)
                if ((unsigned)i < (unsigned)p.src.max_len && (!IN_PLACE || i != j)) {
                    t = where(p.dst, j, false, &wt);
                    f = where(p.src, i, true, &wf);
                    if (f < 0) wt = -1;
                    else if (weights) w = p.pool.acc[wf];
                }
            }
            from[half][tid] = t < 0 ? -1 : f;
            to[half][tid] = t;
        }
        __syncthreads();
        uint4 x[kPieces / kMove], y[kPieces / kMove];
#pragma unroll
        for (int k = 0; k < kPieces / kMove; ++k) {
            const int q = tid + k * kMove;
            const long long f = from[half][q >> lp];
            const long long o = f * p.elem_bytes + (first_piece + (q & ((1 << lp) - 1))) * 16;
            if (f >= 0) {
                x[k] = *reinterpret_cast<const uint4*>(static_cast<const char*>(p.pool.K) + o);
                y[k] = *reinterpret_cast<const uint4*>(static_cast<const char*>(p.pool.V) + o);
            }
        }
        if (IN_PLACE) __syncthreads();
#pragma unroll
        for (int k = 0; k < kPieces / kMove; ++k) {
            const int q = tid + k * kMove;
            const long long o = to[half][q >> lp] * p.elem_bytes + (first_piece + (q & ((1 << lp) - 1))) * 16;
            if (from[half][q >> lp] >= 0) {
                *reinterpret_cast<uint4*>(static_cast<char*>(p.pool.K) + o) = x[k];
                *reinterpret_cast<uint4*>(static_cast<char*>(p.pool.V) + o) = y[k];
            }
        }
        if (weights && wt >= 0) p.pool.acc[wt] = w;
    }
}

}  // namespace
}  // namespace kv

cudaError_t setup_kv_evict() {
    return cudaFuncSetAttribute(kv::select_kernel<512>, cudaFuncAttributeMaxDynamicSharedMemorySize, kv::kMaxKeys * 4);
}
cudaError_t launch_kv_evict(const KvEvictParams& p, int n_sm, cudaStream_t s) {
    using namespace kv;
    // By the longest row that the handle and the table hold, since the host does not know the lengths.  CTAs a row: as many as
    // keep a slice within 4096 slots, while they fit the GPU at two an SM (16 x 16384, 8 heads: 65 us, with four an SM, which
    // come in two waves, 74).  Short rows take CTAs of 128 threads, of which many fit an SM (the selection of 79 requests of 800
    // slots, 8 heads: 24 -> 16 us).  A handle and table for 131072 slots give short rows more CTAs or larger ones than
    // they need: 79 x 800 to 400 64 us in place of 56, 1 x 4096 to 1024 13 in place of 10.6; 32 x 1500..4096 98, as with its own.
    int cs = 1;
    while (cs < 8 && p.src.max_len / cs > 4096 && (long long)p.B * p.n_kv * cs * 2 <= 2 * n_sm) cs *= 2;
    int cap = ((p.src.max_len + cs - 1) / cs + 3) & ~3;
    if (cap > kMaxKeys) cap = kMaxKeys;
    const bool small = p.src.max_len <= 1024;
    const dim3 grid((unsigned)(p.n_kv * cs), (unsigned)p.B);
    cudaError_t e = small ? launch_pdl(select_kernel<128>, grid, dim3(128), cap * 4, s, 1, p, cap)
                          : launch_pdl(select_kernel<512>, grid, dim3(512), cap * 4, s, cs, p, cap);
    if (e != cudaSuccess) return e;
    int slice = p.row_bytes;
    if (p.in_place) {
        while (slice > 64 && (long long)p.B * p.n_kv * (p.row_bytes / slice) < 2 * n_sm) slice /= 2;
        return launch_pdl(move_kernel<true>, dim3((unsigned)(p.row_bytes / slice), (unsigned)p.n_kv, (unsigned)p.B), dim3(kMove), 0, s, 1, p, slice);
    }
    const int rows = kPieces / (slice / 16), most = p.budget < p.src.max_len ? p.budget : p.src.max_len;
    return launch_pdl(move_kernel<false>, dim3((unsigned)((most + rows - 1) / rows), (unsigned)p.n_kv, (unsigned)p.B), dim3(kMove), 0, s, 1, p, slice);
}

}  // namespace et
