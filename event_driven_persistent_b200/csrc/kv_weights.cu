// Adds one decode step's attention weights to the slots' accumulated ones:
//   acc[page][g][slot] += sum over the heads h of group g of exp(x_hj - m_h) / l_h
// Second launch of an attention run that records weights: a slot's weight
// needs its row's final (m, l), which no split knows alone.  It reads the
// scores that the first launch left (4 bytes a slot and head, mostly still in
// L2) instead of K again (2 hd bytes a slot and KV head).
// Bound: L2 and the atomic adds; eight slots a thread and 16-byte adds, so that
// the page numbers and (m, l) are read once for them.  64 requests of 512..4096
// tokens, 32 / 8 heads: 10 us behind an attention of 102 us; K again would be 47 us.
#include "kv_device.cuh"

namespace et {
namespace {

constexpr int kThreads = 256;
constexpr int kSlots = 8 * kThreads;  // a thread takes twice four slots in a row: 16-byte loads, a page number each

__global__ void __launch_bounds__(kThreads) weights_kernel(const __grid_constant__ KvWeightParams p, KvCtl* ctl) {
    __shared__ int tmp[2 * kThreads / 32];
    __shared__ uint16_t id[kKvMaxB];
    extern __shared__ int pre[];
    // before the wait: the lengths are done where the attention before this kernel has released it (its release is behind its own wait)
    const kv::Live live = kv::scan_tiles<kThreads>(pre, id, tmp, p.lens, p.B, kSlots, p.table.max_len, ctl);
    kv::grid_wait();
    const bool fours = p.pool.page_size % 4 == 0 && (reinterpret_cast<uintptr_t>(p.pool.acc) & 15) == 0;
    const long long N = (long long)pre[live.n] * p.n_kv;
    for (long long t = blockIdx.x; t < N; t += gridDim.x) {
        const int i = kv_find_request(pre, live.n, 0, p.n_kv, t), b = id[i];
        const int nt = pre[i + 1] - pre[i];
        const int r = (int)(t - (long long)pre[i] * p.n_kv), u = r / nt;
        const int* pages = p.table.pages + (long long)b * p.table.ld;
        const long long row = (long long)b * p.n_q + u * p.group;
        const int len = p.lens[b], key0 = (r - u * nt) * kSlots + threadIdx.x * 4;
        int page[2], at[2];
        float w[2][4] = {};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int key = min(key0 + k * (kSlots / 2), len - 1);
            const unsigned pg = (unsigned)key / (unsigned)p.pool.page_size;
            page[k] = pages[pg];
            at[k] = key - (int)pg * p.pool.page_size;
        }
#pragma unroll 4
        for (int h = 0; h < p.group; ++h) {
            const float2 ml = p.row_ml[row + h];
            const float* x = p.scores + (row + h) * p.ctx_pad + key0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                if (key0 + k * (kSlots / 2) >= len) continue;
                const float4 s = *reinterpret_cast<const float4*>(x + k * (kSlots / 2));  // past the end: old numbers, not used
                w[k][0] += kv::exp2a(s.x - ml.x) * ml.y;
                w[k][1] += kv::exp2a(s.y - ml.x) * ml.y;
                w[k][2] += kv::exp2a(s.z - ml.x) * ml.y;
                w[k][3] += kv::exp2a(s.w - ml.x) * ml.y;
            }
        }
        // atomic adds: two requests may share a page, and then both count.  A bad page was reported by the first launch.
        float* acc = p.pool.acc + (long long)u * p.pool.page_size;
        const long long page_floats = (long long)p.n_kv * p.pool.page_size;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int key = key0 + k * (kSlots / 2), left = len - key;
            if (left <= 0) continue;
            if (fours && left >= 4) {
                if ((unsigned)page[k] < (unsigned)p.pool.n_pages)
                    asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(acc + page[k] * page_floats + at[k]), "f"(w[k][0]),
                                 "f"(w[k][1]), "f"(w[k][2]), "f"(w[k][3])
                                 : "memory");
                continue;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (e >= left) break;
                const unsigned pg = (unsigned)(key + e) / (unsigned)p.pool.page_size;
                const int pn = pages[pg], in = key + e - (int)pg * p.pool.page_size;
                if ((unsigned)pn < (unsigned)p.pool.n_pages) atomicAdd(acc + pn * page_floats + in, w[k][e]);
            }
        }
    }
}

}  // namespace

cudaError_t launch_kv_weights(const KvWeightParams& p, KvCtl* ctl, int n_sm, cudaStream_t s) {
    return kv::launch_pdl(weights_kernel, dim3((unsigned)(n_sm * 8)), dim3(kThreads), 4 * (p.B + 1), s, 1, p, ctl);
}

}  // namespace et
