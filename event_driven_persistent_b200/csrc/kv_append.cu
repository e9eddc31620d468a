// New tokens' keys and values into the pages, with the per-head RMSNorm and
// rotate-half RoPE of queries and keys:
//   y = x * rsqrt(mean(x^2) + eps) * gain                  (optional)
//   z_i = y_i cos a_i - y_{i+hd/2} sin a_i,  z_{i+hd/2} = y_{i+hd/2} cos a_i + y_i sin a_i,
//   a_i = pos base^(-2i/hd)                                (optional)
//   cache <- round(z / scale) at the token's slot;  q' = round(z)
// Bound: memory, each element read once and written once; a copy reaches 6535 GB/s.
// Measured: 2 prompts of 8100 tokens, 64 / 8 heads of 128 to e4m3, 104 us (6080 GB/s);
// 8 prompts of 511..1537, 32 / 8 heads in bf16 with norms, 37 us (5400 GB/s, the
// loads that 16 warps an SM keep in flight); 64 single tokens 3.4 us, latency.

#include "kv_device.cuh"

namespace et {
namespace kv {
namespace {

constexpr int kThreads = 128;
constexpr int kBatch = 4;   // steps whose loads are in flight together

// two fp32 in one register pair: sm_100 multiplies and adds both in one instruction
struct F2 {
    unsigned long long v;
    __device__ __forceinline__ F2() {}
    __device__ __forceinline__ F2(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b)); }
    __device__ __forceinline__ void get(float& a, float& b) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
};
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return d;
}

// What a lane knows of its token.
struct Token {
    long long off;         // element offset of its row in the pools (head 0)
    int n, page, in_page;
    bool live;
    int dim;               // the first of the lane's eight dims in a half row
    int head, step;        // the heads it takes: head, head + step, ...
};

// The rows of the steps from head hb on: first halves in ua, second in ub.
template <int HD>
__device__ __forceinline__ void fetch(const KvAppendParams& p, const Token& k, int kind, bool live, int hb, uint4* ua, uint4* ub) {
    const int heads = kind == 0 ? p.n_q : p.n_kv;
    const long long ld = kind == 0 ? p.ldq : (kind == 1 ? p.ldk : p.ldv);
    const uint16_t* const src = static_cast<const uint16_t*>(kind == 0 ? p.q : (kind == 1 ? p.k : p.v)) + k.n * ld + k.dim;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
        const int h = hb + i * k.step;
        if (live && h < heads) {
            ua[i] = *reinterpret_cast<const uint4*>(src + h * HD);
            ub[i] = *reinterpret_cast<const uint4*>(src + h * HD + HD / 2);
        }
    }
}
// The head rows of one kind (0 query, 1 key, 2 value) of the warp's tokens, the
// first of them fetched already.  A row is held by L = hd / 16 lanes, eight elements of the first half and the
// eight they rotate with: 16-byte loads and stores, and a rotation needs no
// exchange.  The 32 / L rows of a step are heads of one token, or, when heads
// are few, of several.
template <int HD, class T, bool E4, int KIND>
__device__ __forceinline__ void append_rows(const KvAppendParams& p, const Token& k, const float2* cs, uint4* ua, uint4* ub) {
    constexpr int L = HD / 16, HALF = HD / 2;
    const int heads = KIND == 0 ? p.n_q : p.n_kv;
    // g_a cos, g_a sin, g_b cos, -g_b sin of the lane's pairs, by twos: they serve all of the token's rows
    F2 ac[4], as[4], bc[4], bs[4];
    const uint16_t* const gain = static_cast<const uint16_t*>(KIND == 0 ? p.gq : (KIND == 1 ? p.gk : nullptr));
    const bool norm = KIND != 2 && gain, turn = KIND != 2 && p.pos;
    if (norm || turn) {
        float ga[8], gb[8];
        if (norm) {
            const uint4 va = *reinterpret_cast<const uint4*>(gain + k.dim), vb = *reinterpret_cast<const uint4*>(gain + k.dim + HALF);
            const uint32_t xa[4] = {va.x, va.y, va.z, va.w}, xb[4] = {vb.x, vb.y, vb.z, vb.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                ga[2 * e] = T::lo(xa[e]);
                ga[2 * e + 1] = T::hi(xa[e]);
                gb[2 * e] = T::lo(xb[e]);
                gb[2 * e + 1] = T::hi(xb[e]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) ga[e] = gb[e] = 1.f;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float4 r = make_float4(1.f, 0.f, 1.f, 0.f);
            if (turn) r = *reinterpret_cast<const float4*>(cs + k.dim + 2 * e);
            ac[e] = F2(ga[2 * e] * r.x, ga[2 * e + 1] * r.z);
            as[e] = F2(ga[2 * e] * r.y, ga[2 * e + 1] * r.w);
            bc[e] = F2(gb[2 * e] * r.x, gb[2 * e + 1] * r.z);
            bs[e] = F2(-gb[2 * e] * r.y, -gb[2 * e + 1] * r.w);
        }
    }
    const int rounds = (heads + kBatch * k.step - 1) / (kBatch * k.step);  // the same count in every lane
    for (int round = 0, hb = k.head; round < rounds; ++round, hb += kBatch * k.step) {
        if (round) fetch<HD>(p, k, KIND, k.live, hb, ua, ub);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int h = hb + i * k.step;
            const bool live = k.live && h < heads;
            const long long at = k.off + (long long)h * p.pool.head_stride + k.dim;
            if (KIND == 2 && !E4) {  // a value only moves
                if (live) {
                    uint16_t* dst = static_cast<uint16_t*>(p.pool.V) + at;
                    *reinterpret_cast<uint4*>(dst) = ua[i];
                    *reinterpret_cast<uint4*>(dst + HALF) = ub[i];
                }
                continue;
            }
            F2 a[4], b[4];
            const uint32_t wa[4] = {ua[i].x, ua[i].y, ua[i].z, ua[i].w}, wb[4] = {ub[i].x, ub[i].y, ub[i].z, ub[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                a[e] = F2(T::lo(wa[e]), T::hi(wa[e]));
                b[e] = F2(T::lo(wb[e]), T::hi(wb[e]));
            }
            if (norm) {
                F2 sq = mul2(a[0], a[0]);
                sq = fma2(b[0], b[0], sq);
#pragma unroll
                for (int e = 1; e < 4; ++e) sq = fma2(b[e], b[e], fma2(a[e], a[e], sq));
                float s1, s2;
                sq.get(s1, s2);
                s1 += s2;
#pragma unroll
                for (int d = 1; d < L; d <<= 1) s1 += __shfl_xor_sync(0xFFFFFFFFu, s1, d);  // dead rows' lanes add only to their own
                const float inv = rsqrtf(s1 * (1.f / HD) + p.eps);
                const F2 inv2(inv, inv);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    a[e] = mul2(a[e], inv2);
                    b[e] = mul2(b[e], inv2);
                }
            }
            if (!live) continue;
            if (turn) {  // z_a = a (g_a cos) - b (g_b sin),  z_b = b (g_b cos) + a (g_a sin)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const F2 x = a[e], y = b[e];
                    a[e] = fma2(y, bs[e], mul2(x, ac[e]));
                    b[e] = fma2(x, as[e], mul2(y, bc[e]));
                }
            } else if (norm) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    a[e] = mul2(a[e], ac[e]);
                    b[e] = mul2(b[e], bc[e]);
                }
            }
            float x[8], y[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                a[e].get(x[2 * e], x[2 * e + 1]);
                b[e].get(y[2 * e], y[2 * e + 1]);
            }
            if (KIND == 0 || !E4) {
                uint16_t* dst = KIND == 0 ? static_cast<uint16_t*>(p.q_out) + k.n * p.ldqo + h * HD + k.dim : static_cast<uint16_t*>(p.pool.K) + at;
                *reinterpret_cast<uint4*>(dst) = make_uint4(T::pack(x[0], x[1]), T::pack(x[2], x[3]), T::pack(x[4], x[5]), T::pack(x[6], x[7]));
                *reinterpret_cast<uint4*>(dst + HALF) = make_uint4(T::pack(y[0], y[1]), T::pack(y[2], y[3]), T::pack(y[4], y[5]), T::pack(y[6], y[7]));
            } else {
                // one rounding, from fp32 to e4m3 (times the scale's reciprocal: two fp32 roundings before it, 2^-23 of the value;
                // a division costs 12 % on the long chunk above, 44 % with 16 / 16 heads)
                const float inv = 1.f / (KIND == 1 ? p.pool.k_scale[h] : p.pool.v_scale[h]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    x[e] *= inv;
                    y[e] *= inv;
                }
                uint8_t* dst = static_cast<uint8_t*>(KIND == 1 ? p.pool.K : p.pool.V) + at;
                *reinterpret_cast<uint2*>(dst) = make_uint2(e4m3x2(x[0], x[1]) | e4m3x2(x[2], x[3]) << 16, e4m3x2(x[4], x[5]) | e4m3x2(x[6], x[7]) << 16);
                *reinterpret_cast<uint2*>(dst + HALF) = make_uint2(e4m3x2(y[0], y[1]) | e4m3x2(y[2], y[3]) << 16, e4m3x2(y[4], y[5]) | e4m3x2(y[6], y[7]) << 16);
            }
            // a new token has received no weight yet
            if (KIND == 1 && p.pool.acc && k.dim == 0) p.pool.acc[((long long)k.page * p.n_kv + h) * p.pool.page_size + k.in_page] = 0.f;
        }
    }
}

// A warp takes a token, whose angles it works out once (a part of its heads,
// when tokens are few; several tokens, when heads are few).  With a block for a
// few tokens, tables in shared memory and scalar arithmetic, the kernel ran
// 317 instructions a step and was bound by them.  Places, first rows and angles
// are fetched together, before any of them is used, and 16 warps an SM have registers for
// it (64 tokens 3.7 -> 3.4 us, the long chunk above 107 -> 104; with 20 warps it spills).
template <int HD, class T, bool E4>
__global__ void __launch_bounds__(kThreads, 4) append_kernel(const __grid_constant__ KvAppendParams p, int log_parts, int log_tok) {
    constexpr int L = HD / 16, HALF = HD / 2, RG = 32 / L;
    __shared__ __align__(16) float2 cs[kThreads / 32][RG * HALF];  // of up to RG tokens
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned job = blockIdx.x * (kThreads / 32) + w;
    const int part = job & ((1u << log_parts) - 1), n0 = (int)(job >> log_parts) << log_tok;
    if (n0 >= p.N) return;
    const int hp = RG >> log_tok;  // heads a step
    const int t = lane / L / hp;   // the lane's token among the warp's
    Token k;
    k.dim = (lane % L) * 8;
    k.head = part * hp + lane / L % hp;
    k.step = hp << log_parts;
    k.n = n0 + t;
    k.off = -1;
    k.page = k.in_page = 0;
    grid_wait();
    const bool speak = lane % (L * hp) == 0;  // one lane a token reports
    int slot = -1;
    int req = k.n;
    if (k.n < p.N) {
        slot = p.slots[k.n];
        if (p.req) req = p.req[k.n];
    }
    bool live = false;
    if (slot >= 0) {  // a negative slot: padding
        if (req < 0 || req >= p.B) {
            if (speak) fail(p.ctl, KV_BAD_REQ, k.n, req, p.B);
        } else if (slot >= p.table.max_len) {
            if (speak) fail(p.ctl, KV_BAD_SLOT, k.n, slot, p.table.max_len);
        } else {
            live = true;
        }
    }
    if (!__any_sync(0xFFFFFFFFu, live)) return;
    // the page's number, the first rows and the angles' positions are on their way together
    if (live) {
        const unsigned pg = (unsigned)slot / (unsigned)p.pool.page_size;
        k.in_page = slot - (int)pg * p.pool.page_size;
        k.page = p.table.pages[(long long)req * p.table.ld + pg];
    }
    const int only = gridDim.y == 1 ? -1 : (int)blockIdx.y;  // kinds apart: a warp takes rows of one
    uint4 ua[kBatch], ub[kBatch];
    const int kind = only >= 0 ? only : (p.q ? 0 : 1);
    fetch<HD>(p, k, kind, live, k.head, ua, ub);
    if (p.pos && (gridDim.y == 1 || blockIdx.y != 2)) {
        // The angle in turns, in 64 bits: its fraction is exact to 1e-10 at positions of a million, where 32
        // bits would leave nothing.
        for (int i = lane; i < HALF << log_tok; i += 32) {
            const int n = min(n0 + i / HALF, p.N - 1);
            const double a = (double)p.pos[n] * p.turns[i % HALF];
            float sn, c;
            sincospif(2.f * (float)(a - rint(a)), &sn, &c);
            cs[w][i] = make_float2(c, sn);
        }
        __syncwarp();
    }
    if (live) {
        k.off = kv_row_offset(k.page, k.in_page, p.pool);
        if (k.off < 0 && speak) fail(p.ctl, KV_BAD_PAGE, req, slot, k.page);
    }
    k.live = k.off >= 0;
    const float2* const mine = cs[w] + t * HALF;
    if (kind == 0) append_rows<HD, T, E4, 0>(p, k, mine, ua, ub);
    if (only < 0 || only == 1) {
        if (kind != 1) fetch<HD>(p, k, 1, k.live, k.head, ua, ub);
        append_rows<HD, T, E4, 1>(p, k, mine, ua, ub);
    }
    if (only < 0 || only == 2) {
        if (kind != 2) fetch<HD>(p, k, 2, k.live, k.head, ua, ub);
        append_rows<HD, T, E4, 2>(p, k, mine, ua, ub);
    }
}

template <int HD, class T, bool E4>
cudaError_t append_launch(const KvAppendParams& p, int n_sm, cudaStream_t s) {
    constexpr int RG = 32 / (HD / 16);
    const int heads = p.n_q > p.n_kv ? p.n_q : p.n_kv;
    // Few tokens: kinds apart, and a kind's heads over as many warps as the GPU holds (64 tokens: 4.5 -> 3.5 us).  Many
    // query heads a KV head: kinds apart too, the smaller jobs last, which evens out the end (8200 tokens of 32 and 8
    // heads: 42 -> 38 us; of 16 and 16 heads it costs angles twice for nothing, 70 -> 75 us).
    const bool few = p.N <= 4 * n_sm, apart = few || p.n_q >= 4 * p.n_kv;
    int lp = 0, lt = 0;
    while (few && (RG << lp) < heads && ((long long)p.N << (lp + 1)) <= 8 * n_sm) ++lp;
    // A warp's tokens share its work on places and angles; with many heads two tokens do best, with few each row of a step
    // has one of its own (17000 tokens of 4 and 4 heads of 128: 46 -> 24 us; 16000 of 64 and 8: 112 -> 109 with two, 121
    // with four), as long as there are warps enough.
    if (!few)
        while ((2 << lt) <= RG && (lt == 0 || p.n_q + 2 * p.n_kv <= 32) && (p.N >> (lt + 1)) >= 8 * n_sm) ++lt;
    const long long jobs = ((p.N + (1ll << lt) - 1) >> lt) << lp, ctas = (jobs + kThreads / 32 - 1) / (kThreads / 32);
    return launch_pdl(append_kernel<HD, T, E4>, dim3((unsigned)ctas, apart ? 3 : 1), dim3(kThreads), 0, s, 1, p, lp, lt);
}

template <int HD>
cudaError_t append_dispatch(const KvAppendParams& p, int dtype, int cache, int n_sm, cudaStream_t s) {
    if (dtype == KV_BF16) return cache == KV_E4M3 ? append_launch<HD, Bf16, true>(p, n_sm, s) : append_launch<HD, Bf16, false>(p, n_sm, s);
    return cache == KV_E4M3 ? append_launch<HD, Fp16, true>(p, n_sm, s) : append_launch<HD, Fp16, false>(p, n_sm, s);
}

}  // namespace
}  // namespace kv

cudaError_t launch_kv_append(const KvAppendParams& p, int hd, int dtype, int cache, int n_sm, cudaStream_t s) {
    if (hd == 64) return kv::append_dispatch<64>(p, dtype, cache, n_sm, s);
    if (hd == 128) return kv::append_dispatch<128>(p, dtype, cache, n_sm, s);
    return kv::append_dispatch<256>(p, dtype, cache, n_sm, s);
}

}  // namespace et
