// Device helpers of the paged key-value cache's kernels.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "kv_shared.h"

namespace et {
namespace kv {

// Record the first error of a run (ET_ERR_INVALID) and what caused it; the
// mapped host word lets the next call see it.
__device__ __noinline__ inline void fail(KvCtl* ctl, int what, int a, int b, int c) {
    if (atomicCAS(&ctl->status, 0, 1) == 0) {
        ctl->diag[0] = what;
        ctl->diag[1] = a;
        ctl->diag[2] = b;
        ctl->diag[3] = c;
        *reinterpret_cast<volatile int*>(ctl->host_status) = 1;
        __threadfence_system();
    }
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// 16 bytes global -> shared without a register; `bytes` = 0 writes zeros.
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t* r, uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t* r, uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
// transpose of an 8 x 8 matrix of 16-bit values held as one register a lane
__device__ __forceinline__ uint32_t movm(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

// counts up an event; what the CTA wrote before its last barrier is visible to whom a later arrival tells
__device__ __forceinline__ int arrive(int* p) {
    int old;
    asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;" : "=r"(old) : "l"(p) : "memory");
    return old;
}

// launched with programmatic serialisation: wait for the grid before this one
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void grid_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// ------------------------------------------------------------ 16-bit types ----
struct Bf16 {
    static __device__ __forceinline__ float lo(uint32_t u) { return __uint_as_float(u << 16); }
    static __device__ __forceinline__ float hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {  // a in the low half
        __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&v);
    }
    static __device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};
struct Fp16 {
    static __device__ __forceinline__ float lo(uint32_t u) { return __half2float(__ushort_as_half((unsigned short)u)); }
    static __device__ __forceinline__ float hi(uint32_t u) { return __half2float(__ushort_as_half((unsigned short)(u >> 16))); }
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&v);
    }
    static __device__ __forceinline__ void mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
        asm(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%0, %1, %2, %3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
};

// two e4m3 values (low 16 bits) -> two fp16, exactly (e4m3's range and steps lie inside fp16's)
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t u) {
    uint32_t d;
    asm("{\n\t.reg .b16 x;\n\tcvt.u16.u32 x, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t}" : "=r"(d) : "r"(u));
    return d;
}
// two fp32 -> two e4m3 (a in the low byte), nearest even, saturating at 448
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    uint32_t d;
    asm("{\n\t.reg .b16 x;\n\tcvt.rn.satfinite.e4m3x2.f32 x, %2, %1;\n\tcvt.u32.u16 %0, x;\n\t}" : "=r"(d) : "f"(a), "f"(b));
    return d;
}

// 2^x (ex2.approx: at most 2 ulp off over the whole range)
__device__ __forceinline__ float exp2a(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The requests that have tiles, in order: id[i] is the i-th one's number,
// pre[i] the tiles of those before it (pre[live] all of them; shared memory).
// A length that is out of range counts as 0 and is reported.  All of the CTA's
// threads call; `tmp` holds two ints a warp.
struct Live {
    int n, longest;  // how many, and the most tiles of one
};
template <int kThreads>
__device__ __forceinline__ Live scan_tiles(int* pre, uint16_t* id, int* tmp, const int* lens, int B, int tile, int max_len, KvCtl* ctl) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    auto tiles = [&](int b) {
        if (b >= B) return 0;
        const int len = kv_checked_len(lens[b], max_len);
        if (len < 0) fail(ctl, KV_BAD_LEN, b, lens[b], max_len);
        return len > 0 ? (int)((unsigned)(len + tile - 1) / (unsigned)tile) : 0;
    };
    auto scan = [&](int v) {  // inclusive, over the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, v, o);
            if (lane >= o) v += y;
        }
        return v;
    };
    Live r;
    if (B <= 64) {  // every warp for itself, all writing the same values: no barrier
        const int n0 = tiles(2 * lane), n1 = tiles(2 * lane + 1), inc = scan(n0 + n1);
        const unsigned m0 = __ballot_sync(0xFFFFFFFFu, n0 > 0), m1 = __ballot_sync(0xFFFFFFFFu, n1 > 0), below = (1u << lane) - 1;
        const int at = __popc(m0 & below) + __popc(m1 & below);
        if (n0) {
            id[at] = (uint16_t)(2 * lane);
            pre[at + 1] = inc - n1;
        }
        if (n1) {
            id[at + (n0 > 0)] = (uint16_t)(2 * lane + 1);
            pre[at + (n0 > 0) + 1] = inc;
        }
        if (lane == 0) pre[0] = 0;
        __syncwarp();
        r.n = __popc(m0) + __popc(m1);
        r.longest = __reduce_max_sync(0xFFFFFFFFu, max(n0, n1));
        return r;
    }
    int carry = 0, most = 0;
    r.n = 0;
    for (int b0 = 0; b0 < B; b0 += kThreads) {
        const int b = b0 + threadIdx.x, n = tiles(b), inc = scan(n);
        const unsigned m = __ballot_sync(0xFFFFFFFFu, n > 0);
        most = max(most, n);
        if (lane == 31) {
            tmp[2 * w] = inc;
            tmp[2 * w + 1] = __popc(m);
        }
        __syncthreads();
        int base = carry, all = 0, at = r.n, lives = 0;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) {
            base += i < w ? tmp[2 * i] : 0;
            at += i < w ? tmp[2 * i + 1] : 0;
            all += tmp[2 * i];
            lives += tmp[2 * i + 1];
        }
        at += __popc(m & ((1u << lane) - 1));
        if (n) {
            id[at] = (uint16_t)b;
            pre[at + 1] = base + inc;
        }
        carry += all;
        r.n += lives;
        __syncthreads();
    }
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    if (lane == 0) tmp[w] = most;
    if (threadIdx.x == 0) pre[0] = 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) most = max(most, tmp[i]);
    r.longest = most;
    return r;
}

// Launch with programmatic serialisation: the grid may be set up while the
// one before it drains.  Every kernel here calls grid_wait() before it reads
// or writes anything another launch touches, but for the weights kernel: it
// reads the lengths (and reports a bad one) before.  That is sound because the
// attention it follows releases it behind a grid_wait() of its own: whoever
// wrote the lengths is done by then.
template <class... P>
cudaError_t launch_pdl(void (*f)(P...), dim3 grid, dim3 block, int smem, cudaStream_t s, int cluster, P... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, f, args...);
}

}  // namespace kv
}  // namespace et
