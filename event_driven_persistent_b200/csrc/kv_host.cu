// Host half of the paged key-value cache: its C entry points (include/et.h),
// checks of arguments, workspace and launches.
#include <cuda_runtime.h>
#include <float.h>
#include <math.h>

#include <algorithm>
#include <cstring>
#include <new>
#include <vector>

#include "../../include/et.h"
#include "kv_shared.h"

namespace et {
cudaError_t launch_kv_append(const KvAppendParams& p, int hd, int dtype, int cache, int n_sm, cudaStream_t s);
cudaError_t launch_kv_attn_64(const KvAttnParams* p, int dtype, int cache, int group, int n_sm, cudaStream_t s);
cudaError_t launch_kv_attn_128(const KvAttnParams* p, int dtype, int cache, int group, int n_sm, cudaStream_t s);
cudaError_t launch_kv_attn_256(const KvAttnParams* p, int dtype, int cache, int group, int n_sm, cudaStream_t s);
cudaError_t launch_kv_weights(const KvWeightParams& p, KvCtl* ctl, int n_sm, cudaStream_t s);
cudaError_t setup_kv_evict();
cudaError_t launch_kv_evict(const KvEvictParams& p, int n_sm, cudaStream_t s);
}  // namespace et

using namespace et;

struct et_kv {
    et_kv_desc d;
    int n_sm = 0, elem = 2, ces = 2, n_qt = 1;
    KvCtl* ctl = nullptr;
    int* host_status = nullptr;
    int* host_status_dev = nullptr;
    double* turns = nullptr;
    float* part = nullptr;
    float2* part_ml = nullptr;
    int* arrivals = nullptr;
    int* group_slots = nullptr;
    int arrivals_ld = 0;
    size_t n_arrivals = 0;
    float* scores = nullptr;
    float2* row_ml = nullptr;
    int ctx_pad = 0;
    unsigned long long* owner = nullptr;
    int* new_count = nullptr;
    std::vector<void*> allocs;
};

namespace {

// The handle's device for the length of a call; the caller's own comes back.
struct OnDevice {
    int before = -1;
    bool ok = false;
    explicit OnDevice(int dev) {
        if (cudaGetDevice(&before) != cudaSuccess) return;
        ok = before == dev || cudaSetDevice(dev) == cudaSuccess;
        if (before == dev) before = -1;
    }
    ~OnDevice() {
        if (before >= 0) cudaSetDevice(before);
    }
};

et_status cuda_fail(cudaError_t e) { return e == cudaErrorMemoryAllocation ? ET_ERR_OOM : ET_ERR_CUDA; }

#define KV_CU(call)                                  \
    do {                                             \
        cudaError_t e_ = (call);                     \
        if (e_ != cudaSuccess) return cuda_fail(e_); \
    } while (0)

template <class T>
et_status kv_alloc(et_kv* kv, T** p, size_t n) {
    void* q = nullptr;
    KV_CU(cudaMalloc(&q, std::max<size_t>(n, 1) * sizeof(T)));
    kv->allocs.push_back(q);
    KV_CU(cudaMemset(q, 0, std::max<size_t>(n, 1) * sizeof(T)));
    *p = static_cast<T*>(q);
    return ET_OK;
}

bool al16(const void* p) { return p && ((uintptr_t)p & 15) == 0; }
bool al4(const void* p) { return p && ((uintptr_t)p & 3) == 0; }
bool bad_ld(int64_t ld) { return ld < 0 || ld % 8; }  // rows are read and written in 16-byte pieces

et_status reset_ctl(et_kv* kv) {
    KvCtl h;
    memset(&h, 0, sizeof(h));
    h.host_status = kv->host_status_dev;
    h.evict_run = 1;
    KV_CU(cudaMemcpy(kv->ctl, &h, sizeof(h), cudaMemcpyHostToDevice));
    *reinterpret_cast<volatile int*>(kv->host_status) = 0;
    return ET_OK;
}

// What every run checks: the handle, the pool, the table.
et_status take_pool(const et_kv* kv, const et_kv_pool* in, KvPool* out) {
    if (!kv || !in) return ET_ERR_INVALID;
    if (!al16(in->K) || !al16(in->V)) return ET_ERR_INVALID;
    const et_kv_desc& d = kv->d;
    if (d.cache_dtype == ET_E4M3 && (!al4(in->k_scale) || !al4(in->v_scale))) return ET_ERR_INVALID;
    if (in->acc && !al4(in->acc)) return ET_ERR_INVALID;
    long long ps = in->page_stride, hs = in->head_stride, ss = in->slot_stride;
    if (!ps && !hs && !ss) {
        ss = d.head_dim;
        hs = ss * d.page_size;
        ps = hs * d.n_kv_heads;
    }
    const long long unit = 16 / kv->ces;  // rows are read in 16-byte pieces
    if (ps < 0 || hs < 0 || ss < 0 || ps % unit || hs % unit || ss % unit) return ET_ERR_INVALID;
    out->K = in->K;
    out->V = in->V;
    out->k_scale = in->k_scale;
    out->v_scale = in->v_scale;
    out->acc = in->acc;
    out->page_stride = ps;
    out->head_stride = hs;
    out->slot_stride = ss;
    out->n_pages = d.n_pages;
    out->page_size = d.page_size;
    out->n_kv = d.n_kv_heads;
    return ET_OK;
}
et_status take_table(const et_kv* kv, int B, const int32_t* table, int64_t ld, KvTable* out) {
    if (B < 1 || B > kv->d.max_B || !al4(table) || ld < 1 || ld > 0x7FFFFFFF / B) return ET_ERR_INVALID;
    out->pages = table;
    out->ld = ld;
    out->max_len = (int)std::min<long long>(kv->d.max_ctx, (long long)ld * kv->d.page_size);
    return ET_OK;
}
et_status not_pending(const et_kv* kv) {
    return *reinterpret_cast<volatile const int*>(kv->host_status) ? ET_ERR_PENDING : ET_OK;
}

#define KV_TRY(x)                   \
    do {                            \
        et_status s_ = (x);         \
        if (s_ != ET_OK) return s_; \
    } while (0)

auto* attn_of(const et_kv_desc& d) {
    return d.head_dim == 64 ? launch_kv_attn_64 : (d.head_dim == 128 ? launch_kv_attn_128 : launch_kv_attn_256);
}

et_status build(et_kv* kv) {
    const et_kv_desc& d = kv->d;
    KV_CU(attn_of(d)(nullptr, d.dtype, d.cache_dtype, d.n_heads / d.n_kv_heads, kv->n_sm, nullptr));
    KV_CU(setup_kv_evict());
    KV_TRY(kv_alloc(kv, &kv->ctl, 1));
    void* hp = nullptr;
    KV_CU(cudaHostAlloc(&hp, sizeof(int), cudaHostAllocMapped));
    kv->host_status = static_cast<int*>(hp);
    void* dp = nullptr;
    KV_CU(cudaHostGetDevicePointer(&dp, hp, 0));
    kv->host_status_dev = static_cast<int*>(dp);
    KV_TRY(reset_ctl(kv));
    std::vector<double> turns(d.head_dim / 2);
    for (int i = 0; i < d.head_dim / 2; ++i)
        turns[i] = pow((double)d.rope_base, -2.0 * i / d.head_dim) / 6.283185307179586476925;
    KV_TRY(kv_alloc(kv, &kv->turns, turns.size()));
    KV_CU(cudaMemcpy(kv->turns, turns.data(), turns.size() * sizeof(double), cudaMemcpyHostToDevice));
    const size_t slots = (size_t)kv_part_slots(kv->n_sm);
    const int group = d.n_heads / d.n_kv_heads;
    const size_t cols = group <= 4 ? 4 : (group <= 8 ? 8 : kv_unit_heads(d.head_dim, d.cache_dtype == ET_E4M3));
    KV_TRY(kv_alloc(kv, &kv->part, slots * cols * d.head_dim));
    KV_TRY(kv_alloc(kv, &kv->part_ml, slots * cols));
    kv->arrivals_ld = kv_arrivals(kv->n_sm);
    kv->n_arrivals = (size_t)d.max_B * d.n_kv_heads * kv->n_qt * kv->arrivals_ld;
    KV_TRY(kv_alloc(kv, &kv->arrivals, kv->n_arrivals));
    KV_TRY(kv_alloc(kv, &kv->group_slots, kv->n_arrivals));
    KV_TRY(kv_alloc(kv, &kv->row_ml, (size_t)d.max_B * d.n_heads));
    kv->ctx_pad = (d.max_ctx + 7) / 8 * 8;
    if (d.track_weights) KV_TRY(kv_alloc(kv, &kv->scores, (size_t)d.max_B * d.n_heads * kv->ctx_pad));
    KV_TRY(kv_alloc(kv, &kv->owner, (size_t)d.n_pages));
    KV_TRY(kv_alloc(kv, &kv->new_count, (size_t)d.max_B));
    KV_CU(cudaDeviceSynchronize());
    return ET_OK;
}

}  // namespace

extern "C" {

et_status et_build_kv(const et_kv_desc* desc, et_kv** out) {
    if (!desc || !out) return ET_ERR_INVALID;
    *out = nullptr;
    et_kv_desc d = *desc;
    if (d.page_size == 0) d.page_size = 16;
    if (d.n_heads == 0) d.n_heads = 32;
    if (d.n_kv_heads == 0) d.n_kv_heads = 8;
    if (d.head_dim == 0) d.head_dim = 128;
    if (d.rope_base == 0.f) d.rope_base = 500000.f;
    if (d.rms_eps == 0.f) d.rms_eps = 1e-5f;
    if (d.max_B < 1 || d.max_ctx < 1 || d.n_pages < 1 || d.page_size < 1 || d.n_heads < 1 || d.n_kv_heads < 1)
        return ET_ERR_INVALID;
    if (!(d.rope_base > 0.f) || !(d.rms_eps > 0.f)) return ET_ERR_INVALID;
    if (d.dtype != ET_BF16 && d.dtype != ET_FP16) return ET_ERR_INVALID;
    if (d.cache_dtype != d.dtype && d.cache_dtype != ET_E4M3) return ET_ERR_INVALID;
    if (d.n_heads % d.n_kv_heads) return ET_ERR_INVALID;
    if (d.head_dim != 64 && d.head_dim != 128 && d.head_dim != 256) return ET_ERR_UNSUPPORTED;
    if (d.max_B > kKvMaxB || d.n_heads > 1024 || d.page_size > 4096 || d.max_ctx > (1 << 24)) return ET_ERR_UNSUPPORTED;
    et_kv* kv = new (std::nothrow) et_kv();
    if (!kv) return ET_ERR_OOM;
    kv->d = d;
    kv->ces = d.cache_dtype == ET_E4M3 ? 1 : 2;
    const int most = kv_unit_heads(d.head_dim, d.cache_dtype == ET_E4M3);
    kv->n_qt = (d.n_heads / d.n_kv_heads + most - 1) / most;
    et_status st = ET_ERR_CUDA;
    {
        OnDevice on(d.device);
        int major = 0;
        if (on.ok && cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, d.device) == cudaSuccess &&
            cudaDeviceGetAttribute(&kv->n_sm, cudaDevAttrMultiProcessorCount, d.device) == cudaSuccess) {
            if (major != 10 || kv_longest_run(d.max_B, d.max_ctx, d.n_kv_heads * kv->n_qt, kv->n_sm) >= 1 << 30) {
                st = ET_ERR_UNSUPPORTED;
            } else {
                try {
                    st = build(kv);
                } catch (...) {  // no C++ exception leaves a C entry
                    st = ET_ERR_OOM;
                }
            }
        }
    }
    if (st != ET_OK) {
        et_destroy_kv(kv);
        return st;
    }
    *out = kv;
    return ET_OK;
}

void et_destroy_kv(et_kv* kv) {
    if (!kv) return;
    {
        OnDevice on(kv->d.device);
        if (!kv->allocs.empty()) cudaDeviceSynchronize();
        for (void* p : kv->allocs) cudaFree(p);
        if (kv->host_status) cudaFreeHost(kv->host_status);
    }
    delete kv;
}

et_status et_run_kv_append(et_kv* kv, const et_kv_pool* pool, const et_kv_append_args* a, void* stream) {
    KvAppendParams p;
    KV_TRY(take_pool(kv, pool, &p.pool));
    if (!a) return ET_ERR_INVALID;
    KV_TRY(take_table(kv, a->B, a->table, a->ld_table, &p.table));
    if (a->N < 0 || a->N > 1 << 30) return ET_ERR_INVALID;
    if (a->N == 0) return ET_OK;
    if (!al4(a->slots) || (a->req && !al4(a->req)) || (a->pos && !al4(a->pos))) return ET_ERR_INVALID;
    if (!al16(a->k) || !al16(a->v) || bad_ld(a->ldk) || bad_ld(a->ldv)) return ET_ERR_INVALID;
    if (a->q && (!al16(a->q) || !al16(a->q_out) || bad_ld(a->ldq) || bad_ld(a->ldqo))) return ET_ERR_INVALID;
    // rows of the output must not overlap
    if (a->q && a->N > 1 && a->ldqo < (int64_t)kv->d.n_heads * kv->d.head_dim) return ET_ERR_INVALID;
    if ((a->gq && !al16(a->gq)) || (a->gk && !al16(a->gk))) return ET_ERR_INVALID;
    if (!a->req && a->N > a->B) return ET_ERR_INVALID;  // token i belongs to request i
    KV_TRY(not_pending(kv));
    OnDevice on(kv->d.device);
    if (!on.ok) return ET_ERR_CUDA;
    p.ctl = kv->ctl;
    p.turns = kv->turns;
    p.q = a->q;
    p.k = a->k;
    p.v = a->v;
    p.q_out = a->q_out;
    p.ldq = a->ldq;
    p.ldk = a->ldk;
    p.ldv = a->ldv;
    p.ldqo = a->ldqo;
    p.gq = a->gq;
    p.gk = a->gk;
    p.req = a->req;
    p.slots = a->slots;
    p.pos = a->pos;
    p.eps = kv->d.rms_eps;
    p.N = a->N;
    p.B = a->B;
    p.n_q = a->q ? kv->d.n_heads : 0;
    p.n_kv = kv->d.n_kv_heads;
    KV_CU(launch_kv_append(p, kv->d.head_dim, kv->d.dtype, kv->d.cache_dtype, kv->n_sm, (cudaStream_t)stream));
    return ET_OK;
}

et_status et_run_kv_attn(et_kv* kv, const et_kv_pool* pool, const et_kv_attn_args* a, void* stream) {
    KvAttnParams p;
    KV_TRY(take_pool(kv, pool, &p.pool));
    if (!a) return ET_ERR_INVALID;
    KV_TRY(take_table(kv, a->B, a->table, a->ld_table, &p.table));
    const et_kv_desc& d = kv->d;
    const float scale = a->scale;
    const bool accumulate = a->accumulate != 0;
    if (!al4(a->lens) || !al16(a->q) || !al16(a->out) || bad_ld(a->ldq) || bad_ld(a->ldo) || (a->lse && !al4(a->lse)))
        return ET_ERR_INVALID;
    if (a->B > 1 && a->ldo < (int64_t)d.n_heads * d.head_dim) return ET_ERR_INVALID;  // rows of the output would overlap
    if (!(scale >= 0.f) || !(scale * 1.4426950408889634 <= FLT_MAX)) return ET_ERR_INVALID;  // the kernel's scale is log2(e) of it
    if (accumulate && (!pool->acc || !kv->scores)) return ET_ERR_INVALID;
    KV_TRY(not_pending(kv));
    OnDevice on(d.device);
    if (!on.ok) return ET_ERR_CUDA;
    p.ctl = kv->ctl;
    p.lens = a->lens;
    p.q = a->q;
    p.out = a->out;
    p.lse = a->lse;
    p.ldq = a->ldq;
    p.ldo = a->ldo;
    p.scale_log2 = (float)((scale > 0.f ? (double)scale : 1.0 / sqrt((double)d.head_dim)) * 1.4426950408889634);
    p.B = a->B;
    p.n_q = d.n_heads;
    p.n_kv = d.n_kv_heads;
    p.group = d.n_heads / d.n_kv_heads;
    p.n_qt = kv->n_qt;
    // the rounded-up reciprocal is exact: i < 2^21 + 8, page_groups <= 512 (1 has none in 32 bits and needs none)
    p.page_groups = d.page_size % 8 ? 0 : d.page_size / 8;
    p.page_magic = p.page_groups > 1 ? (unsigned)(((1ull << 32) + p.page_groups - 1) / p.page_groups) : 0;
    p.warp_share_log = p.cta_share_log = kKvShareLog;
    p.warp_parts = kKvWarpParts;
    p.warp_extra = kKvWarpExtra;
    p.cta_extra = kv_cta_extra(d.head_dim * kv->ces);
    p.part = kv->part;
    p.part_ml = kv->part_ml;
    p.arrivals = kv->arrivals;
    p.group_slots = kv->group_slots;
    p.arrivals_ld = kv->arrivals_ld;
    p.scores = accumulate ? kv->scores : nullptr;
    p.row_ml = kv->row_ml;
    p.ctx_pad = kv->ctx_pad;
    cudaStream_t s = (cudaStream_t)stream;
    KV_CU(attn_of(d)(&p, d.dtype, d.cache_dtype, p.group, kv->n_sm, s));
    if (accumulate) {
        KvWeightParams wp;
        wp.pool = p.pool;
        wp.table = p.table;
        wp.lens = a->lens;
        wp.scores = kv->scores;
        wp.row_ml = kv->row_ml;
        wp.B = a->B;
        wp.n_q = p.n_q;
        wp.n_kv = p.n_kv;
        wp.group = p.group;
        wp.ctx_pad = kv->ctx_pad;
        KV_CU(launch_kv_weights(wp, kv->ctl, kv->n_sm, s));
    }
    return ET_OK;
}

et_status et_run_kv_evict(et_kv* kv, const et_kv_pool* pool, const et_kv_evict_args* a, void* stream) {
    KvEvictParams p;
    KV_TRY(take_pool(kv, pool, &p.pool));
    if (!a) return ET_ERR_INVALID;
    KV_TRY(take_table(kv, a->B, a->table, a->ld_table, &p.src));
    KV_TRY(take_table(kv, a->B, a->dst_table, a->ld_dst, &p.dst));
    if (!pool->acc || !al4(a->lens) || !al4(a->new_lens) || !al4(a->kept)) return ET_ERR_INVALID;
    if (a->budget < 1 || a->n_recent < 0 || a->n_sink < 0 || a->n_recent > a->budget || a->n_sink > a->budget - a->n_recent)
        return ET_ERR_INVALID;
    // the slots that can stay have to fit the destination
    if (std::min(a->budget, p.src.max_len) > (long long)a->ld_dst * kv->d.page_size) return ET_ERR_INVALID;
    p.in_place = a->dst_table == a->table;
    if (p.in_place && a->ld_dst != a->ld_table) return ET_ERR_INVALID;
    KV_TRY(not_pending(kv));
    OnDevice on(kv->d.device);
    if (!on.ok) return ET_ERR_CUDA;
    p.ctl = kv->ctl;
    p.lens = a->lens;
    p.new_lens = a->new_lens;
    p.new_count = kv->new_count;
    p.kept = a->kept;
    p.owner = kv->owner;
    p.B = a->B;
    p.n_kv = kv->d.n_kv_heads;
    p.budget = a->budget;
    p.n_recent = a->n_recent;
    p.n_sink = a->n_sink;
    p.row_bytes = kv->d.head_dim * kv->ces;
    p.elem_bytes = kv->ces;
    p.page_shift = (kv->d.page_size & (kv->d.page_size - 1)) ? -1 : __builtin_ctz(kv->d.page_size);
    p.fours = kv->d.page_size % 4 == 0 && al16(pool->acc);
    KV_CU(launch_kv_evict(p, kv->n_sm, (cudaStream_t)stream));
    return ET_OK;
}

et_status et_sync_kv(et_kv* kv, void* stream, int32_t* diag4) {
    if (!kv) return ET_ERR_INVALID;
    OnDevice on(kv->d.device);
    if (!on.ok) return ET_ERR_CUDA;
    KV_CU(cudaStreamSynchronize((cudaStream_t)stream));
    KvCtl h;
    KV_CU(cudaMemcpy(&h, kv->ctl, sizeof(h), cudaMemcpyDeviceToHost));
    if (diag4) memcpy(diag4, h.diag, 4 * sizeof(int32_t));
    if (h.status == 0) return ET_OK;
    KV_CU(cudaDeviceSynchronize());
    KV_TRY(reset_ctl(kv));
    KV_CU(cudaMemset(kv->arrivals, 0, kv->n_arrivals * sizeof(int)));
    KV_CU(cudaMemset(kv->owner, 0, (size_t)kv->d.n_pages * sizeof(unsigned long long)));
    KV_CU(cudaDeviceSynchronize());
    return (et_status)h.status;
}

}  // extern "C"
