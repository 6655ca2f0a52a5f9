// paged_api.cu -- the C ABI of the paged KV cache (include/vc.h): argument checks and launches.
#include <cuda_runtime.h>
#include <limits.h>

#include "../../include/vc.h"
#include "paged.cuh"

namespace vc {

vc_status record_cuda_failure(cudaError_t e, const char* where);

static bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
static bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }
static size_t up256(size_t v) { return (v + 255) / 256 * 256; }

bool paged_sizes_ok(const vc_paged_kv& c) {
    if (c.layers < 1 || c.pages < 1 || c.kv_heads < 1 || c.q_heads < 1 || c.q_heads % c.kv_heads || c.seqs < 1 ||
        c.columns < 1 || c.window < 0 || c.sinks < 0)
        return false;
    if (c.page_size < 16 || c.page_size > 256 || (c.page_size & (c.page_size - 1))) return false;
    if (c.head_dim != 32 && c.head_dim != 64 && c.head_dim != 128 && c.head_dim != 256) return false;
    const long long lim = INT_MAX;
    return (long long)c.columns * c.page_size <= (1 << 30) && (long long)c.seqs * c.columns <= lim &&
           (long long)c.seqs * c.kv_heads <= lim && (long long)c.kv_heads * c.page_size <= lim &&
           (long long)c.pages * c.kv_heads * c.page_size <= lim && (long long)c.q_heads * c.head_dim <= lim;
}

PagedWorkspace paged_carve(const vc_paged_kv& c, void* base) {
    PagedWorkspace w{};
    size_t off = 0;
    auto take = [&](size_t bytes) {
        uint8_t* p = (uint8_t*)base + off;
        off = up256(off + bytes);
        return p;
    };
    w.head = (int*)take(256);
    w.ticket = (int*)take(256);
    w.merge = (int*)take((size_t)kMaxSplitCtas * 4);
    w.copies = (int*)take((size_t)c.seqs * 12);
    w.ok = (int*)take((size_t)c.seqs * 4);
    w.first = (int*)take((size_t)c.seqs * 4);
    w.rows = (int4*)take((size_t)c.seqs * 16);
    w.need = (int*)take((size_t)c.seqs * 8);
    w.chunk_live = (int*)take(((size_t)c.pages / kCompactChunk + 1) * 4);
    w.rename = (int*)take((size_t)c.pages * 4);
    w.moves = (int*)take((size_t)c.pages * 8);
    w.partial = (float*)take((size_t)(c.head_dim == 64 ? kRecordRows64 : kRecordRows) * (c.head_dim + 2) * 4);
    w.bytes = off;
    return w;
}

PagedKv paged_kernel_kv(const vc_paged_kv& c) {
    PagedKv d{};
    d.k = (uint16_t*)c.k; d.v = (uint16_t*)c.v;
    d.table = c.table; d.len = c.len; d.refs = c.refs; d.status = c.status;
    d.layers = c.layers; d.pages = c.pages; d.page = c.page_size; d.page_shift = __builtin_ctz((unsigned)c.page_size);
    d.Hk = c.kv_heads; d.Dh = c.head_dim; d.Hq = c.q_heads; d.seqs = c.seqs; d.columns = c.columns;
    // positions are below 2^30: a window or sinks of that many cover all, and differences of positions stay in 32 bits
    d.window = c.window < (1 << 30) ? c.window : 1 << 30;
    d.sinks = c.sinks < (1 << 30) ? c.sinks : 1 << 30;
    return d;
}

bool paged_kv_ok(const vc_paged_kv* c) {
    return c && paged_sizes_ok(*c) && c->k && c->v && c->table && c->len && c->refs && c->status && c->workspace &&
           aligned16(c->k) && aligned16(c->v) && aligned16(c->table) && aligned16(c->len) && aligned16(c->refs) &&
           aligned4(c->status) && aligned16(c->workspace) && c->workspace_bytes >= paged_carve(*c, nullptr).bytes;
}

static float scale_to_log2(float scale, int head_dim) {
    return (scale != 0.0f ? scale : 1.0f / sqrtf((float)head_dim)) * 1.4426950408889634f;
}

PagedAttnArgs paged_rows(const uint16_t* qkv, int ld, int Hq, int Hk, int Dh, uint16_t* out, int out_ld, int widen, int pdl) {
    PagedAttnArgs a{};
    a.q = qkv; a.kn = qkv + (size_t)Hq * Dh; a.vn = a.kn + (size_t)Hk * Dh; a.out = out;
    a.q_ld = a.k_ld = a.v_ld = ld; a.out_ld = out_ld;
    a.scale_log2 = scale_to_log2(0.0f, Dh);
    a.widen = widen;
    a.pdl = pdl;
    return a;
}

cudaError_t paged_attend(const vc_paged_kv& kv, int layer, PagedAttnArgs a, cudaStream_t s) {
    a.c = paged_kernel_kv(kv);
    const size_t lay = (size_t)layer * kv.pages * kv.kv_heads * kv.page_size * kv.head_dim;
    a.c.k += lay; a.c.v += lay;
    a.f16 = kv.f16 != 0;
    const PagedWorkspace w = paged_carve(kv, kv.workspace);
    a.merge = w.merge;
    a.ticket = w.ticket;
    a.partial = w.partial;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&a.num_sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (a.num_sms > kMaxSms) a.num_sms = kMaxSms;
    if (!a.cu_rows) {
        e = launch_paged_frames(a, s);
        if (e != cudaErrorNotSupported) return e;
    }
    if (a.kn && (e = launch_paged_append(a, s)) != cudaSuccess) return e;
    if (a.cu_rows) {
        e = launch_paged_prompts(a, s);
        if (e != cudaErrorNotSupported) return e;
    }
    return launch_paged_tiles(a, s);
}

}  // namespace vc

using namespace vc;

#define CKP(call)                                                        \
    do {                                                                 \
        cudaError_t e_ = (call);                                         \
        if (e_ != cudaSuccess) return record_cuda_failure(e_, __func__); \
    } while (0)

extern "C" size_t vc_paged_workspace_bytes(const vc_paged_kv* kv) {
    if (!kv || !paged_sizes_ok(*kv)) return 0;
    return paged_carve(*kv, nullptr).bytes;
}

extern "C" vc_status vc_paged_resize(const vc_paged_kv* kv, int n, const int32_t* seqs, const int32_t* lens, int add,
                                     int32_t* pos, vc_stream_t stream) {
    if (!paged_kv_ok(kv) || n < 1 || n > kv->seqs || !aligned4(seqs) || !aligned4(lens) || !aligned4(pos))
        return VC_ERR_INVALID_ARG;
    CKP(launch_paged_resize(paged_kernel_kv(*kv), paged_carve(*kv, kv->workspace), n, seqs, lens, add, pos,
                            1, (cudaStream_t)stream));
    return VC_OK;
}

extern "C" vc_status vc_paged_fork(const vc_paged_kv* kv, int n, const int32_t* src, const int32_t* dst,
                                   const vc_session_part* parts, int n_parts, int32_t* done, vc_stream_t stream) {
    if (!paged_kv_ok(kv) || n < 1 || n > kv->seqs || !src || !dst || !aligned4(src) || !aligned4(dst) || !aligned4(done))
        return VC_ERR_INVALID_ARG;
    if (n_parts < 0 || n_parts > 8 || (n_parts && !parts)) return VC_ERR_INVALID_ARG;
    for (int i = 0; i < n_parts; ++i) {
        const vc_session_part& p = parts[i];
        if (!p.base || !aligned16(p.base) || p.bytes < 4 || p.bytes % 4 || p.outer < 1) return VC_ERR_INVALID_ARG;
        if (p.stride < p.bytes || p.stride % 4 || p.outer_stride % 4) return VC_ERR_INVALID_ARG;
        // a session's block of one outer index may not reach into the next one's
        if (p.outer > 1 && p.outer_stride < (int64_t)(kv->seqs - 1) * p.stride + p.bytes) return VC_ERR_INVALID_ARG;
    }
    CKP(launch_paged_fork(paged_kernel_kv(*kv), paged_carve(*kv, kv->workspace), n, src, dst, parts, n_parts, done,
                          (cudaStream_t)stream));
    return VC_OK;
}

extern "C" vc_status vc_paged_compact(const vc_paged_kv* kv, int32_t* live, vc_stream_t stream) {
    if (!paged_kv_ok(kv) || !aligned4(live)) return VC_ERR_INVALID_ARG;
    CKP(launch_paged_compact(paged_kernel_kv(*kv), paged_carve(*kv, kv->workspace), live, (cudaStream_t)stream));
    return VC_OK;
}

extern "C" vc_status vc_paged_attend(const vc_paged_kv* kv, int layer, const vc_attn_rows* rows, vc_stream_t stream) {
    if (!paged_kv_ok(kv) || !rows || layer < 0 || layer >= kv->layers) return VC_ERR_INVALID_ARG;
    const vc_attn_rows& r = *rows;
    if (!r.q || !r.out || !r.pos || (!r.k != !r.v) || r.batch < 1 || r.batch > kv->seqs || r.rows < 1 ||
        (!r.cu_rows && r.rows != r.batch))
        return VC_ERR_INVALID_ARG;
    const int64_t qw = (int64_t)kv->q_heads * kv->head_dim, kw = (int64_t)kv->kv_heads * kv->head_dim;
    if (!aligned16(r.q) || !aligned16(r.out) || !aligned16(r.k) || !aligned16(r.v) || !aligned4(r.seqs) ||
        !aligned4(r.pos) || !aligned4(r.cu_rows) || r.q_stride < qw || r.out_stride < qw || r.q_stride % 8 ||
        r.out_stride % 8)
        return VC_ERR_INVALID_ARG;
    if (r.k && (r.k_stride < kw || r.v_stride < kw || r.k_stride % 8 || r.v_stride % 8)) return VC_ERR_INVALID_ARG;
    if (!(r.scale > -3e38f && r.scale < 3e38f)) return VC_ERR_INVALID_ARG;   // NaN and infinities
    const int group = kv->q_heads / kv->kv_heads;
    if ((long long)r.rows * group > INT_MAX - 4096) return VC_ERR_INVALID_ARG;
    PagedAttnArgs a{};
    a.q = (const uint16_t*)r.q; a.kn = (const uint16_t*)r.k; a.vn = (const uint16_t*)r.v; a.out = (uint16_t*)r.out;
    a.q_ld = r.q_stride; a.k_ld = r.k_stride; a.v_ld = r.v_stride; a.out_ld = r.out_stride;
    a.seqs = r.seqs; a.pos = r.pos; a.cu_rows = r.cu_rows;
    a.batch = r.batch; a.rows = r.rows;
    a.scale_log2 = scale_to_log2(r.scale, kv->head_dim);
    a.pdl = 1;
    CKP(paged_attend(*kv, layer, a, (cudaStream_t)stream));
    return VC_OK;
}
