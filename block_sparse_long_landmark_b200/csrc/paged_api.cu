// paged_api.cu -- the C entry points of the paged 8-bit cache: argument
// checks, workspace sizing, dispatch.  See include/sparse_attn.h.
#include <limits.h>
#include <math.h>

#include "paged.cuh"

using namespace sa;

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }

int resolve_paged(const sa_paged_params *p, PagedShape &s) {
    if (!p) return SA_ERR_ARG;
    if (p->B <= 0 || p->Hq <= 0 || p->Hkv <= 0 || p->block <= 0 || p->pages <= 0 || p->max_blocks <= 0 ||
        p->tokens < 0)
        return SA_ERR_ARG;
    if (p->Hq % p->Hkv) return SA_ERR_ARG;
    if (p->dtype != SA_BF16 && p->dtype != SA_FP32) return SA_ERR_ARG;
    if (p->code != SA_E4M3 && p->code != SA_INT8) return SA_ERR_ARG;
    if (p->top_k < 0 || p->top_k > 256) return SA_ERR_ARG;
    if (p->flags & ~(SA_SINK | SA_LOCAL | SA_GATE | SA_HIER | SA_CAUSAL | SA_SELECT_PER_QHEAD)) return SA_ERR_ARG;
    if (!(p->scale >= 0.f) || isinf(p->scale)) return SA_ERR_ARG;
    if (p->d != 64 && p->d != 128) return SA_ERR_UNSUPPORTED;
    if (p->block < 16 || p->block > 128 || p->block % 16) return SA_ERR_UNSUPPORTED;
    if ((p->flags & SA_GATE) && (p->flags & SA_HIER)) return SA_ERR_UNSUPPORTED;
    if ((p->flags & SA_GATE) && !(p->flags & SA_LOCAL)) return SA_ERR_UNSUPPORTED;
    // one launch dimension per head, three offsets per sequence in shared memory
    if (p->B > 16384 || p->Hq > 65535) return SA_ERR_UNSUPPORTED;
    const long long most = (1ll << 31) - 1;
    if ((long long)p->pages * p->block * p->Hkv > most || (long long)p->B * p->max_blocks > most ||
        (long long)p->max_blocks * p->block > most - 256 || (long long)p->B * p->Hq * (p->top_k + 2) > most ||
        p->tokens > most - 256)
        return SA_ERR_UNSUPPORTED;
    s.B = p->B;
    s.Hq = p->Hq;
    s.Hkv = p->Hkv;
    s.G = p->Hq / p->Hkv;
    s.d = p->d;
    s.bs = p->block;
    s.pages = p->pages;
    s.maxb = p->max_blocks;
    s.tokens = p->tokens;
    s.cap = p->top_k + 2;
    s.flags = p->flags;
    s.dtype = p->dtype;
    s.code = p->code;
    const bool perq = p->flags & SA_SELECT_PER_QHEAD;
    s.Hsel = perq ? p->Hq : p->Hkv;
    s.heads_per = perq ? 1 : s.G;
    s.scale = p->scale > 0.f ? p->scale : 1.0f / sqrtf((float)p->d);
    return SA_OK;
}

// Strides of packed rows: dense when both are 0, else rows and heads must not
// overlap and every row must start on 16 bytes.
int resolve_strides(const PagedShape &s, long long &ts, long long &hs) {
    if (ts == 0 && hs == 0) {
        hs = s.d;
        ts = (long long)s.Hkv * s.d;
        return SA_OK;
    }
    const long long per16 = s.dtype == SA_BF16 ? 8 : 4;
    if (ts < s.d || hs < s.d || ts % per16 || hs % per16) return SA_ERR_ARG;
    if (ts >= (1ll << 31) || hs >= (1ll << 31)) return SA_ERR_UNSUPPORTED;
    if (ts < (s.Hkv - 1) * hs + s.d && hs < (s.tokens - 1ll) * ts + s.d) return SA_ERR_ARG;
    return SA_OK;
}

}  // namespace

extern "C" {

size_t sparse_attn_paged_workspace_size(const sa_paged_params *p, int op) {
    PagedShape s;
    if (resolve_paged(p, s) != SA_OK) return 0;
    switch (op) {
        case SA_OP_PAGED_TABLES:
        case SA_OP_PAGED_APPEND:
        case SA_OP_PAGED_GATHER: return kStatusBytes;
        case SA_OP_PAGED_DECODE: return kStatusBytes + al256(paged_decode_scratch(s, false));
        case SA_OP_PAGED_PREFILL: {
            // one kernel after the other, in the same place
            const int few = paged_rows_limit(s, true);
            const size_t rows = few > 0 ? paged_decode_scratch(s, true) : 0;
            const size_t tiles = few < INT_MAX && s.tokens > 0 && paged_prefill_supported(s) ? paged_prefill_scratch(s) : 0;
            return kStatusBytes + al256(rows > tiles ? rows : tiles);
        }
        default: return 0;
    }
}

int sparse_attn_paged_tables(const sa_paged_params *p, const int32_t *cur_len, const int32_t *new_len,
                             int32_t *free_pages, const int32_t *n_free, int32_t *n_free_out, int32_t *table,
                             int32_t *cu, int64_t *slot, void *ws, size_t ws_bytes, void *stream) {
    PagedShape s;
    const int r = resolve_paged(p, s);
    if (r != SA_OK) return r;
    if (!cur_len || !new_len || !free_pages || !n_free || !n_free_out || !table || !cu || !ws) return SA_ERR_ARG;
    if (s.tokens > 0 && !slot) return SA_ERR_ARG;
    if (n_free == n_free_out || !aligned16(ws)) return SA_ERR_ARG;
    if (ws_bytes < kStatusBytes) return SA_ERR_WORKSPACE;
    return launch_result(launch_paged_tables(s, cur_len, new_len, free_pages, n_free, n_free_out, table, cu, slot,
                                             (unsigned *)ws, (cudaStream_t)stream));
}

int sparse_attn_paged_append(const sa_paged_params *p, const void *K, const void *V, long long tok_stride,
                             long long head_stride, const int64_t *slot, const int32_t *cu, const int32_t *new_len,
                             void *K8, void *V8, float *kscale, float *vscale, void *L, void *ws, size_t ws_bytes,
                             void *stream) {
    PagedShape s;
    int r = resolve_paged(p, s);
    if (r != SA_OK) return r;
    if ((r = resolve_strides(s, tok_stride, head_stride)) != SA_OK) return r;
    if (!K8 || !V8 || !kscale || !vscale || !ws) return SA_ERR_ARG;
    if (s.tokens > 0 && (!K || !V || !slot)) return SA_ERR_ARG;
    if (L && (!cu || !new_len)) return SA_ERR_ARG;
    if (!aligned16(K) || !aligned16(V) || !aligned16(K8) || !aligned16(V8) || !aligned16(L) || !aligned16(ws))
        return SA_ERR_ARG;
    if (ws_bytes < kStatusBytes) return SA_ERR_WORKSPACE;
    return launch_result(launch_paged_append(s, K, V, tok_stride, head_stride, slot, cu, new_len, (uint8_t *)K8,
                                             (uint8_t *)V8, kscale, vscale, L, (unsigned *)ws,
                                             (cudaStream_t)stream));
}

int sparse_attn_paged_gather(const sa_paged_params *p, const int64_t *slot, const void *K8, const void *V8,
                             const float *kscale, const float *vscale, void *K, void *V, long long tok_stride,
                             long long head_stride, void *ws, size_t ws_bytes, void *stream) {
    PagedShape s;
    int r = resolve_paged(p, s);
    if (r != SA_OK) return r;
    if ((r = resolve_strides(s, tok_stride, head_stride)) != SA_OK) return r;
    if (!K8 || !V8 || !kscale || !vscale || !ws) return SA_ERR_ARG;
    if (s.tokens > 0 && (!K || !V || !slot)) return SA_ERR_ARG;
    if (!aligned16(K) || !aligned16(V) || !aligned16(K8) || !aligned16(V8) || !aligned16(ws)) return SA_ERR_ARG;
    if (ws_bytes < kStatusBytes) return SA_ERR_WORKSPACE;
    return launch_result(launch_paged_gather(s, slot, (const uint8_t *)K8, (const uint8_t *)V8, kscale, vscale, K, V,
                                             tok_stride, head_stride, (unsigned *)ws, (cudaStream_t)stream));
}

int sparse_attn_paged_decode(const sa_paged_params *p, const void *q, const void *K8, const void *V8,
                             const float *kscale, const float *vscale, const int32_t *table, const int32_t *seq_len,
                             const int32_t *idx, const float *score, const int32_t *count, void *o, float *lse,
                             void *ws, size_t ws_bytes, void *stream) {
    PagedShape s;
    const int r = resolve_paged(p, s);
    if (r != SA_OK) return r;
    if (!q || !K8 || !V8 || !kscale || !vscale || !table || !seq_len || !o || !lse || !ws) return SA_ERR_ARG;
    const bool lists = idx != nullptr;
    if (lists != (score != nullptr) || lists != (count != nullptr)) return SA_ERR_ARG;
    // gates and block weights come from the lists' scores
    if (!lists && (s.flags & (SA_GATE | SA_HIER))) return SA_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(K8) || !aligned16(V8) || !aligned16(o) || !aligned16(ws)) return SA_ERR_ARG;
    if (ws_bytes < sparse_attn_paged_workspace_size(p, SA_OP_PAGED_DECODE)) return SA_ERR_WORKSPACE;
    const PagedCache c{(const uint8_t *)K8, (const uint8_t *)V8, kscale, vscale, table, seq_len};
    const PagedLists l{idx, score, count};
    if (paged_decode_supported(s))
        return launch_result(launch_paged_decode(s, q, nullptr, c, l, o, lse, (unsigned *)ws,
                                                 (unsigned char *)ws + kStatusBytes, (cudaStream_t)stream));
    return launch_result(launch_paged_simt(s, q, nullptr, c, l, o, lse, (unsigned *)ws, (cudaStream_t)stream));
}

int sparse_attn_paged_prefill(const sa_paged_params *p, const void *Q, const int32_t *cu, const void *K8,
                              const void *V8, const float *kscale, const float *vscale, const int32_t *table,
                              const int32_t *seq_len, void *O, float *lse, void *ws, size_t ws_bytes, void *stream) {
    PagedShape s;
    const int r = resolve_paged(p, s);
    if (r != SA_OK) return r;
    if (s.flags & (SA_GATE | SA_HIER)) return SA_ERR_UNSUPPORTED;
    if (!cu || !K8 || !V8 || !kscale || !vscale || !table || !seq_len || !ws) return SA_ERR_ARG;
    if (s.tokens > 0 && (!Q || !O || !lse)) return SA_ERR_ARG;
    if (!aligned16(Q) || !aligned16(K8) || !aligned16(V8) || !aligned16(O) || !aligned16(ws)) return SA_ERR_ARG;
    if (ws_bytes < sparse_attn_paged_workspace_size(p, SA_OP_PAGED_PREFILL)) return SA_ERR_WORKSPACE;
    if (s.tokens == 0) return SA_OK;
    const PagedCache c{(const uint8_t *)K8, (const uint8_t *)V8, kscale, vscale, table, seq_len};
    const int few = paged_rows_limit(s);
    if (few > 0) {
        const int done = launch_result(launch_paged_decode(s, Q, cu, c, PagedLists{}, O, lse, (unsigned *)ws,
                                                           (unsigned char *)ws + kStatusBytes, (cudaStream_t)stream));
        if (done != SA_OK || few == INT_MAX) return done;
    }
    if (paged_prefill_supported(s))
        return launch_result(launch_paged_prefill(s, Q, cu, c, O, lse, few, (unsigned *)ws,
                                                  (unsigned char *)ws + kStatusBytes, (cudaStream_t)stream));
    return launch_result(
        launch_paged_simt(s, Q, cu, c, PagedLists{}, O, lse, (unsigned *)ws, (cudaStream_t)stream));
}

}  // extern "C"
