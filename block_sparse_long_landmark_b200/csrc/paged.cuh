// paged.cuh -- shared pieces of the paged 8-bit key/value cache: the resolved
// shape of a call, code <-> value conversions, and the internal launchers.
//
// A page holds `bs` tokens of every kv-head: codes [pages][Hkv][bs][d], one
// byte each, and one fp32 scale per (page, head) for the keys and one for the
// values.  A cached value is code * scale.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace sa {

// Status bits of the paged calls besides those of common.cuh.
constexpr unsigned kStatusPool = 16u;   // block tables: pages or slots ran out

struct PagedShape {
    int B, Hq, Hkv, G, d, bs, pages, maxb, tokens, cap, flags, dtype, code;
    int Hsel;        // heads that own a kept list (Hkv, or Hq with SA_SELECT_PER_QHEAD)
    int heads_per;   // query heads that share one list
    float scale;
};

// Softmax weights of the tensor-core forms are fp16, 2^(z - reference).  The
// reference is raised only when a logit passes it by kWeightLift + kWeightSlack,
// to kWeightLift below that logit: weights stay below 2^15 (fp16 holds 2^16), and
// one that falls below fp16's normal range is off by 2^-25 2^-kWeightLift = 2^-32
// of the row's largest at most.  With the reference at the largest logit (2^-25)
// a row whose weight lies on one key without a value (a sink) lost what the
// others left of it: all of it at 2^-27.  No instruction more.
constexpr float kWeightLift = 7.f, kWeightSlack = 8.f;

// Cache length of sequence b, clamped to [0, maxb * bs].
__device__ __forceinline__ int paged_len(const PagedShape &s, const int32_t *seq_len, int b) {
    return min(max(seq_len[b], 0), s.maxb * s.bs);
}

// Four codes of one word as fp32, in byte order (exact; the NaN patterns of
// e4m3, which the append never writes, are NaN).
template <int kCode>
__device__ __forceinline__ void code_values4(uint32_t w, float *f) {
    if (kCode == SA_E4M3) {
        uint32_t lo, hi;
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}" : "=r"(lo), "=r"(hi) : "r"(w));
        const float2 a = __half22float2(*reinterpret_cast<__half2 *>(&lo));
        const float2 b = __half22float2(*reinterpret_cast<__half2 *>(&hi));
        f[0] = a.x;
        f[1] = a.y;
        f[2] = b.x;
        f[3] = b.y;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = (float)(signed char)((w >> (8 * i)) & 0xffu);
    }
}
template <int kCode>
__device__ __forceinline__ float code_value(unsigned byte) {
    float f[4];
    code_values4<kCode>(byte, f);
    return f[0];
}
// Two finite values rounded to codes (nearest, ties to even; saturating), the
// first in the low byte.
template <int kCode>
__device__ __forceinline__ uint32_t codes_of2(float a, float b) {
    if (kCode == SA_E4M3) {
        uint16_t r;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
        return r;
    }
    const int x = __float2int_rn(fminf(fmaxf(a, -127.f), 127.f));
    const int y = __float2int_rn(fminf(fmaxf(b, -127.f), 127.f));
    return (uint32_t)(x & 0xff) | ((uint32_t)(y & 0xff) << 8);
}


cudaError_t launch_paged_tables(const PagedShape &s, const int32_t *cur, const int32_t *want, int32_t *free_pages,
                                const int32_t *n_free, int32_t *n_free_out, int32_t *table, int32_t *cu,
                                int64_t *slot, unsigned *status, cudaStream_t st);
cudaError_t launch_paged_append(const PagedShape &s, const void *K, const void *V, long long tok_stride,
                                long long head_stride, const int64_t *slot, const int32_t *cu, const int32_t *new_len,
                                uint8_t *K8, uint8_t *V8, float *ks, float *vs, void *L, unsigned *status,
                                cudaStream_t st);
cudaError_t launch_paged_gather(const PagedShape &s, const int64_t *slot, const uint8_t *K8, const uint8_t *V8,
                                const float *ks, const float *vs, void *K, void *V, long long tok_stride,
                                long long head_stride, unsigned *status, cudaStream_t st);

// What the attention over the cache reads.
struct PagedCache {
    const uint8_t *K, *V;
    const float *ks, *vs;
    const int32_t *table;     // [B][maxb]
    const int32_t *seq_len;   // [B]
};
// Kept lists of a decode (idx null: every block of the sequence).
struct PagedLists {
    const int32_t *idx;
    const float *score;
    const int32_t *count;
};
// One query per sequence (cu null), or packed chunk rows (cu given, no lists).
cudaError_t launch_paged_simt(const PagedShape &s, const void *q, const int32_t *cu, const PagedCache &c,
                              const PagedLists &l, void *o, float *lse, unsigned *status, cudaStream_t st);

// The tensor-core decode: bf16, `scratch` of paged_decode_scratch bytes.  With
// cu it takes packed chunks (no lists): the sequences of up to
// paged_rows_limit rows a kv-head (0: none, INT_MAX: all of them).
bool paged_decode_supported(const PagedShape &s);
// `least`: the lowest limit that a call has whose shape differs in its tables'
// length only.
int paged_rows_limit(const PagedShape &s, bool least = false);
size_t paged_decode_scratch(const PagedShape &s, bool chunk);
cudaError_t launch_paged_decode(const PagedShape &s, const void *q, const int32_t *cu, const PagedCache &c,
                                const PagedLists &l, void *o, float *lse, unsigned *status, void *scratch,
                                cudaStream_t st);
// The tensor-core chunk attention: bf16, up to 128 query heads per kv-head; the
// sequences of more than `few` rows a kv-head.
bool paged_prefill_supported(const PagedShape &s);
size_t paged_prefill_scratch(const PagedShape &s);
cudaError_t launch_paged_prefill(const PagedShape &s, const void *Q, const int32_t *cu, const PagedCache &c, void *O,
                                 float *lse, int few, unsigned *status, void *scratch, cudaStream_t st);

}  // namespace sa
