// paged_attend.cu -- attention over the paged 8-bit cache on the CUDA cores:
// every type, head size, block size and mode, in fp32.
//
// One CTA of four warps per (query row, query head).  The warps take the
// row's blocks in turn; in a block each lane owns a key (its dot product runs
// over the query in shared memory), the block's 32-key steps update an online
// softmax, and for P V each lane owns d / 32 dimensions.  A value's scale
// multiplies its weight, a key's its logit, so codes are never rescaled.
// Hierarchical mode keeps a second state per block, folded in with weight
// 2^score at the block's end.  Latency bound: it is the form for fp32 and for
// shapes the tensor-core kernels do not take.
#include <math_constants.h>

#include "paged.cuh"

namespace sa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct SimtArgs {
    PagedShape s;
    PagedCache c;
    PagedLists l;
    const int32_t *cu;      // packed chunk rows, or null: one row per sequence
    unsigned *status;
};

template <int kD>
struct State {
    float m, l, acc[kD / 32];
    __device__ __forceinline__ void reset() {
        m = -CUDART_INF_F;
        l = 0.f;
#pragma unroll
        for (int i = 0; i < kD / 32; ++i) acc[i] = 0.f;
    }
    // raises the reference to nm (log2 units) and returns the factor applied
    __device__ __forceinline__ void raise(float nm) {
        const float f = m == -CUDART_INF_F ? 0.f : exp2f(m - nm);
        m = nm;
        l *= f;
#pragma unroll
        for (int i = 0; i < kD / 32; ++i) acc[i] *= f;
    }
};

__device__ __forceinline__ int row_owner(const int32_t *cu, int B, int r) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (cu[m] <= r) lo = m;
        else hi = m;
    }
    return lo;
}

template <typename T, int kCode, int kD>
__global__ void __launch_bounds__(128)
paged_simt_kernel(SimtArgs a, const T *__restrict__ q, T *__restrict__ o, float *__restrict__ lse) {
    constexpr int DL = kD / 32;
    const PagedShape &s = a.s;
    __shared__ float qs[kD];
    __shared__ float sm_m[4], sm_l[4], sm_acc[4][kD];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int r = blockIdx.x, h = blockIdx.y, g = h / s.G;
    int b = r, keys;
    if (a.cu) {
        // offsets that do not ascend within the rows: nothing is done
        int bad = 0;
        for (int i = tid; i < s.B; i += 128)
            bad |= !(a.cu[i] >= 0 && a.cu[i] <= a.cu[i + 1] && a.cu[i + 1] <= s.tokens);
        if (__syncthreads_or(bad)) {
            if (tid == 0) set_status(a.status, kStatusBadIndex);
            return;
        }
        if (r < a.cu[0] || r >= a.cu[s.B]) return;      // rows of no sequence stay as they are
        b = row_owner(a.cu, s.B, r);
        const int n = paged_len(s, a.c.seq_len, b);
        keys = s.flags & SA_CAUSAL ? max(0, n - (a.cu[b + 1] - r) + 1) : n;
        keys = min(keys, n);
    } else {
        keys = paged_len(s, a.c.seq_len, b);
    }
    for (int i = tid; i < kD; i += 128) qs[i] = to_f(q[((size_t)r * s.Hq + h) * kD + i]) * s.scale * kLog2e;
    __syncthreads();
    const int blocks = (keys + s.bs - 1) / s.bs, local = blocks - 1;
    const bool hier = s.flags & SA_HIER;
    const int32_t *il = nullptr;
    const float *sc = nullptr;
    int cnt = blocks;
    float s_loc = 0.f;
    if (a.l.idx) {
        const size_t u = (size_t)b * s.Hsel + (s.flags & SA_SELECT_PER_QHEAD ? h : g);
        il = a.l.idx + u * s.cap;
        sc = a.l.score + u * s.cap;
        cnt = keys > 0 ? max(0, min(a.l.count[u], s.cap)) : 0;
        s_loc = cnt > 0 ? sc[cnt - 1] : 0.f;
    }
    State<kD> run, blkst;
    run.reset();
    for (int e = warp; e < cnt; e += 4) {
        const int blk = il ? il[e] : e;
        bool good = blk >= 0 && blk <= local && !(il && e > 0 && il[e - 1] >= blk);
        const int page = good ? a.c.table[(size_t)b * s.maxb + blk] : -1;
        good = good && page >= 0 && page < s.pages;
        if (!good) {
            if (lane == 0) set_status(a.status, kStatusBadIndex);
            continue;
        }
        const bool forced = (blk == local && (s.flags & SA_LOCAL)) || (blk == 0 && (s.flags & SA_SINK));
        const float gate = il && (s.flags & SA_GATE) && !forced ? log_sigmoid(sc[e] - s_loc) * kLog2e : 0.f;
        const size_t ph = (size_t)page * s.Hkv + g;
        const float ksc = a.c.ks[ph], vsc = a.c.vs[ph];
        const uint8_t *kb = a.c.K + ph * s.bs * kD, *vb = a.c.V + ph * s.bs * kD;
        const int nk = min(s.bs, keys - blk * s.bs);
        State<kD> &st = hier ? blkst : run;
        if (hier) blkst.reset();
        for (int k0 = 0; k0 < nk; k0 += 32) {
            const int key = k0 + lane;
            float z = -CUDART_INF_F;
            if (key < nk) {
                float dot = 0.f;
                const uint4 *kr = reinterpret_cast<const uint4 *>(kb + (size_t)key * kD);
#pragma unroll
                for (int c = 0; c < kD / 16; ++c) {
                    const uint4 u = kr[c];
                    float f[16];
                    code_values4<kCode>(u.x, f);
                    code_values4<kCode>(u.y, f + 4);
                    code_values4<kCode>(u.z, f + 8);
                    code_values4<kCode>(u.w, f + 12);
#pragma unroll
                    for (int i = 0; i < 16; ++i) dot = fmaf(f[i], qs[16 * c + i], dot);
                }
                z = fmaf(dot, ksc, gate);
            }
            float mx = z;
#pragma unroll
            for (int w = 16; w; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, w));
            if (mx > st.m) st.raise(mx);
            const float p = exp2f(z - (st.m == -CUDART_INF_F ? 0.f : st.m));
            float ps = p;
#pragma unroll
            for (int w = 16; w; w >>= 1) ps += __shfl_xor_sync(~0u, ps, w);
            st.l += ps;
            const int nn = min(32, nk - k0);
            for (int j = 0; j < nn; ++j) {
                const float w = __shfl_sync(~0u, p, j) * vsc;
                const uint8_t *vr = vb + (size_t)(k0 + j) * kD + lane * DL;
#pragma unroll
                for (int i = 0; i < DL; ++i) st.acc[i] = fmaf(w, code_value<kCode>(vr[i]), st.acc[i]);
            }
        }
        // no key (NaN goes on), or no weight
        if (hier && blkst.l != 0.f && sc[e] != -CUDART_INF_F) {
            const float w2 = sc[e] * kLog2e;
            if (w2 > run.m) run.raise(w2);
            const float w = exp2f(w2 - run.m);
            run.l += w;
#pragma unroll
            for (int i = 0; i < DL; ++i) run.acc[i] += w / blkst.l * blkst.acc[i];
        }
    }
    if (lane == 0) {
        sm_m[warp] = run.m;
        sm_l[warp] = run.l;
    }
#pragma unroll
    for (int i = 0; i < DL; ++i) sm_acc[warp][lane * DL + i] = run.acc[i];
    __syncthreads();
    const float M = fmaxf(fmaxf(sm_m[0], sm_m[1]), fmaxf(sm_m[2], sm_m[3]));
    float f[4], lt = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        f[w] = sm_m[w] == -CUDART_INF_F ? 0.f : exp2f(sm_m[w] - M);
        lt += sm_l[w] * f[w];
    }
    const float inv = lt > 0.f ? 1.f / lt : 0.f;
    for (int i = tid; i < kD; i += 128) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < 4; ++w) x += f[w] == 0.f ? 0.f : sm_acc[w][i] * f[w];
        from_f(o[((size_t)r * s.Hq + h) * kD + i], lt == 0.f ? 0.f : lt == lt ? x * inv : lt);
    }
    if (tid == 0) lse[(size_t)r * s.Hq + h] = lt == 0.f ? -CUDART_INF_F : (M + log2f(lt)) * kLn2;
}

template <typename T, int kCode>
cudaError_t run(const SimtArgs &a, const void *q, void *o, float *lse, cudaStream_t st) {
    const dim3 grid((unsigned)(a.cu ? a.s.tokens : a.s.B), (unsigned)a.s.Hq);
    if (grid.x == 0) return cudaSuccess;
    auto k = a.s.d == 128 ? paged_simt_kernel<T, kCode, 128> : paged_simt_kernel<T, kCode, 64>;
    k<<<grid, 128, 0, st>>>(a, (const T *)q, (T *)o, lse);
    note_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_simt(const PagedShape &s, const void *q, const int32_t *cu, const PagedCache &c,
                              const PagedLists &l, void *o, float *lse, unsigned *status, cudaStream_t st) {
    const SimtArgs a{s, c, l, cu, status};
    if (s.dtype == SA_BF16)
        return s.code == SA_E4M3 ? run<__nv_bfloat16, SA_E4M3>(a, q, o, lse, st)
                                 : run<__nv_bfloat16, SA_INT8>(a, q, o, lse, st);
    return s.code == SA_E4M3 ? run<float, SA_E4M3>(a, q, o, lse, st) : run<float, SA_INT8>(a, q, o, lse, st);
}

}  // namespace sa
