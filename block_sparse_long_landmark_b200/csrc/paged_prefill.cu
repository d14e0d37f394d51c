// paged_prefill.cu -- packed chunks of queries over the paged 8-bit cache on
// the tensor cores (bf16, up to 128 query heads per kv-head).
//
//   S = q code_k^T,  p = 2^(scale log2e ks S - m),  O = sum (p vs) code_v / sum p
//
// A unit is up to 256 query rows of one (sequence, kv-head): tokens times the
// group's heads, so each cached tile of 128 keys is read and converted once
// for all of them.  The rows form two M = 128 tiles with their own softmax
// warpgroup, S and O in tensor memory; while one warpgroup works, the tensor
// core runs the other's products.  Tensor work 4 rows d flops a key against
// d conversions a key and d bytes: tensor and exponential bound at 256 rows,
// cache-read bound when a chunk has few.
//   * TMA brings a tile's codes from its pages to shared memory, and a
//     converter warpgroup makes fp16 of them, exactly and with one conversion
//     instruction per two codes (bf16 takes five).  The launch before has put
//     the queries into fp16, each row scaled by a power of two so that its
//     largest element lies in [2^14, 2^15): what falls below fp16's range is
//     under 2^-38 of it.  Scales stay out of the matrices: the key's and the
//     row's multiply the logit, the value's the weight;
//   * weights are rounded to fp16.  p vs spans the scales' range, so O has a
//     reference of its own: with m the row's largest logit and m' its largest
//     logit + log2 vs, less kWeightLift, l sums p = 2^(z - m) unrounded and the
//     tensor core gets p vs 2^(m - m'), below 2^15 whatever the scales (a
//     reference is raised once it is passed by 2^8 more than it was raised
//     for).  Rounding is off by half a step, 2^-11, of a p vs, or 2^-32 of the
//     row's largest where that is more;
//   * S of a key tile comes in two halves of 64 keys with a buffer each, so
//     the tensor core fills one while the softmax empties the other (one S of
//     128 keys left the softmax waiting 30 % of the time);
//   * the work is one line of (unit, key tile) steps cut into one equal range
//     per CTA, whatever the lengths: a few queries over a long cache spread
//     over every SM, and a causal triangle is balanced.  Units that ranges
//     share leave fp32 records (at most two a CTA), joined by a second launch.
//
// Warps: 0 takes segments from the line and loads Q by TMA, 1 owns tensor
// memory and issues the MMAs of Q tile 0, 3 those of Q tile 1 (one warp for
// both would hold one tile's products back while it waits, quarter by quarter,
// for the other's weights: 3.39 against 3.06 ms for a 4K chunk at 32K), 2
// loads codes and scales; 4-7 convert; 8-11 and 12-15 softmax.
// The warps' loops share the instruction caches, so code is kept short: with
// the issuers', converters', rescaling and epilogue loops unrolled, 114 KB, a 4K
// chunk at 32K took 2.32 ms and any line more or less moved it by 10 %; rolled,
// 78 KB, 2.1 to 2.2 ms, and it holds still.
// Registers: launched at 128; 112 + 112 + 2 * 144 = 4 * 128.
// Every wait is bounded; when one runs out the CTA sets the status word, lets
// its copies land, frees tensor memory and exits.
#include <math_constants.h>

#include "paged.cuh"
#include "tc_ptx.cuh"

namespace sa {
namespace {

using namespace tc;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kThreads = 512;
constexpr int kRegsLaunch = 128, kRegsIssue = 112, kRegsConv = 112, kRegsSoft = 144;
static_assert(128 * (kRegsIssue + kRegsConv + 2 * kRegsSoft) <= kThreads * kRegsLaunch, "register split");
constexpr int kMaxGrid = 148;
constexpr int kMinRange = 2;                 // key tiles: a shorter range is mostly fill and drain
constexpr uint32_t kChunk = 128 * 128;       // 128 rows x 64 bf16
constexpr int kStages = 2;
constexpr int kScaleSlots = 4;

// One step list entry: a unit's query rows; `pre` counts key tiles before it.
struct Tile {
    int b, t0, kt, pad;
    long long pre;
};
struct PlanHead {
    int n, pad;
    long long total;    // key tiles of one kv-head
};
// A unit that several ranges share: who it is and how many records it has.
struct Job {
    int n, row0, ntok, h;
};

struct PreArgs {
    PagedShape s;
    PagedCache c;
    const int32_t *cu;
    __nv_bfloat16 *O;
    float *lse;
    unsigned *status;
    PlanHead *head;
    Tile *tiles;
    int cap_tiles;
    Job *jobs;          // [grid]
    const __nv_bfloat16 *Q;
    __half *qh;         // [tokens][Hq][d] queries in fp16
    float *qf;          // [tokens][Hq] logit scale of a row of qh, log2 units
    float *rec;         // [grid][2][d + 3][256]: O, m, l, m'
    int tpt;            // tokens per 128-row tile
    int box;            // rows of one copy: 16 to 128 keys of one page
    int few;            // sequences of up to so many rows a kv-head are done elsewhere
};

struct Seg {
    int b, h, row0, ntok;    // first packed row, tokens
    int pos0, n;             // position of the first token, keys of the sequence
    int ta, tb;              // key tiles
    int nq;                  // 128-row tiles with tokens
    int out;                 // 0: whole unit, 1: record slot 0, 2: record slot 1
};

// ---------------------------------------------------------------------------
// CTA 0: the step list: units in order of (sequence, token), each with its
// number of key tiles and the tiles before it.  The others: fp16 queries.
// ---------------------------------------------------------------------------
__device__ __forceinline__ int last_le(const int *off, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (off[m] <= x) lo = m;
        else hi = m;
    }
    return lo;
}

__device__ __forceinline__ long long scan1024(long long v, long long *tmp, long long &total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(~0u, v, o);
        if (lane >= o) v += t;
    }
    if (lane == 31) tmp[w] = v;
    __syncthreads();
    long long add = 0;
    total = 0;
    for (int i = 0; i < 32; ++i) {
        const long long x = tmp[i];
        if (i < w) add += x;
        total += x;
    }
    __syncthreads();
    return v + add;
}

__device__ __forceinline__ void rows_of(const PreArgs &a, int b, int &r0, int &r1) {
    r0 = max(0, min(a.cu[b], a.s.tokens));
    r1 = max(r0, min(a.cu[b + 1], a.s.tokens));
}

// Units of a sequence's rows r0 .. r1 - 1.
__device__ __forceinline__ int units_in(const PreArgs &a, int r0, int r1) {
    return (long long)(r1 - r0) * a.s.G <= a.few ? 0 : (r1 - r0 + 2 * a.tpt - 1) / (2 * a.tpt);
}

__global__ void __launch_bounds__(1024)
paged_plan_kernel(PreArgs a) {
    extern __shared__ int off_s[];
    __shared__ long long tmp[32];
    __shared__ int bad_s;
    const PagedShape &s = a.s;
    const int tid = threadIdx.x, tpu = 2 * a.tpt;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (blockIdx.x > 0) {
        // a row per half warp or quarter: d / 8 lanes of eight elements
        const int lpr = s.d / 8, l = tid % lpr;
        const long long rows = (long long)max(0, min(a.cu[s.B], s.tokens)) * s.Hq;
        const long long step = (long long)(gridDim.x - 1) * (1024 / lpr);
        long long row = (long long)(blockIdx.x - 1) * (1024 / lpr) + tid / lpr;
        for (const long long end = (rows + 3) / 4 * 4; row < end; row += step) {   // whole warps
            const bool in = row < rows;
            uint4 x = make_uint4(0, 0, 0, 0);
            if (in) x = *reinterpret_cast<const uint4 *>(a.Q + row * s.d + 8 * l);
            unsigned big = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                    __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
            big = max(big & 0xffffu, big >> 16);
            for (int o = 1; o < lpr; o <<= 1) big = max(big, __shfl_xor_sync(~0u, big, o));
            const int up = max(-113, min(126, 14 - ((int)(big >> 7) - 127)));
            const float f = __uint_as_float((unsigned)(up + 127) << 23);
            float v[8];
            load16(reinterpret_cast<const __nv_bfloat16 *>(&x), v);
            __half2 h[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = __floats2half2_rn(v[2 * i] * f, v[2 * i + 1] * f);
            if (in) {
                *reinterpret_cast<uint4 *>(a.qh + row * s.d + 8 * l) = *reinterpret_cast<const uint4 *>(h);
                if (l == 0) a.qf[row] = s.scale * kLog2e * __uint_as_float((unsigned)(127 - up) << 23);
            }
        }
        return;
    }
    if (tid == 0) bad_s = 0;
    __syncthreads();
    const int share = (s.B + 1023) / 1024, b0 = min(s.B, tid * share), b1 = min(s.B, b0 + share);
    long long n = 0, total;
    for (int b = b0; b < b1; ++b) {
        int r0, r1;
        rows_of(a, b, r0, r1);
        n += units_in(a, r0, r1);
        if (!(a.cu[b] >= 0 && a.cu[b] <= a.cu[b + 1] && a.cu[b + 1] <= s.tokens)) bad_s = 1;
    }
    long long at = scan1024(n, tmp, total) - n;
    // offsets that do not ascend within the rows: nothing is done
    const bool bad = bad_s;
    for (int b = b0; b < b1; ++b) {
        int r0, r1;
        rows_of(a, b, r0, r1);
        off_s[b] = bad ? 0 : (int)at;
        at += units_in(a, r0, r1);
    }
    __syncthreads();
    const int units = bad ? 0 : (int)total;
    long long carry = 0;
    for (int i0 = 0; i0 < units; i0 += 1024) {
        const int i = i0 + tid;
        Tile t{};
        if (i < units) {
            t.b = last_le(off_s, s.B, i);
            t.t0 = (i - off_s[t.b]) * tpu;
            int r0, r1;
            rows_of(a, t.b, r0, r1);
            const int len = paged_len(s, a.c.seq_len, t.b);
            const int last = min(tpu, r1 - r0 - t.t0) + t.t0;    // tokens of the chunk up to the unit's end
            const int see = s.flags & SA_CAUSAL ? min(len, len - (r1 - r0) + last) : len;
            t.kt = max(1, (see + 127) / 128);
        }
        long long sum;
        const long long inc = scan1024(t.kt, tmp, sum);
        if (i < units) {
            t.pre = carry + inc - t.kt;
            a.tiles[i] = t;
        }
        carry += sum;
    }
    if (tid == 0) {
        *a.head = PlanHead{units, 0, carry};
        if (bad) set_status(a.status, kStatusBadIndex);
    }
}

// ---------------------------------------------------------------------------
// Attention
// ---------------------------------------------------------------------------

// Four codes as fp16 pairs (bytes 0, 1 and 2, 3), exactly.
template <int kCode>
__device__ __forceinline__ void to_h4(uint32_t x, uint32_t &a, uint32_t &b) {
    if (kCode == SA_E4M3) {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}" : "=r"(a), "=r"(b) : "r"(x));
    } else {
        // 1024 + (code + 128) under fp16's exponent of 2^10, then minus 1152
        x ^= 0x80808080u;
        uint32_t p = __byte_perm(x, 0x64646464u, 0x4140), q = __byte_perm(x, 0x64646464u, 0x4342);
        const __half2 off = __half2half2(__ushort_as_half(0x6480));
        const __half2 ha = __hsub2(*reinterpret_cast<__half2 *>(&p), off), hb = __hsub2(*reinterpret_cast<__half2 *>(&q), off);
        a = *reinterpret_cast<const uint32_t *>(&ha);
        b = *reinterpret_cast<const uint32_t *>(&hb);
    }
}
// Key scale times row scale, never 0: the mask's -inf survives it.
__device__ __forceinline__ float logit_scale(float ks, float qf) { return fmaxf(ks * qf, 1.17549435e-38f); }

enum {
    C_Q = 0,                     // Q tiles landed (one phase per segment)
    C_QFREE = 1,                 // every QK of the segment done, 2 arrivals
    C_KF = 2,                    // [2] K tile converted, 4 arrivals
    C_VF = C_KF + kStages,       // [2]
    C_KE = C_VF + kStages,       // [2] K stage free, 2 arrivals (one per Q tile)
    C_VE = C_KE + kStages,
    C_S = C_VE + kStages,        // [2 Q tiles][2 halves] S of 64 keys ready
    C_P = C_S + 4,               // [2 Q tiles][2 halves][2] P of 32 keys written, 4 arrivals
    C_PV = C_P + 8,              // [2 Q tiles] PV of a half done
    C_OD = C_PV + 2,             // [2 Q tiles] last PV of the segment done
    C_L = C_OD + 2,              // [2] segment described
    C_LF = C_L + 2,              // [2] segment released, 15 arrivals
    C_SC = C_LF + 2,             // [4] scales of a key tile written
    C_RK = C_SC + kScaleSlots,   // codes of K landed
    C_RV = C_RK + 1,
    C_RKF = C_RV + 1,            // codes of K read, 4 arrivals
    C_RVF = C_RKF + 1,
    C_END = C_RVF + 1,           // [2 Q tiles]
    NBAR = C_END + 2
};

template <int kD>
constexpr uint32_t tile_bytes() { return kD / 64 * kChunk; }
template <int kD>
constexpr uint32_t k_off() { return 2 * tile_bytes<kD>(); }
template <int kD>
constexpr uint32_t v_off() { return k_off<kD>() + kStages * tile_bytes<kD>(); }
template <int kD>
constexpr uint32_t raw_off() { return v_off<kD>() + kStages * tile_bytes<kD>(); }   // codes of K, then of V
template <int kD>
constexpr uint32_t bar_off() { return raw_off<kD>() + 2 * 128 * kD; }
template <int kD>
constexpr uint32_t smem_bytes() { return bar_off<kD>() + 2048 + 1024; }
static_assert(smem_bytes<128>() <= 227 * 1024, "shared memory");

template <int kD, int kCode>
__global__ void __launch_bounds__(kThreads, 1)
paged_prefill_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, PreArgs a) {
    constexpr uint32_t kTile = tile_bytes<kD>();
    const PagedShape &s = a.s;
    extern __shared__ unsigned char pre_raw[];
    unsigned char *smem = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(pre_raw) + 1023) &
                                                            ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + bar_off<kD>());
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + bar_off<kD>() + 8 * NBAR);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + bar_off<kD>() + 8 * NBAR + 4);
    Seg *segs = reinterpret_cast<Seg *>(smem + bar_off<kD>() + 512);                       // [2]
    // [4][8]: per 16 keys the key scale, the value scale, its log2, and 0 or,
    // where the keys have no page, -inf for their logits
    float4 *scales = reinterpret_cast<float4 *>(smem + bar_off<kD>() + 640);
    static_assert(8 * NBAR + 8 <= 512 && 2 * sizeof(Seg) <= 128 && 640 + kScaleSlots * 128 <= 2048, "shared memory");
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < NBAR; ++i)
            mbar_init(bar(i), (i >= C_P && i < C_P + 8) ? 4
                              : (i == C_LF || i == C_LF + 1) ? 15
                              : (i >= C_KE && i < C_S) || i == C_QFREE ? 2
                              : (i >= C_KF && i < C_KE) || i == C_RKF || i == C_RVF ? 4 : 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "n"(512));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");

    if (warp == 0) {
        // ---- segments and Q ------------------------------------------------
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
        const PlanHead hd = *a.head;
        const long long total = hd.total * s.Hkv;
        const long long per = max((long long)kMinRange, (total + gridDim.x - 1) / gridDim.x);
        long long x = blockIdx.x * per;
        const long long x1 = min(total, x + per);
        Job job{0, 0, 0, 0};
        bool ok = true;
        int n = 0, qlast = -1;
        if (x < x1) {
            // the entry that holds step x: 32 probes a round
            int h = (int)(x / hd.total), lo = 0, hi = hd.n;
            const long long r = x - h * hd.total;
            while (hi - lo > 1) {
                const int step = (hi - lo + 31) / 32, i = lo + lane * step;
                const bool le = i < hi && a.tiles[i].pre <= r;
                const int k = 31 - __clz((int)__ballot_sync(~0u, le));   // lane 0's probe always holds
                lo += k * step;
                hi = min(hi, lo + step);
            }
            int e = lo;
            while (x < x1) {
                const Tile t = a.tiles[e];
                const long long u0 = h * hd.total + t.pre;               // the unit's first step
                Seg g;
                g.b = t.b;
                g.h = h;
                int r0, r1;
                rows_of(a, t.b, r0, r1);
                g.row0 = r0 + t.t0;
                g.ntok = min(2 * a.tpt, r1 - g.row0);
                g.n = paged_len(s, a.c.seq_len, t.b);
                g.pos0 = g.n - (r1 - r0) + t.t0;
                g.ta = (int)(x - u0);
                g.tb = (int)min((long long)t.kt, x1 - u0);
                g.nq = g.ntok > a.tpt ? 2 : 1;
                g.out = g.tb - g.ta == t.kt ? 0 : g.ta > 0 ? 1 : 2;
                if (g.out == 2) job = Job{(int)((u0 + t.kt - 1) / per) - (int)blockIdx.x + 1, g.row0, g.ntok, h};
                const int slot = n & 1;
                if (n >= 2) ok = mbar_wait_lazy(bar(C_LF + slot), ((n >> 1) - 1) & 1, abort_flag, a.status);
                if (!__all_sync(~0u, ok)) { ok = false; break; }
                if (lane == 0) {
                    segs[slot] = g;
                    mbar_arrive(bar(C_L + slot));
                    // Q: the group's heads of the unit's tokens, token-major rows
                    if (n >= 1) ok = mbar_wait_lazy(bar(C_QFREE), (n - 1) & 1, abort_flag, a.status);
                    if (ok) {
                        mbar_expect_tx(bar(C_Q), (uint32_t)(g.nq * (kD / 64) * a.tpt * s.G * 128));
                        for (int q = 0; q < g.nq; ++q)
                            for (int c = 0; c < kD / 64; ++c)
                                asm volatile(
                                    "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
                                    "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(sbase + q * kTile + c * kChunk),
                                    "l"(reinterpret_cast<uint64_t>(&tmQ)), "r"(bar(C_Q)), "r"(64 * c), "r"(h * s.G),
                                    "r"(g.row0 + q * a.tpt)
                                    : "memory");
                        qlast = n;
                    }
                }
                ok = __shfl_sync(~0u, ok, 0);
                if (!ok) break;
                ++n;
                x = u0 + g.tb;
                if (g.tb == t.kt && ++e == hd.n) {
                    e = 0;
                    ++h;
                }
            }
        }
        if (lane == 0) a.jobs[blockIdx.x] = job;
        if (ok) {
            // the end: a segment without tiles
            const int slot = n & 1;
            if (n >= 2) ok = mbar_wait_lazy(bar(C_LF + slot), ((n >> 1) - 1) & 1, abort_flag, a.status);
            if (__all_sync(~0u, ok) && lane == 0) {
                segs[slot].ta = segs[slot].tb = 0;
                mbar_arrive(bar(C_L + slot));
            }
        }
        if (lane == 0 && *abort_flag && qlast >= 0) {
            volatile int never = 0;
            mbar_wait_lazy(bar(C_Q), qlast & 1, &never, a.status);
        }
    } else if (warp == 1 || warp == 3) {
        // ---- MMA issuers: Q tile 0 and Q tile 1 --------------------------------
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
        constexpr uint32_t kFp16 = ~((1u << 7) | (1u << 10));     // the operand formats' bits: fp16 instead of bf16
        constexpr uint32_t idq = idesc_bf16(false, 64) & kFp16, idp = idesc_bf16(true, kD) & kFp16;
        const int q = warp >> 1;
        const uint32_t tS = tmem + q * 128, tO = tmem + 256 + q * 128;
        const uint64_t dq = desc_k_sw128(sbase + q * kTile);
        // S of half h of key tile gg (64 keys)
        auto qk = [&](int gg, int h) {
            const uint64_t db = desc_k_sw128(sbase + k_off<kD>() + (gg % kStages) * kTile + h * 8192);
#pragma unroll 2
            for (int k = 0; k < kD / 16; ++k) {
                const uint32_t off = ((k >> 2) * kChunk + (k & 3) * 32) >> 4;
                mma_ss_w(tS + 64 * h, dq + off, db + off, idq, k > 0);
            }
            mma_commit_w(bar(C_S + 2 * q + h));
            if (h == 1) mma_commit_w(bar(C_KE + gg % kStages));
        };
        // O += P V for 32 keys (e of half h); P (fp16) is the first 32 columns of its S
        auto pv = [&](int gg, int h, int e, bool acc) {
            const uint64_t db = desc_mn_sw128(sbase + v_off<kD>() + (gg % kStages) * kTile, kChunk);
#pragma unroll
            for (int k = 2 * e; k < 2 * e + 2; ++k)
                mma_ts_w(tO, tS + 64 * h + 8 * k, db + (((4 * h + k) * 2048) >> 4), idp, acc || k > 0);
        };
        auto wait = [&](int i, int parity) {
            return __all_sync(~0u, mbar_wait_lazy(bar(i), parity, abort_flag, a.status));
        };
        bool ok = true;
        int gt = 0, gq = 0, n = 0;       // key tiles so far, those of this Q tile, segments
        for (;; ++n) {
            const int slot = n & 1;
            if (!(ok = wait(C_L + slot, (n >> 1) & 1))) break;
            const int T = segs[slot].tb - segs[slot].ta;
            const bool mine = q < segs[slot].nq;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C_LF + slot));
            if (T == 0) break;
            if (!mine) {
                // no rows here: only the arrivals that the stages count on
                // (each after the phase before has ended)
                if (!(ok = wait(C_Q, n & 1))) break;
                if (lane == 0) mbar_arrive(bar(C_QFREE));
                for (int t = 0; ok && t < T; ++t, ++gt) {
                    if (!(ok = wait(C_KF + gt % kStages, (gt / kStages) & 1))) break;
                    if (lane == 0) mbar_arrive(bar(C_KE + gt % kStages));
                    if (!(ok = wait(C_VF + gt % kStages, (gt / kStages) & 1))) break;
                    if (lane == 0) mbar_arrive(bar(C_VE + gt % kStages));
                }
                if (!ok) break;
                continue;
            }
            if (!(ok = wait(C_Q, n & 1))) break;
            if (!(ok = wait(C_KF + gt % kStages, (gt / kStages) & 1))) break;
            tc_fence_after();
#pragma unroll 1
            for (int h = 0; h < 2; ++h) qk(gt, h);
            if (T == 1) mma_commit_w(bar(C_QFREE));
            for (int t = 0; ok && t < T; ++t, ++gt, ++gq) {
                if (!(ok = wait(C_VF + gt % kStages, (gt / kStages) & 1))) break;
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
#pragma unroll 1
                    for (int e = 0; e < 2; ++e) {
                        if (!(ok = wait(C_P + 4 * q + 2 * h + e, gq & 1))) break;
                        tc_fence_after();
                        pv(gt, h, e, t > 0 || h > 0 || e > 0);
                    }
                    if (!ok) break;
                    mma_commit_w(bar(C_PV + q));
                    if (h == 1) mma_commit_w(bar(C_VE + gt % kStages));
                    if (h == 1 && t + 1 == T) mma_commit_w(bar(C_OD + q));
                    if (t + 1 < T) {
                        // the next tile's half, in the place of the one just used up
                        if (h == 0 && !(ok = wait(C_KF + (gt + 1) % kStages, ((gt + 1) / kStages) & 1))) break;
                        tc_fence_after();
                        qk(gt + 1, h);
                        if (h == 1 && t + 2 == T) mma_commit_w(bar(C_QFREE));
                    }
                }
            }
            if (!ok) break;
        }
        // every MMA issued above has completed once this arrives
        mma_commit_w(bar(C_END + q));
        volatile int never = 0;
        mbar_wait_lazy(bar(C_END + q), 0, &never, a.status);
    } else if (warp == 2) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
        // ---- codes and scales of each key tile ----------------------------
        const int boxes = 128 / a.box;
        bool ok = true;
        int gt = 0, klast = -1, vlast = -1;
        for (int n = 0; ok; ++n) {
            const int slot = n & 1;
            ok = mbar_wait_lazy(bar(C_L + slot), (n >> 1) & 1, abort_flag, a.status);
            if (!__all_sync(~0u, ok)) break;
            const Seg g = segs[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C_LF + slot));
            if (g.tb == g.ta) break;
            // lane i < 8: page of keys 128 t + 16 i .. + 15 (-1: no such keys,
            // -2: a table entry out of range), its scales
            auto page_at = [&](int t) {
                const int key = 128 * t + 16 * lane;
                if (lane >= 8 || t >= g.tb || key >= g.n) return -1;
                const int pg = a.c.table[(size_t)g.b * s.maxb + key / s.bs];
                return pg < 0 ? -2 : pg;
            };
            auto scale_at = [&](int &pg, float2 &f) {
                f = make_float2(0.f, 0.f);
                if (pg < 0 || pg >= s.pages) {
                    if (pg != -1) {
                        set_status(a.status, kStatusBadIndex);
                        pg = -2;
                    }
                    return;
                }
                const size_t ph = (size_t)pg * s.Hkv + g.h;
                f = make_float2(a.c.ks[ph], a.c.vs[ph]);
            };
            // codes of keys without a page: zeros, so that nothing spoils the
            // products with their weight of 0
            auto zero = [&](uint32_t at) {
                for (int i = 0; i < a.box * kD; i += 16)
                    asm volatile("st.shared.v4.b32 [%0], {%1,%1,%1,%1};" ::"r"(at + i), "r"(0) : "memory");
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            };
            int pg = page_at(g.ta), pg1 = page_at(g.ta + 1);
            float2 f, f1;
            scale_at(pg, f);
            for (int t = g.ta; t < g.tb; ++t, ++gt) {
                const int pg2 = page_at(t + 2);
                scale_at(pg1, f1);
                const int key = 128 * t + a.box * lane;
                const int mine = __shfl_sync(~0u, pg, (lane * a.box >> 4) & 7);
                const bool live = lane < boxes && mine >= 0 && key < g.n;
                const uint32_t bytes = (uint32_t)__popc(__ballot_sync(~0u, live)) * a.box * kD;
                const int y = (mine * s.Hkv + g.h) * s.bs + key % s.bs;
                const uint32_t dst = sbase + raw_off<kD>() + lane * a.box * kD;
                if (gt >= 1) ok = mbar_wait_lazy(bar(C_RKF), (gt - 1) & 1, abort_flag, a.status);
                if (!__all_sync(~0u, ok)) { ok = false; break; }
                if (lane < 8)
                    scales[(gt % kScaleSlots) * 8 + lane] =
                        make_float4(f.x, f.y, log2f(f.y), pg == -2 ? -CUDART_INF_F : 0.f);
                if (lane < boxes && mine == -2) zero(dst);
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(C_SC + gt % kScaleSlots));
                    if (bytes) mbar_expect_tx(bar(C_RK), bytes);
                    else mbar_arrive(bar(C_RK));
                }
                __syncwarp();
                if (live) tma_load_2d(dst, &tmK, bar(C_RK), 0, y);
                klast = gt;
                if (gt >= 1) ok = mbar_wait_lazy(bar(C_RVF), (gt - 1) & 1, abort_flag, a.status);
                if (!__all_sync(~0u, ok)) { ok = false; break; }
                if (lane < boxes && mine == -2) zero(dst + 128 * kD);
                __syncwarp();
                if (lane == 0) {
                    if (bytes) mbar_expect_tx(bar(C_RV), bytes);
                    else mbar_arrive(bar(C_RV));
                }
                __syncwarp();
                if (live) tma_load_2d(dst + 128 * kD, &tmV, bar(C_RV), 0, y);
                vlast = gt;
                pg = pg1;
                f = f1;
                pg1 = pg2;
            }
        }
        if (lane == 0 && *abort_flag) {
            // let the copies in flight land before the CTA exits (bounded)
            volatile int never = 0;
            if (klast >= 0) mbar_wait_lazy(bar(C_RK), klast & 1, &never, a.status);
            if (vlast >= 0) mbar_wait_lazy(bar(C_RV), vlast & 1, &never, a.status);
        }
    } else if (warp < 8) {
        // ---- converters: codes -> fp16 tiles -----------------------------------
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConv));
        constexpr int LPR = kD / 16;              // lanes per row
        constexpr int NS = 32 / (32 / LPR);       // steps per warp: 32 rows each
        const int cw = warp - 4, r0 = 32 * cw + lane / LPR, l = lane % LPR;
        const uint32_t raw = sbase + raw_off<kD>() + 32 * cw * kD + lane * 16;
        // lanes 4-7 of a 128-wide row fill the other chunk: they store their
        // halves in the other order, which keeps the eight lanes of a row on
        // different banks
        const int u = 2 * (l & 3), swap = l >> 2;
        bool ok = true;
        int gt = 0;
        auto convert = [&](uint32_t src, uint32_t tile, bool tail, int freed) {
            uint4 x[NS];
#pragma unroll
            for (int i = 0; i < NS; ++i)
                asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(x[i].x), "=r"(x[i].y), "=r"(x[i].z), "=r"(x[i].w) : "r"(src + i * 512));
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(freed));
            if (kCode == SA_E4M3 && tail) {
                // behind the sequence's end lies any byte, and a NaN must not
                // meet its weight of 0: those patterns become 256
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    x[i].x -= ((((x[i].x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7) * 7;
                    x[i].y -= ((((x[i].y & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7) * 7;
                    x[i].z -= ((((x[i].z & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7) * 7;
                    x[i].w -= ((((x[i].w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7) * 7;
                }
            }
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                const int r = r0 + i * (32 / LPR);
                uint4 lo, hi;
                to_h4<kCode>(x[i].x, lo.x, lo.y);
                to_h4<kCode>(x[i].y, lo.z, lo.w);
                to_h4<kCode>(x[i].z, hi.x, hi.y);
                to_h4<kCode>(x[i].w, hi.z, hi.w);
                const uint32_t row = tile + swap * kChunk + r * 128;
                const uint32_t p0 = row + (((u + swap) ^ (r & 7)) << 4), p1 = row + (((u + 1 - swap) ^ (r & 7)) << 4);
                const uint4 v0 = swap ? hi : lo, v1 = swap ? lo : hi;
                asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(p0), "r"(v0.x), "r"(v0.y), "r"(v0.z),
                             "r"(v0.w) : "memory");
                asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(p1), "r"(v1.x), "r"(v1.y), "r"(v1.z),
                             "r"(v1.w) : "memory");
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
        };
        auto wait = [&](int i, int parity) {
            return __all_sync(~0u, mbar_wait_lazy(bar(i), parity, abort_flag, a.status));
        };
        for (int n = 0; ok; ++n) {
            const int slot = n & 1;
            if (!(ok = wait(C_L + slot, (n >> 1) & 1))) break;
            const int ta = segs[slot].ta, tb = segs[slot].tb, keys = segs[slot].n;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C_LF + slot));
            if (ta == tb) break;
            for (int t = ta; t < tb; ++t, ++gt) {
                const int st = gt % kStages, use = gt / kStages;
                // keys, then values
#pragma unroll 1
                for (int v = 0; v < 2; ++v) {
                    if (gt >= kStages && !(ok = wait((v ? C_VE : C_KE) + st, (use - 1) & 1))) break;
                    if (!(ok = wait(C_RK + v, gt & 1))) break;
                    convert(raw + v * 128 * kD, sbase + (v ? v_off<kD>() : k_off<kD>()) + st * kTile,
                            v && 128 * (t + 1) > keys, C_RKF + v);
                    if (lane == 0) mbar_arrive(bar((v ? C_VF : C_KF) + st));
                }
                if (!ok) break;
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
        // ---- softmax warpgroups ----------------------------------------------
        const int q = (warp - 8) >> 2, qq = warp & 3, r = 32 * qq + lane;
        const uint32_t lane_off = (uint32_t)(32 * qq) << 16;
        const uint32_t tS = tmem + lane_off + q * 128, tO = tmem + lane_off + 256 + q * 128;
        const int tok_r = r / s.G, head_r = r - tok_r * s.G;
        bool ok = true;
        int gt = 0, gp = 0, done = 0;      // key tiles so far, this Q tile's, its segments
        for (int n = 0; ok; ++n) {
            const int slot = n & 1;
            ok = mbar_wait_lazy(bar(C_L + slot), (n >> 1) & 1, abort_flag, a.status);
            if (!__all_sync(~0u, ok)) break;
            const Seg &g = segs[slot];      // released at the segment's end
            const int T = g.tb - g.ta;
            if (T == 0) break;
            if (q >= g.nq) {
                gt += T;
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(C_LF + slot));
                continue;
            }
            const int tok = q * a.tpt + tok_r;
            const bool row_ok = tok_r < a.tpt && tok < g.ntok;
            // keys the row sees, from the half tile at hand on
            int vis = (s.flags & SA_CAUSAL ? max(0, min(g.n, g.pos0 + tok + 1)) : g.n) - 128 * g.ta;
            const size_t row = row_ok ? (size_t)(g.row0 + tok) * s.Hq + g.h * s.G + head_r : 0;
            const float qf = row_ok ? a.qf[row] : 0.f;
            float m_run = -CUDART_INF_F, mv_run = -CUDART_INF_F, l = 0.f;   // references of l and of O
            for (int t = 0; t < T; ++t, ++gt, ++gp) {
                ok = mbar_wait_lazy(bar(C_SC + gt % kScaleSlots), (gt / kScaleSlots) & 1, abort_flag, a.status);
#pragma unroll 1
                for (int h = 0; h < 2; ++h, vis -= 64) {
                    ok = ok && mbar_wait_lazy(bar(C_S + 2 * q + h), gp & 1, abort_flag, a.status);
                    if (!__all_sync(~0u, ok)) { ok = false; break; }
                    tc_fence_after();
                    float x[64];
                    tmem_ld32(tS + 64 * h, x);
                    tmem_ld32(tS + 64 * h + 32, x + 32);
                    tmem_wait_ld();
                    reg_fence<64>(x);
                    if (vis < 64) {
#pragma unroll
                        for (int k = 0; k < 64; ++k) x[k] = k < vis ? x[k] : -CUDART_INF_F;
                    }
                    // 16 keys share a page, so a scale: the largest logit of each
                    // group (four chains side by side)
                    const float4 *sc = scales + (gt % kScaleSlots) * 8 + 4 * h;
                    float gm[4], sk[4], lv[4], hole[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) gm[i] = fmaxf(x[16 * i], x[16 * i + 1]);
#pragma unroll
                    for (int k = 2; k < 16; k += 2)
#pragma unroll
                        for (int i = 0; i < 4; ++i) gm[i] = fmax3(gm[i], x[16 * i + k], x[16 * i + k + 1]);
                    float mx = -CUDART_INF_F, mv = -CUDART_INF_F;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 f = sc[i];
                        sk[i] = logit_scale(f.x, qf);
                        lv[i] = f.z;
                        hole[i] = f.w;
                        gm[i] = fmaf(gm[i], sk[i], f.w);
                        mx = fmaxf(mx, gm[i]);
                        mv = fmaxf(mv, gm[i] + lv[i]);
                    }
                    const bool need = mx > m_run + kWeightSlack || mv > mv_run + (kWeightLift + kWeightSlack);
                    if (__any_sync(~0u, need)) {
                        float corr = 1.f;
                        if (need) {
                            const float m1 = fmaxf(mx, m_run), v1 = fmaxf(mv - kWeightLift, mv_run);
                            l *= m_run == m1 ? 1.f : ex2(m_run - m1);
                            corr = mv_run == v1 ? 1.f : ex2(mv_run - v1);
                            m_run = m1;
                            mv_run = v1;
                        }
                        if (t > 0 || h > 0) {
                            // O is stable once the product of the half before
                            // is done (S ready: the one before that is; this
                            // half's waits for the weights below)
                            ok = mbar_wait_lazy(bar(C_PV + q), (2 * gp + h - 1) & 1, abort_flag, a.status);
                            if (!__all_sync(~0u, ok)) { ok = false; break; }
                            tc_fence_after();
#pragma unroll 2
                            for (int cc = 0; cc < kD / 8; ++cc) {
                                float o[8];
                                tmem_ld8(tO + 8 * cc, o);
                                tmem_wait_ld();
                                reg_fence<8>(o);
#pragma unroll
                                for (int k = 0; k < 8; ++k) o[k] *= corr;
                                tmem_st8(tO + 8 * cc, reinterpret_cast<const uint32_t *>(o));
                            }
                            tmem_wait_st();
                        }
                    }
                    // w = p vs 2^(m - m') = 2^(z - m + e), e = log2 vs + m - m'
                    // of the group: one exponential a key; l gets the group's
                    // sum times 2^-e.  Limits on e keep 2^-e and the exponential
                    // finite and change no result: at e = -40 (vs = 0) w
                    // vanishes in fp16 and l still counts p down to 2^-86; above
                    // 300, where l takes nothing any more (p is under 2^-285),
                    // the output is under fp32's range.  (With a limit of 100,
                    // values of scale 2^40 a hundred bits below a page without
                    // any came out 2^10 too small.)
                    const float ref = m_run == -CUDART_INF_F ? 0.f : m_run;
                    const float vf = mv_run == -CUDART_INF_F ? 0.f : ref - mv_run;
                    // The 16-key groups run as a pipeline: a group's exponentials
                    // are issued before the group before it is rounded, summed
                    // and stored, so the exponential unit does not wait.
                    float ex[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        ex[i] = fmaxf(fminf(lv[i] + vf, 300.f), -40.f);
                        const float2 f2 = make_float2(sk[i], sk[i]), b2 = make_float2(ex[i] - ref + hole[i], ex[i] - ref + hole[i]);
#pragma unroll
                        for (int k = 16 * i; k < 16 * i + 16; k += 2) {
                            const float2 z = ffma2(make_float2(x[k], x[k + 1]), f2, b2);
                            x[k] = z.x;
                            x[k + 1] = z.y;
                        }
                    }
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 5; ++i) {
                        if (i < 4) {
#pragma unroll
                            for (int k = 16 * i; k < 16 * i + 16; ++k) x[k] = ex2(x[k]);
                        }
                        if (i == 0) continue;
                        const int g0 = 16 * (i - 1);
                        float2 p[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            p[k] = make_float2(x[g0 + 2 * k], x[g0 + 2 * k + 1]);
                            const __half2 h2 = __floats2half2_rn(p[k].x, p[k].y);
                            pk[8 * ((i - 1) & 1) + k] = *reinterpret_cast<const uint32_t *>(&h2);
                        }
#pragma unroll
                        for (int w = 4; w; w >>= 1)
#pragma unroll
                            for (int k = 0; k < w; ++k) p[k] = fadd2(p[k], p[k + w]);
                        l = fmaf(p[0].x + p[0].y, ex2(-ex[i - 1]), l);
                        if (i == 2) tmem_st16(tS + 64 * h, pk);
                        if (i == 4) {
                            // the first 32 keys are handed over once the others
                            // are computed, so that their store is not waited for
                            tmem_wait_st();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(bar(C_P + 4 * q + 2 * h));
                            tmem_st16(tS + 64 * h + 16, pk);
                        }
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C_P + 4 * q + 2 * h + 1));
                }
                if (!ok) break;
            }
            if (!ok) break;
            // ---- epilogue ------------------------------------------------------
            ok = mbar_wait_lazy(bar(C_OD + q), done & 1, abort_flag, a.status);
            if (!__all_sync(~0u, ok)) { ok = false; break; }
            ++done;
            tc_fence_after();
            const float inv = l == 0.f ? 0.f : mv_run == -CUDART_INF_F ? 0.f * l : ex2(mv_run - m_run) / l;   // NaN stays NaN
            float *rec = a.rec + ((size_t)blockIdx.x * 2 + (g.out == 2 ? 1 : 0)) * (kD + 3) * 256 + 128 * q + r;
#pragma unroll 1
            for (int cc = 0; cc < kD / 32; ++cc) {
                float o[32];
                tmem_ld32(tO + 32 * cc, o);
                tmem_wait_ld();
                reg_fence<32>(o);
                if (!row_ok) continue;
                if (g.out == 0) {
#pragma unroll
                    for (int v = 0; v < 32; v += 8) {
                        float f[8];
#pragma unroll
                        for (int k = 0; k < 8; ++k) f[k] = l == 0.f ? 0.f : o[v + k] * inv;
                        store16(a.O + row * kD + 32 * cc + v, f);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) rec[(size_t)(32 * cc + k) * 256] = o[k];
                }
            }
            if (row_ok) {
                if (g.out == 0) {
                    a.lse[row] = l == 0.f ? -CUDART_INF_F : (m_run + log2f(l)) * kLn2;
                } else {
                    rec[(size_t)kD * 256] = m_run;
                    rec[(size_t)(kD + 1) * 256] = l;
                    rec[(size_t)(kD + 2) * 256] = mv_run;
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C_LF + slot));
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512));
    }
}

// Joins the records of a unit that the ranges from blockIdx.x on share:
// 32 rows per CTA (lane = row), kD / 8 columns per warp.
template <int kD>
__global__ void __launch_bounds__(256)
paged_prefill_merge_kernel(PreArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const Job job = a.jobs[blockIdx.x];
    if (job.n < 2) return;
    constexpr int NC = kD / 8;
    const int warp = threadIdx.x >> 5, r = 32 * blockIdx.y + (threadIdx.x & 31);
    const int q = r >> 7, tok_r = (r & 127) / a.s.G, head = (r & 127) - tok_r * a.s.G, tok = q * a.tpt + tok_r;
    if (tok_r >= a.tpt || tok >= job.ntok) return;
    auto rec = [&](int i) { return a.rec + ((size_t)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * (kD + 3) * 256 + r; };
    float M = -CUDART_INF_F, MV = -CUDART_INF_F, l = 0.f, o[NC];
    for (int i = 0; i < job.n; ++i) {
        M = fmaxf(M, rec(i)[kD * 256]);
        MV = fmaxf(MV, rec(i)[(kD + 2) * 256]);
    }
#pragma unroll
    for (int k = 0; k < NC; ++k) o[k] = 0.f;
    for (int i = 0; i < job.n; ++i) {
        const float *p = rec(i);
        const float m = p[kD * 256], v = p[(kD + 2) * 256], f = v == -CUDART_INF_F ? 0.f : ex2(v - MV);
        l += p[(kD + 1) * 256] * (m == -CUDART_INF_F ? 1.f : ex2(m - M));     // at -inf it is 0, or NaN
#pragma unroll
        for (int k = 0; k < NC; ++k) o[k] += p[(warp * NC + k) * 256] * f;
    }
    const size_t row = (size_t)(job.row0 + tok) * a.s.Hq + job.h * a.s.G + head;
    const float inv = l == 0.f ? 0.f : MV == -CUDART_INF_F ? 0.f * l : ex2(MV - M) / l;
#pragma unroll
    for (int k = 0; k < NC; ++k) o[k] = l == 0.f ? 0.f : o[k] * inv;
#pragma unroll
    for (int k = 0; k < NC; k += 8) store16(a.O + row * kD + warp * NC + k, o + k);
    if (warp == 0) a.lse[row] = l == 0.f ? -CUDART_INF_F : (M + log2f(l)) * kLn2;
}

size_t al(size_t x) { return (x + 255) & ~(size_t)255; }
int cap_tiles(const PagedShape &s) { return s.tokens / (2 * (128 / s.G)) + s.B + 1; }

template <int kD, int kCode>
cudaError_t run(const PreArgs &a, int grid, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                cudaStream_t st) {
    auto kern = paged_prefill_kernel<kD, kCode>;
    // the register split assumes the launch's count
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, kern);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != kRegsLaunch) return cudaErrorInvalidDeviceFunction;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_bytes<kD>());
    if (e != cudaSuccess) return e;
    const size_t plan_smem = (size_t)(a.s.B + 1) * sizeof(int);
    if (plan_smem > 40 * 1024) {
        e = cudaFuncSetAttribute(paged_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)plan_smem);
        if (e != cudaSuccess) return e;
    }
    // queries: up to one CTA per SM beside the one that lists the steps
    const long long conv = ((long long)a.s.tokens * a.s.Hq * a.s.d / 8 + 1023) / 1024;
    if ((e = launch_pdl(paged_plan_kernel, dim3(1 + (unsigned)min(conv, (long long)grid)), dim3(1024), plan_smem, st, a)) != cudaSuccess) return e;
    note_launch();
    if ((e = launch_pdl(kern, dim3((unsigned)grid), dim3(kThreads), smem_bytes<kD>(), st, mq, mk, mv, a)) != cudaSuccess)
        return e;
    note_launch();
    if ((e = launch_pdl(paged_prefill_merge_kernel<kD>, dim3((unsigned)grid, 8), dim3(256), 0, st, a)) != cudaSuccess)
        return e;
    note_launch();
    return cudaGetLastError();
}

}  // namespace

bool paged_prefill_supported(const PagedShape &s) { return s.dtype == SA_BF16 && s.G <= 128; }

size_t paged_prefill_scratch(const PagedShape &s) {
    return al((size_t)s.tokens * s.Hq * s.d * 2) + al((size_t)s.tokens * s.Hq * 4) + al(sizeof(PlanHead)) + al(cap_tiles(s) * sizeof(Tile)) + al(kMaxGrid * sizeof(Job)) +
           (size_t)kMaxGrid * 2 * (s.d + 3) * 256 * sizeof(float);
}

cudaError_t launch_paged_prefill(const PagedShape &s, const void *Q, const int32_t *cu, const PagedCache &c, void *O,
                                 float *lse, int few, unsigned *status, void *scratch, cudaStream_t st) {
    PreArgs a{};
    a.few = few;
    a.s = s;
    a.c = c;
    a.cu = cu;
    a.O = (__nv_bfloat16 *)O;
    a.lse = lse;
    a.status = status;
    a.tpt = 128 / s.G;
    a.cap_tiles = cap_tiles(s);
    unsigned char *w = (unsigned char *)scratch;
    a.Q = (const __nv_bfloat16 *)Q;
    a.qh = (__half *)w;
    w += al((size_t)s.tokens * s.Hq * s.d * 2);
    a.qf = (float *)w;
    w += al((size_t)s.tokens * s.Hq * 4);
    a.head = (PlanHead *)w;
    w += al(sizeof(PlanHead));
    a.tiles = (Tile *)w;
    w += al(a.cap_tiles * sizeof(Tile));
    a.jobs = (Job *)w;
    w += al(kMaxGrid * sizeof(Job));
    a.rec = (float *)w;
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorNoDevice;
    auto enc = tensor_map_encoder();
    if (!enc) return cudaErrorNotSupported;
    CUtensorMap mq;
    cuuint64_t dims[3] = {(cuuint64_t)s.d, (cuuint64_t)s.Hq, (cuuint64_t)s.tokens};
    cuuint64_t strides[2] = {(cuuint64_t)s.d * 2, (cuuint64_t)s.Hq * s.d * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)s.G, (cuuint32_t)a.tpt};
    cuuint32_t estr[3] = {1, 1, 1};
    if (enc(&mq, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, a.qh, dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    // codes as they lie; a box is the largest power of two of keys in one page
    a.box = s.bs & -s.bs;
    CUtensorMap mk, mv;
    cuuint64_t cdims[2] = {(cuuint64_t)s.d, (cuuint64_t)s.pages * s.Hkv * s.bs};
    cuuint64_t cstrides[1] = {(cuuint64_t)s.d};
    cuuint32_t cbox[2] = {(cuuint32_t)s.d, (cuuint32_t)a.box};
    for (int i = 0; i < 2; ++i)
        if (enc(i ? &mv : &mk, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(i ? c.V : c.K), cdims, cstrides,
                cbox, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
                CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
            return cudaErrorInvalidValue;
    const int grid = min(sms, kMaxGrid);
    if (s.d == 128)
        return s.code == SA_E4M3 ? run<128, SA_E4M3>(a, grid, mq, mk, mv, st)
                                 : run<128, SA_INT8>(a, grid, mq, mk, mv, st);
    return s.code == SA_E4M3 ? run<64, SA_E4M3>(a, grid, mq, mk, mv, st) : run<64, SA_INT8>(a, grid, mq, mk, mv, st);
}

}  // namespace sa
