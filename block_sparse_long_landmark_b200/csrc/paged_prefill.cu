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
//   * codes reach shared memory as bf16 (exact for e4m3 and int8) through the
//     registers of a converter warpgroup, which loads one tile ahead straight
//     from the pages; scales stay out of the matrices: the key's multiplies
//     the logit, the value's the weight before it is rounded to bf16 (2^-8 of
//     each weight; bf16 because p vs spans the scales' range);
//   * the work is one line of (unit, key tile) steps cut into one equal range
//     per CTA, whatever the lengths: a few queries over a long cache spread
//     over every SM, and a causal triangle is balanced.  Units that ranges
//     share leave fp32 records (at most two a CTA), joined by a second launch.
//
// Warps: 0 takes segments from the line and loads Q by TMA, 1 owns tensor
// memory and issues the MMAs, 2-3 idle; 4-7 convert; 8-11 and 12-15 softmax.
// Registers: launched at 128; 56 + 88 + 2 * 184 = 4 * 128.
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
constexpr int kRegsLaunch = 128, kRegsIssue = 56, kRegsConv = 88, kRegsSoft = 184;
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
    float *rec;         // [grid][2][d + 2][256]
    int tpt;            // tokens per 128-row tile
};

struct Seg {
    int b, h, row0, ntok;    // first packed row, tokens
    int pos0, n;             // position of the first token, keys of the sequence
    int ta, tb;              // key tiles
    int nq;                  // 128-row tiles with tokens
    int out;                 // 0: whole unit, 1: record slot 0, 2: record slot 1
};

// ---------------------------------------------------------------------------
// The step list: units in order of (sequence, token), each with its number of
// key tiles and the tiles before it.  One CTA.
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

__global__ void __launch_bounds__(1024)
paged_plan_kernel(PreArgs a) {
    extern __shared__ int off_s[];
    __shared__ long long tmp[32];
    const PagedShape &s = a.s;
    const int tid = threadIdx.x, tpu = 2 * a.tpt;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int share = (s.B + 1023) / 1024, b0 = min(s.B, tid * share), b1 = min(s.B, b0 + share);
    long long n = 0, total;
    for (int b = b0; b < b1; ++b) {
        int r0, r1;
        rows_of(a, b, r0, r1);
        n += (r1 - r0 + tpu - 1) / tpu;
    }
    long long at = scan1024(n, tmp, total) - n;
    // offsets that overlap would list more units than rows
    const bool bad = total > a.cap_tiles;
    for (int b = b0; b < b1; ++b) {
        int r0, r1;
        rows_of(a, b, r0, r1);
        off_s[b] = bad ? 0 : (int)at;
        at += (r1 - r0 + tpu - 1) / tpu;
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

// Two e4m3 or int8 codes (bytes i, i + 1 of x) as a bf16 pair, exactly.
template <int kCode>
__device__ __forceinline__ uint32_t to_bf2(uint32_t x, bool high) {
    if (kCode == SA_E4M3) {
        // sign and seven value bits under bf16's 8-bit exponent give value * 2^-120
        const uint32_t w = __byte_perm(x, 0, high ? 0x3424 : 0x1404);
        uint32_t v = ((w >> 4) & 0x07f007f0u) | (w & 0x80008000u);
        const __nv_bfloat162 up = __bfloat162bfloat162(__ushort_as_bfloat16(0x7b80));   // 2^120
        __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162 *>(&v), up);
        return *reinterpret_cast<uint32_t *>(&r);
    }
    // 128 + low seven bits, minus 128 or (sign bit: the exponent's lowest) 256
    const uint32_t w = __byte_perm(x, 0x43434343u, high ? 0x4342 : 0x4140);
    uint32_t lo = w & 0xff7fff7fu, off = w & 0xff80ff80u;
    __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162 *>(&lo), *reinterpret_cast<__nv_bfloat162 *>(&off));
    return *reinterpret_cast<uint32_t *>(&r);
}

enum {
    C_Q = 0,                     // Q tiles landed (one phase per segment)
    C_QFREE = 1,                 // every QK of the segment done
    C_KF = 2,                    // [2] K tile converted, 4 arrivals
    C_VF = C_KF + kStages,       // [2]
    C_KE = C_VF + kStages,       // [2] K stage free
    C_VE = C_KE + kStages,
    C_S = C_VE + kStages,        // [2 Q tiles] S ready
    C_P = C_S + 2,               // [2 Q tiles][4 quarters] P written, 128 arrivals
    C_OD = C_P + 8,              // [2 Q tiles] last PV of the segment done
    C_L = C_OD + 2,              // [2] segment described
    C_LF = C_L + 2,              // [2] segment released, 13 arrivals
    C_SC = C_LF + 2,             // [4] scales of a key tile written
    C_END = C_SC + kScaleSlots,
    NBAR
};

template <int kD>
constexpr uint32_t tile_bytes() { return kD / 64 * kChunk; }
template <int kD>
constexpr uint32_t k_off() { return 2 * tile_bytes<kD>(); }
template <int kD>
constexpr uint32_t v_off() { return k_off<kD>() + kStages * tile_bytes<kD>(); }
template <int kD>
constexpr uint32_t bar_off() { return v_off<kD>() + kStages * tile_bytes<kD>(); }
template <int kD>
constexpr uint32_t smem_bytes() { return bar_off<kD>() + 1024 + 1024; }

template <int kD, int kCode>
__global__ void __launch_bounds__(kThreads, 1)
paged_prefill_kernel(const __grid_constant__ CUtensorMap tmQ, PreArgs a) {
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
    float2 *scales = reinterpret_cast<float2 *>(smem + bar_off<kD>() + 640);               // [4][8]: key, value
    static_assert(8 * NBAR + 8 <= 512 && 2 * sizeof(Seg) <= 128 && 640 + kScaleSlots * 64 <= 1024, "shared memory");
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < NBAR; ++i)
            mbar_init(bar(i), (i >= C_P && i < C_P + 8) ? 128
                              : (i == C_LF || i == C_LF + 1) ? 13
                              : (i >= C_KF && i < C_KE) ? 4 : 1);
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
                if (n >= 2) ok = mbar_wait(bar(C_LF + slot), ((n >> 1) - 1) & 1, abort_flag, a.status);
                if (!__all_sync(~0u, ok)) { ok = false; break; }
                if (lane == 0) {
                    segs[slot] = g;
                    mbar_arrive(bar(C_L + slot));
                    // Q: the group's heads of the unit's tokens, token-major rows
                    if (n >= 1) ok = mbar_wait(bar(C_QFREE), (n - 1) & 1, abort_flag, a.status);
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
            if (n >= 2) ok = mbar_wait(bar(C_LF + slot), ((n >> 1) - 1) & 1, abort_flag, a.status);
            if (__all_sync(~0u, ok) && lane == 0) {
                segs[slot].ta = segs[slot].tb = 0;
                mbar_arrive(bar(C_L + slot));
            }
        }
        if (lane == 0 && *abort_flag && qlast >= 0) {
            volatile int never = 0;
            mbar_wait(bar(C_Q), qlast & 1, &never, a.status);
        }
    } else if (warp == 1) {
        // ---- MMA issuer ------------------------------------------------------
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
        constexpr uint32_t idq = idesc_bf16(false, 128), idp = idesc_bf16(true, kD);
        auto qk = [&](int q, int gg) {
            const uint64_t da = desc_k_sw128(sbase + q * kTile);
            const uint64_t db = desc_k_sw128(sbase + k_off<kD>() + (gg % kStages) * kTile);
#pragma unroll
            for (int k = 0; k < kD / 16; ++k) {
                const uint32_t off = ((k >> 2) * kChunk + (k & 3) * 32) >> 4;
                mma_ss_w(tmem + q * 128, da + off, db + off, idq, k > 0);
            }
            mma_commit_w(bar(C_S + q));
        };
        // O_q += P_q V for keys 32 h .. 32 h + 31; P_q (bf16) is the first 64 columns of S_q
        auto pv = [&](int q, int gg, int h, bool acc) {
            const uint64_t db = desc_mn_sw128(sbase + v_off<kD>() + (gg % kStages) * kTile, kChunk);
#pragma unroll
            for (int k = 2 * h; k < 2 * h + 2; ++k)
                mma_ts_w(tmem + 256 + q * 128, tmem + q * 128 + 8 * k, db + ((k * 2048) >> 4), idp, acc || k > 0);
        };
        auto wait = [&](int i, int parity) {
            return __all_sync(~0u, mbar_wait(bar(i), parity, abort_flag, a.status));
        };
        bool ok = true;
        int gt = 0, g1 = 0, n = 0;       // key tiles so far, those of Q tile 1, segments
        for (;; ++n) {
            const int slot = n & 1;
            if (!(ok = wait(C_L + slot, (n >> 1) & 1))) break;
            const int T = segs[slot].tb - segs[slot].ta;
            const bool two = segs[slot].nq == 2;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C_LF + slot));
            if (T == 0) break;
            if (!(ok = wait(C_Q, n & 1))) break;
            if (!(ok = wait(C_KF + gt % kStages, (gt / kStages) & 1))) break;
            tc_fence_after();
            qk(0, gt);
            if (two) qk(1, gt);
            mma_commit_w(bar(C_KE + gt % kStages));
            if (T == 1) mma_commit_w(bar(C_QFREE));
            for (int t = 0; ok && t < T; ++t) {
                const int gg = gt + t;
                for (int h = 0; ok && h < 4; ++h) {
                    if (!(ok = wait(C_P + h, gg & 1))) break;
                    if (h == 0 && !(ok = wait(C_VF + gg % kStages, (gg / kStages) & 1))) break;
                    tc_fence_after();
                    pv(0, gg, h, t > 0 || h > 0);
                }
                if (!ok) break;
                if (!two) mma_commit_w(bar(C_VE + gg % kStages));
                if (t == T - 1) mma_commit_w(bar(C_OD));
                if (t + 1 < T) {
                    if (!(ok = wait(C_KF + (gg + 1) % kStages, ((gg + 1) / kStages) & 1))) break;
                    tc_fence_after();
                    qk(0, gg + 1);
                    if (!two) {
                        mma_commit_w(bar(C_KE + (gg + 1) % kStages));
                        if (t + 2 == T) mma_commit_w(bar(C_QFREE));
                    }
                }
                if (two) {
                    for (int h = 0; ok && h < 4; ++h) {
                        if (!(ok = wait(C_P + 4 + h, (g1 + t) & 1))) break;
                        tc_fence_after();
                        pv(1, gg, h, t > 0 || h > 0);
                    }
                    if (!ok) break;
                    mma_commit_w(bar(C_VE + gg % kStages));
                    if (t == T - 1) mma_commit_w(bar(C_OD + 1));
                    if (t + 1 < T) {
                        qk(1, gg + 1);
                        mma_commit_w(bar(C_KE + (gg + 1) % kStages));
                        if (t + 2 == T) mma_commit_w(bar(C_QFREE));
                    }
                }
            }
            if (!ok) break;
            gt += T;
            if (two) g1 += T;
        }
        // every MMA issued above has completed once this arrives
        mma_commit_w(bar(C_END));
        volatile int never = 0;
        mbar_wait(bar(C_END), 0, &never, a.status);
    } else if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    } else if (warp < 8) {
        // ---- converters: cached codes -> bf16 tiles -----------------------------
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConv));
        constexpr int LPR = kD / 16;              // lanes per row
        constexpr int RPW = 32 / LPR;             // rows per warp and step
        constexpr int NS = 128 / (4 * RPW);       // steps per tile
        const int cw = warp - 4, sub = lane / LPR, l = lane % LPR;
        const float qs = s.scale * kLog2e;
        bool ok = true;
        int gt = 0;
        for (int n = 0; ok; ++n) {
            const int slot = n & 1;
            ok = mbar_wait(bar(C_L + slot), (n >> 1) & 1, abort_flag, a.status);
            if (!__all_sync(~0u, ok)) break;
            const Seg g = segs[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C_LF + slot));
            if (g.tb == g.ta) break;
            // lane i < 8: page of keys 128 t + 16 i .. + 15 (-1: none)
            auto page_at = [&](int t) {
                const int key = 128 * t + 16 * lane;
                if (lane >= 8 || t >= g.tb || key >= g.n) return -1;
                const int pg = a.c.table[(size_t)g.b * s.maxb + key / s.bs];
                if (pg >= 0 && pg < s.pages) return pg;
                set_status(a.status, kStatusBadIndex);
                return -1;
            };
            // byte offset of the lane's 16 codes in step i of tile t; false: no such key
            auto where = [&](int t, int pages, int i, size_t &at) {
                const int r = i * 4 * RPW + cw * RPW + sub, grp = (i * 4 * RPW + cw * RPW) >> 4;
                const int pg = __shfl_sync(~0u, pages, grp), key = 128 * t + r;
                at = (((size_t)max(pg, 0) * s.Hkv + g.h) * s.bs + key % s.bs) * kD + l * 16;
                return pg >= 0 && key < g.n;
            };
            auto load = [&](const uint8_t *base, int t, int pages, uint4 *raw) {
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    size_t at;
                    const bool in = where(t, pages, i, at);
                    raw[i] = in ? __ldg(reinterpret_cast<const uint4 *>(base + at)) : make_uint4(0, 0, 0, 0);
                }
            };
            auto put = [&](uint32_t tile, const uint4 *raw) {
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    const int r = i * 4 * RPW + cw * RPW + sub;
                    uint4 lo, hi;
                    lo.x = to_bf2<kCode>(raw[i].x, false);
                    lo.y = to_bf2<kCode>(raw[i].x, true);
                    lo.z = to_bf2<kCode>(raw[i].y, false);
                    lo.w = to_bf2<kCode>(raw[i].y, true);
                    hi.x = to_bf2<kCode>(raw[i].z, false);
                    hi.y = to_bf2<kCode>(raw[i].z, true);
                    hi.z = to_bf2<kCode>(raw[i].w, false);
                    hi.w = to_bf2<kCode>(raw[i].w, true);
                    // lanes 4-7 of a 128-wide row fill the other chunk: they
                    // store their halves in the other order, which keeps the
                    // eight lanes of a row on different banks
                    const int u = 2 * (l & 3), swap = l >> 2;
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
            uint4 kr[NS], vr[NS];
            int pg = page_at(g.ta), pg1 = page_at(g.ta + 1);
            load(a.c.K, g.ta, pg, kr);
            load(a.c.V, g.ta, pg, vr);
            for (int t = g.ta; t < g.tb; ++t, ++gt) {
                const int st = gt % kStages, use = gt / kStages;
                if (gt >= kStages) ok = mbar_wait(bar(C_KE + st), (use - 1) & 1, abort_flag, a.status);
                if (!__all_sync(~0u, ok)) { ok = false; break; }
                if (cw == 0) {
                    if (lane < 8) {
                        float2 f = make_float2(0.f, 0.f);
                        if (pg >= 0) {
                            const size_t ph = (size_t)pg * s.Hkv + g.h;
                            f = make_float2(a.c.ks[ph], a.c.vs[ph]);
                        }
                        // a key scale of 0 as the smallest number: the mask's -inf survives it
                        scales[(gt % kScaleSlots) * 8 + lane] = make_float2(fmaxf(f.x * qs, 1.17549435e-38f), f.y);
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(C_SC + gt % kScaleSlots));
                }
                put(sbase + k_off<kD>() + st * kTile, kr);
                if (lane == 0) mbar_arrive(bar(C_KF + st));
                if (t + 1 < g.tb) load(a.c.K, t + 1, pg1, kr);
                if (gt >= kStages) ok = mbar_wait(bar(C_VE + st), (use - 1) & 1, abort_flag, a.status);
                if (!__all_sync(~0u, ok)) { ok = false; break; }
                put(sbase + v_off<kD>() + st * kTile, vr);
                if (lane == 0) mbar_arrive(bar(C_VF + st));
                if (t + 1 < g.tb) load(a.c.V, t + 1, pg1, vr);
                pg = pg1;
                pg1 = page_at(t + 2);
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
            ok = mbar_wait(bar(C_L + slot), (n >> 1) & 1, abort_flag, a.status);
            if (!__all_sync(~0u, ok)) break;
            const Seg g = segs[slot];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(C_LF + slot));
            const int T = g.tb - g.ta;
            if (T == 0) break;
            if (q >= g.nq) {
                gt += T;
                continue;
            }
            const int tok = q * a.tpt + tok_r;
            const bool row_ok = tok_r < a.tpt && tok < g.ntok;
            const int see = s.flags & SA_CAUSAL ? max(0, min(g.n, g.pos0 + tok + 1)) : g.n;
            float m_run = -CUDART_INF_F, l = 0.f;
            for (int t = g.ta; t < g.tb; ++t, ++gt, ++gp) {
                ok = mbar_wait(bar(C_SC + gt % kScaleSlots), (gt / kScaleSlots) & 1, abort_flag, a.status) &&
                     mbar_wait(bar(C_S + q), gp & 1, abort_flag, a.status);
                if (!__all_sync(~0u, ok)) { ok = false; break; }
                tc_fence_after();
                float x[128];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, x + 32 * c);
                tmem_wait_ld();
                reg_fence<128>(x);
                const float2 *sc = scales + (gt % kScaleSlots) * 8;
                const int vis = see - 128 * t;             // keys of this tile the row sees
                if (vis < 128) {
#pragma unroll
                    for (int k = 0; k < 128; ++k) x[k] = k < vis ? x[k] : -CUDART_INF_F;
                }
                // 16 keys share a page, so a scale: the largest logit of each group
                float mx = -CUDART_INF_F;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float m0 = fmax3(x[16 * i], x[16 * i + 1], x[16 * i + 2]);
                    float m1 = fmax3(x[16 * i + 3], x[16 * i + 4], x[16 * i + 5]);
                    m0 = fmax3(m0, x[16 * i + 6], x[16 * i + 7]);
                    m1 = fmax3(m1, x[16 * i + 8], x[16 * i + 9]);
                    m0 = fmax3(m0, x[16 * i + 10], x[16 * i + 11]);
                    m1 = fmax3(m1, x[16 * i + 12], x[16 * i + 13]);
                    m0 = fmax3(m0, x[16 * i + 14], x[16 * i + 15]);
                    mx = fmaxf(mx, fmaxf(m0, m1) * sc[i].x);
                }
                if (t == g.ta) {
                    m_run = mx;
                } else {
                    const bool need = mx > m_run + 8.f;
                    if (__any_sync(~0u, need)) {
                        // the PV before this S has completed: O is stable
                        const float corr = need ? ex2(m_run - mx) : 1.f;
                        if (need) {
                            l *= corr;
                            m_run = mx;
                        }
#pragma unroll
                        for (int cc = 0; cc < kD / 32; ++cc) {
                            float o[32];
                            tmem_ld32(tO + 32 * cc, o);
                            tmem_wait_ld();
                            reg_fence<32>(o);
#pragma unroll
                            for (int k = 0; k < 32; ++k) o[k] *= corr;
                            tmem_st32(tO + 32 * cc, reinterpret_cast<const uint32_t *>(o));
                        }
                        tmem_wait_st();
                    }
                }
                const float ref = m_run == -CUDART_INF_F ? 0.f : m_run;
                const float2 b2 = make_float2(-ref, -ref);
                float2 la = make_float2(0.f, 0.f), lb = make_float2(0.f, 0.f);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float2 f = sc[2 * c + i];
                        const float2 sk = make_float2(f.x, f.x), sv = make_float2(f.y, f.y);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int e = 32 * c + 16 * i + 2 * k;
                            const float2 z = ffma2(make_float2(x[e], x[e + 1]), sk, b2);
                            float2 p = make_float2(ex2(z.x), ex2(z.y));
                            if (k & 1) lb = fadd2(lb, p);
                            else la = fadd2(la, p);
                            p = ffma2(p, sv, make_float2(0.f, 0.f));
                            const __nv_bfloat162 h2 = __floats2bfloat162_rn(p.x, p.y);
                            pk[8 * i + k] = *reinterpret_cast<const uint32_t *>(&h2);
                        }
                    }
                    tmem_st16(tS + 16 * c, pk);
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(bar(C_P + 4 * q + c));
                }
                l += (la.x + la.y) + (lb.x + lb.y);
            }
            if (!ok) break;
            // ---- epilogue ------------------------------------------------------
            ok = mbar_wait(bar(C_OD + q), done & 1, abort_flag, a.status);
            if (!__all_sync(~0u, ok)) { ok = false; break; }
            ++done;
            tc_fence_after();
            const size_t row = row_ok ? (size_t)(g.row0 + tok) * s.Hq + g.h * s.G + head_r : 0;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            float *rec = a.rec + ((size_t)blockIdx.x * 2 + (g.out == 2 ? 1 : 0)) * (kD + 2) * 256 + 128 * q + r;
#pragma unroll
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
                }
            }
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
    auto rec = [&](int i) { return a.rec + ((size_t)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * (kD + 2) * 256 + r; };
    float M = -CUDART_INF_F, l = 0.f, o[NC];
    for (int i = 0; i < job.n; ++i) M = fmaxf(M, rec(i)[kD * 256]);
#pragma unroll
    for (int k = 0; k < NC; ++k) o[k] = 0.f;
    for (int i = 0; i < job.n; ++i) {
        const float *p = rec(i);
        const float m = p[kD * 256], f = m == -CUDART_INF_F ? 0.f : ex2(m - M);
        l += p[(kD + 1) * 256] * f;
#pragma unroll
        for (int k = 0; k < NC; ++k) o[k] += p[(warp * NC + k) * 256] * f;
    }
    const size_t row = (size_t)(job.row0 + tok) * a.s.Hq + job.h * a.s.G + head;
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int k = 0; k < NC; ++k) o[k] = l == 0.f ? 0.f : o[k] * inv;
#pragma unroll
    for (int k = 0; k < NC; k += 8) store16(a.O + row * kD + warp * NC + k, o + k);
    if (warp == 0) a.lse[row] = l == 0.f ? -CUDART_INF_F : (M + log2f(l)) * kLn2;
}

size_t al(size_t x) { return (x + 255) & ~(size_t)255; }
int cap_tiles(const PagedShape &s) { return s.tokens / (2 * (128 / s.G)) + s.B + 1; }

template <int kD, int kCode>
cudaError_t run(const PreArgs &a, int grid, const CUtensorMap &mq, cudaStream_t st) {
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
    if ((e = launch_pdl(paged_plan_kernel, dim3(1), dim3(1024), plan_smem, st, a)) != cudaSuccess) return e;
    note_launch();
    if ((e = launch_pdl(kern, dim3((unsigned)grid), dim3(kThreads), smem_bytes<kD>(), st, mq, a)) != cudaSuccess)
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
    return al(sizeof(PlanHead)) + al(cap_tiles(s) * sizeof(Tile)) + al(kMaxGrid * sizeof(Job)) +
           (size_t)kMaxGrid * 2 * (s.d + 2) * 256 * sizeof(float);
}

cudaError_t launch_paged_prefill(const PagedShape &s, const void *Q, const int32_t *cu, const PagedCache &c, void *O,
                                 float *lse, unsigned *status, void *scratch, cudaStream_t st) {
    PreArgs a{};
    a.s = s;
    a.c = c;
    a.cu = cu;
    a.O = (__nv_bfloat16 *)O;
    a.lse = lse;
    a.status = status;
    a.tpt = 128 / s.G;
    a.cap_tiles = cap_tiles(s);
    unsigned char *w = (unsigned char *)scratch;
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
    if (enc(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(Q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    const int grid = min(sms, kMaxGrid);
    if (s.d == 128)
        return s.code == SA_E4M3 ? run<128, SA_E4M3>(a, grid, mq, st) : run<128, SA_INT8>(a, grid, mq, st);
    return s.code == SA_E4M3 ? run<64, SA_E4M3>(a, grid, mq, st) : run<64, SA_INT8>(a, grid, mq, st);
}

}  // namespace sa
