// paged_decode.cu -- decode over the paged 8-bit cache for bf16 queries: one
// pass over the kept pages, warp-level tensor-core tiles.
//
//   z = scale ks <q, code_k> + gate,   o = sum p vs code_v / sum p,
//   p = 2^(z log2 e - m)
//
// HBM bound: 2 d bytes a key and kv-head, 4 G flops a byte.  So everything is
// built to keep loads in flight and to spend few instructions per byte:
//   * the work is one line of stages (up to 64 keys of one unit: a page, half
//     a page of more than 64 tokens, or several small pages), units one after
//     the other, cut into equal ranges, one per warp of the grid whatever the
//     lengths or lists are.  A warp streams its range by itself, through one
//     stage of shared memory: the next stage's keys are sent for once this
//     one's scores are made, its values once this one's are used; no warp
//     waits for another (twelve warps with a stage each keep more in flight
//     than six with two).  A unit that lies in one range is finished by its
//     warp; the others leave a record (max, sum, acc) per range, at most two a
//     warp, which a second launch joins in range order;
//   * a unit is a list's query heads, up to 16; a chunk of few rows (drafted
//     tokens) is units of 8 or 16 rows, each with its keys per row;
//   * codes become fp16 in registers (exact), so the tensor core multiplies
//     them as they are, and scales stay out of the matrices: a key's scale
//     multiplies its logits, a value's the finished product of its page;
//   * keys are the M side of both products (S^T = K q^T, O^T = V^T P^T): a
//     tile holds 16 keys x 8 query heads, so a group of 4 to 8 heads wastes
//     little, and P^T comes out of S^T by a register transpose (movmatrix);
//   * a matrix row of a tile is any key or dimension as long as both operands
//     agree, so the byte order that ldmatrix gives is used as it is: for S the
//     query is loaded in that order, for O the even and odd dimensions of 16
//     form rows 0-7 and 8-15.
// fp16 queries: each row is scaled by a power of two so that its largest
// element lies in [2^14, 2^15); what falls below fp16's range is under 2^-38
// of the largest.  P is rounded to fp16: half a step, 2^-11, of each weight, or
// 2^-32 of the row's largest where that is more (kWeightLift in paged.cuh); the
// sum counts the weights before they are rounded.
#include <cuda.h>
#include <limits.h>
#include <math_constants.h>

#include "paged.cuh"
#include "tc_ptx.cuh"

namespace sa {
namespace {

using namespace tc;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Ranges (warps) per CTA: one stage of 64 keys each (16 KB at d = 128) fills
// shared memory at 12; two head tiles need more registers than 12 warps have.
template <int kNT>
constexpr int warps_of() { return kNT == 1 ? 12 : 8; }
constexpr int kMaxWarps = 12;
constexpr int kMinRange = 2;   // stages: shorter ranges cost more in records than they save
// stage flags: first / last stage of its unit in this range, the unit lies in
// this range as a whole, it begins before this range, some keys are not there
enum { F_NEW = 1, F_LAST = 2, F_WHOLE = 4, F_CUT = 8, F_TAIL = 16 };

struct DecArgs {
    PagedShape s;
    PagedCache c;
    PagedLists l;
    const __nv_bfloat16 *q;
    __nv_bfloat16 *o;
    float *lse;
    unsigned *status;
    int4 *info;          // [units] first range, ranges (0: nothing to join), list, group
    float *rec;          // [ranges][2] records
    const int32_t *cu;   // packed chunk rows, or null: one query per sequence
    int lists, units;    // B * Hsel lists; the most units (groups of a list's rows) there can be
    int ranges;          // warps of the grid
    int limit;           // chunk: lists of more rows are left to the tiles
    int group;           // rows per group
    int sub, rows, pps;  // stage geometry: parts per page, rows per part, parts per stage
};

// A part's record for the stage that reads it.
struct __align__(16) Part {
    float ks, vs, gate;   // key scale, value scale, gate (hierarchical: score), log2 units
    int nk;               // valid keys (0: not loaded)
};
struct Place {
    int y, nk;            // first cache row of a part, its valid keys
};

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t *r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a));
}
__device__ __forceinline__ void mma_f16(float *c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_h2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Four codes to two fp16 pairs, exactly.  kEven: bytes (0, 2) and (1, 3), else
// (0, 1) and (2, 3).
template <int kCode, bool kEven>
__device__ __forceinline__ void to_h2(uint32_t x, uint32_t &p, uint32_t &q) {
    if (kCode == SA_E4M3) {
        if (kEven) x = __byte_perm(x, 0, 0x3120);
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}" : "=r"(p), "=r"(q) : "r"(x));
    } else {
        // 1024 + (code + 128) under fp16's exponent of 2^10, then minus 1152
        x ^= 0x80808080u;
        uint32_t a = __byte_perm(x, 0x64646464u, kEven ? 0x4240 : 0x4140);
        uint32_t b = __byte_perm(x, 0x64646464u, kEven ? 0x4341 : 0x4342);
        const __half2 off = __half2half2(__ushort_as_half(0x6480));
        __half2 ha = __hsub2(*reinterpret_cast<__half2 *>(&a), off), hb = __hsub2(*reinterpret_cast<__half2 *>(&b), off);
        p = *reinterpret_cast<uint32_t *>(&ha);
        q = *reinterpret_cast<uint32_t *>(&hb);
    }
}
// Byte offset of 16-byte chunk c of row r: the swizzle of the TMA box (128-
// byte rows: chunk ^ row % 8; 64-byte rows: chunk ^ row / 2 % 4).
template <int kD>
__device__ __forceinline__ uint32_t swz(int r, int c) {
    return kD == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// A list and the query rows that read it: the query heads of the list, or with
// a chunk its tokens times the group's heads, token-major.
struct ListAt {
    int b, g, head0;       // head0: first query head of the list, or of the group
    int n, listed;         // keys of the sequence, entries listed
    int first, T, rows;    // chunk: first packed row, tokens; rows that read the list
};
__device__ __forceinline__ ListAt list_at(const DecArgs &a, int lu) {
    const PagedShape &s = a.s;
    ListAt w;
    const int hs = lu % s.Hsel;
    const bool perq = s.flags & SA_SELECT_PER_QHEAD;
    w.b = lu / s.Hsel;
    w.listed = a.l.idx ? a.l.count[lu] : 0;     // all loads in flight
    const int c0 = a.cu ? a.cu[w.b] : 0, c1 = a.cu ? a.cu[w.b + 1] : 0;
    w.n = paged_len(s, a.c.seq_len, w.b);
    w.g = perq ? hs / s.G : hs;
    w.head0 = perq ? hs : hs * s.G;
    w.first = max(0, min(c0, s.tokens));
    w.T = max(w.first, min(c1, s.tokens)) - w.first;
    w.rows = a.cu ? w.T * s.G : s.heads_per;
    return w;
}
// A unit: a group of up to a.group rows of one list, r0 .. r0 + rn - 1.
struct UnitAt {
    ListAt l;
    int r0, rn;
};
__device__ __forceinline__ UnitAt unit_at(const DecArgs &a, int lu, int grp) {
    UnitAt w{list_at(a, lu), grp * a.group, 0};
    w.rn = min(a.group, w.l.rows - w.r0);
    return w;
}
// Row of q, o and lse that the unit's row i is, and the keys it sees.
__device__ __forceinline__ size_t row_at(const DecArgs &a, const UnitAt &w, int i) {
    if (!a.cu) return (size_t)w.l.b * a.s.Hq + w.l.head0 + w.r0 + i;
    const int t = (w.r0 + i) / a.s.G;
    return (size_t)(w.l.first + t) * a.s.Hq + w.l.head0 + (w.r0 + i - t * a.s.G);
}
__device__ __forceinline__ int sees(const DecArgs &a, const ListAt &l, int r) {
    return !a.cu || !(a.s.flags & SA_CAUSAL) ? l.n : l.n - l.T + r / a.s.G + 1;
}
__device__ __forceinline__ int groups_of(const DecArgs &a, const ListAt &l) {
    return l.rows > a.limit ? 0 : (l.rows + a.group - 1) / a.group;
}

// Entries (blocks) of a unit: its list's, or every block that one of its rows
// sees.
__device__ __forceinline__ int entries_of(const DecArgs &a, const ListAt &l, int grp) {
    if (a.l.idx) return l.n > 0 ? max(0, min(l.listed, a.s.cap)) : 0;
    const int n = max(0, min(l.n, sees(a, l, min(l.rows, (grp + 1) * a.group) - 1)));
    return (n + a.s.bs - 1) / a.s.bs;
}
__device__ __forceinline__ int stages_of(const DecArgs &a, int entries) {
    return (entries * a.sub + a.pps - 1) / a.pps;
}

template <int kD, int kNT>
constexpr int rec_floats() { return (kD / 16 * kNT * 4 + 4 * kNT) * 32; }

// Softmax state of one warp: heads 8 nt + 2 tq + {0, 1} per lane, dimensions
// 16 t + 2 gq + {0, 1}.
template <int kD, int kNT>
struct Acc {
    float m[2 * kNT], l[2 * kNT];
    float o[kD / 16][kNT][4];     // [][][e]: dimension 16 t + 2 gq + (e >> 1), head 8 nt + 2 tq + (e & 1)
    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int i = 0; i < 2 * kNT; ++i) {
            m[i] = -CUDART_INF_F;
            l[i] = 0.f;
        }
#pragma unroll
        for (int t = 0; t < kD / 16; ++t)
#pragma unroll
            for (int n = 0; n < kNT; ++n) o[t][n][0] = o[t][n][1] = o[t][n][2] = o[t][n][3] = 0.f;
    }
    __device__ __forceinline__ void scale(const float *f) {
#pragma unroll
        for (int t = 0; t < kD / 16; ++t)
#pragma unroll
            for (int n = 0; n < kNT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[t][n][e] *= f[2 * n + (e & 1)];
    }
    __device__ __forceinline__ void save(float *r, int lane) const {
        int i = 0;
#pragma unroll
        for (int t = 0; t < kD / 16; ++t)
#pragma unroll
            for (int n = 0; n < kNT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) r[32 * i++ + lane] = o[t][n][e];
#pragma unroll
        for (int k = 0; k < 2 * kNT; ++k) {
            r[32 * i++ + lane] = m[k];
            r[32 * i++ + lane] = l[k];
        }
    }
    __device__ __forceinline__ void store(const DecArgs &a, const UnitAt &w, int lane) const {
        const int gq = lane >> 2, tq = lane & 3;
#pragma unroll
        for (int k = 0; k < 2 * kNT; ++k) {
            const int h = 8 * (k >> 1) + 2 * tq + (k & 1);
            if (h >= w.rn) continue;
            const float inv = l[k] > 0.f ? 1.f / l[k] : 0.f;
            const size_t row = row_at(a, w, h);
            __nv_bfloat16 *dst = a.o + row * kD + 2 * gq;
#pragma unroll
            for (int t = 0; t < kD / 16; ++t)
                *reinterpret_cast<__nv_bfloat162 *>(dst + 16 * t) = __floats2bfloat162_rn(
                    l[k] == 0.f ? 0.f : o[t][k >> 1][k & 1] * inv, l[k] == 0.f ? 0.f : o[t][k >> 1][2 + (k & 1)] * inv);
            if (gq == 0) a.lse[row] = l[k] == 0.f ? -CUDART_INF_F : (m[k] + log2f(l[k])) * kLn2;
        }
    }
};

// What a warp loads next: up to 32 parts of one unit, one per lane, in steps
// so that the chain count -> list -> table -> scales is in flight behind the
// stages before it.
struct Batch {
    int list, grp, entries;     // list -1: none
    int s0, s1;                 // stages of the unit
    int flags;                  // F_NEW: s0 is the unit's first stage here; F_LAST: s1 - 1 its last; F_WHOLE, F_CUT
    int step;                   // load steps done
    int page;                   // lane: block, then page of its part (-1: none)
    int nk;                     // lane: valid keys
    float gate, ks, vs;
};

// kSingle: a stage is one part, so one page.  Every stage is worked through as
// 64 keys without a branch (a missing tile's keys are masked like a missing
// key): branches around the tiles had cut the arithmetic into pieces too short
// to hide its latencies, 1.6 times the time.
template <int kD, int kCode, int kNT, bool kSingle>
__global__ void __launch_bounds__(32 * warps_of<kNT>(), 1)
paged_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, DecArgs a) {
    constexpr uint32_t kHalfBytes = 64 * kD;
    constexpr int kWarps = warps_of<kNT>(), kThreads = 32 * kWarps;
    extern __shared__ unsigned char dec_raw[];
    unsigned char *sm = reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(dec_raw) + 1023) &
                                                          ~uintptr_t(1023));
    __shared__ Part parts[kWarps][2][32];     // of two batches
    __shared__ Place places[kWarps][32];      // of the batch being issued
    __shared__ uint64_t bars[kWarps][2];      // the warp's keys, its values
    __shared__ long long pre[kThreads + 1];
    __shared__ long long wtot[kWarps];
    __shared__ int preu[kThreads + 1], wtotu[kWarps];
    __shared__ volatile int abort_s, bad_s;
    const PagedShape &s = a.s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gq = lane >> 2, tq = lane & 3;
    const bool hier = s.flags & SA_HIER;
    if (tid == 0) {
        for (int i = 0; i < kWarps * 2; ++i) mbar_init(smem_u32(&bars[0][0] + i), 1);
        abort_s = 0;
        bad_s = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    __syncthreads();

    // ---- the line of stages: offsets of each thread's share of the lists ------
    const int share = (a.lists + kThreads - 1) / kThreads;
    const int l0 = min(a.lists, tid * share), l1 = min(a.lists, l0 + share);
    {
        long long n = 0;
        int nu = 0;
        bool none = false;        // a unit of this CTA's lists keeps nothing
        for (int lu = l0; lu < l1; ++lu) {
            const ListAt l = list_at(a, lu);
            if (a.cu && !(a.cu[l.b] >= 0 && a.cu[l.b] <= a.cu[l.b + 1] && a.cu[l.b + 1] <= s.tokens)) bad_s = 1;
            const int ng = groups_of(a, l);
            for (int grp = 0; grp < ng; ++grp) {
                const int e = entries_of(a, l, grp);
                n += stages_of(a, e);
                none |= e == 0 && lu % gridDim.x == blockIdx.x;
            }
            nu += ng;
        }
        long long inc = n;
        int incu = nu;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(~0u, inc, o);
            const int yu = __shfl_up_sync(~0u, incu, o);
            if (lane >= o) {
                inc += y;
                incu += yu;
            }
        }
        if (lane == 31) {
            wtot[warp] = inc;
            wtotu[warp] = incu;
        }
        __syncthreads();
        for (int w = 0; w < warp; ++w) {
            inc += wtot[w];
            incu += wtotu[w];
        }
        pre[tid] = inc - n;
        preu[tid] = incu - nu;
        if (tid == kThreads - 1) {
            pre[kThreads] = inc;
            preu[kThreads] = incu;
        }
        __syncthreads();
        if (bad_s) {
            // a chunk's offsets do not ascend within its rows: nothing is done
            for (int id = blockIdx.x * kThreads + tid; id < a.units; id += gridDim.x * kThreads)
                a.info[id] = make_int4(0, 0, 0, 0);
            if (tid == 0) set_status(a.status, kStatusBadIndex);
            return;
        }
        if (none) {
            int id = incu - nu;
            for (int lu = l0; lu < l1; ++lu) {
                const ListAt l = list_at(a, lu);
                const int ng = groups_of(a, l);
                for (int grp = 0; grp < ng; ++grp, ++id) {
                    if (entries_of(a, l, grp) > 0 || lu % gridDim.x != blockIdx.x) continue;
                    // nothing kept: zeros
                    a.info[id] = make_int4(0, 0, 0, 0);
                    const UnitAt w = unit_at(a, lu, grp);
                    for (int h = 0; h < w.rn; ++h) {
                        const size_t row = row_at(a, w, h);
                        for (int i = 0; i < kD; i += 8)
                            *reinterpret_cast<uint4 *>(a.o + row * kD + i) = make_uint4(0, 0, 0, 0);
                        a.lse[row] = -CUDART_INF_F;
                    }
                }
            }
        }
        // units that this call does not have
        for (int id = preu[kThreads] + blockIdx.x * kThreads + tid; id < a.units; id += gridDim.x * kThreads)
            a.info[id] = make_int4(0, 0, 0, 0);
    }
    const long long total = pre[kThreads];
    const long long per = max((long long)kMinRange, (total + a.ranges - 1) / a.ranges);
    // neighbouring ranges go to different SMs, so that a small call spreads out
    const int range = warp * gridDim.x + blockIdx.x;
    const long long x0 = range * per, x1 = min(total, x0 + per);
    if (x0 >= x1) return;

    // ---- issue side ----------------------------------------------------------
    int batch = 1;                     // batches issued (records alternate between two places)
    // The unit of stage xi, the next one to put in a batch: list, group, number
    // in the call, and its first stage.
    int wl, wg = 0, wid;
    long long bpu, xi = x0;
    {
        int best = 0;
        for (int t = lane; t < kThreads; t += 32)
            if (pre[t] <= x0) best = t;
        best = __reduce_max_sync(~0u, best);
        wl = best * share;
        bpu = pre[best];
        wid = preu[best];
    }
    ListAt wlist = list_at(a, wl);
    // step 0: unit and part of the line
    auto open = [&](Batch &t) {
        t.step = 0;
        t.list = -1;
        if (xi >= x1) return;
        int n;
        for (;;) {
            if (wg == groups_of(a, wlist)) {
                wg = 0;
                wlist = list_at(a, ++wl);
                continue;
            }
            t.entries = entries_of(a, wlist, wg);
            n = stages_of(a, t.entries);
            if (xi < bpu + n) break;
            bpu += n;
            ++wg;
            ++wid;
        }
        t.list = wl;
        t.grp = wg;
        t.s0 = (int)(xi - bpu);
        t.s1 = (int)min((long long)min(n, t.s0 + 32 / a.pps), x1 - bpu);
        t.flags = (t.s0 == 0 || xi == x0 ? F_NEW : 0) | (t.s1 == n || bpu + t.s1 == x1 ? F_LAST : 0) |
                  (bpu < x0 ? F_CUT : 0) | (bpu >= x0 && bpu + n <= x1 ? F_WHOLE : 0);
        if (t.s0 == 0 && lane == 0) {
            // how many ranges the unit's first one shares it with
            const int r1 = (int)((bpu + n - 1) / per);
            a.info[wid] = r1 == range ? make_int4(0, 0, 0, 0) : make_int4(range, r1 - range + 1, wl, wg);
        }
        xi = bpu + t.s1;
        t.step = 1;
    };
    // steps 1 to 3, one dependent load each
    auto more = [&](Batch &t) {
        const ListAt w = list_at(a, t.list);
        if (t.step == 1) {
            const int c = t.s0 * a.pps + lane, e = c / a.sub;
            t.page = -1;
            t.gate = 0.f;
            t.nk = 0;
            if (lane < (t.s1 - t.s0) * a.pps && e < t.entries) {
                const int n = w.n, local = (n + s.bs - 1) / s.bs - 1;
                int blk = e;
                if (a.l.idx) {
                    const int32_t *il = a.l.idx + (size_t)t.list * s.cap;
                    const float *sc = a.l.score + (size_t)t.list * s.cap;
                    const int before = e > 0 ? il[e - 1] : -1;
                    const float mine = sc[e], loc = sc[t.entries - 1];
                    blk = il[e];
                    if (blk <= before || blk < 0 || blk > local) {
                        set_status(a.status, kStatusBadIndex);
                        blk = -1;
                    }
                    const bool forced = (blk == local && (s.flags & SA_LOCAL)) || (blk == 0 && (s.flags & SA_SINK));
                    t.gate = hier ? mine * kLog2e
                                  : ((s.flags & SA_GATE) && !forced ? log_sigmoid(mine - loc) * kLog2e : 0.f);
                }
                const int row0 = (c - e * a.sub) * a.rows;
                t.nk = min(min(a.rows, s.bs - row0), n - blk * s.bs - row0);
                if (t.nk > 0) t.page = blk;
            }
        } else if (t.step == 2) {
            if (t.page >= 0) {
                t.page = a.c.table[(size_t)w.b * s.maxb + t.page];
                if (t.page < 0 || t.page >= s.pages) {
                    set_status(a.status, kStatusBadIndex);
                    t.page = -1;
                }
            }
        } else {
            const int ph = max(t.page, 0) * s.Hkv + w.g;
            if (t.page < 0) t.nk = 0;
            places[warp][lane] = Place{ph * s.bs + (t.s0 * a.pps + lane) % a.sub * a.rows, t.nk};
            // in flight while the first stage's keys are sent for
            t.ks = t.page >= 0 ? a.c.ks[ph] : 0.f;
            t.vs = t.page >= 0 ? a.c.vs[ph] : 0.f;
            __syncwarp();
        }
        ++t.step;
    };
    // The batch being issued (its records are in shared memory) and the one
    // being loaded behind it, whose last step waits until it takes over.
    Batch nxt{};
    // list, group, first stage, stages, flags, stages issued
    int cu_list = -1, cu_grp = 0, cu_s0 = 0, cu_n = 0, cu_flags = 0, ci = 0;
    const uint32_t kb = smem_u32(sm) + warp * 2 * kHalfBytes, vb = kb + kHalfBytes;
    const uint32_t bar_k = smem_u32(&bars[warp][0]), bar_v = smem_u32(&bars[warp][1]);
    const uint32_t part_bytes = (uint32_t)a.rows * kD;
    // tile t of a stage lies in part t >> psh, as its (t & pmask)th 16 keys
    const int psh = kSingle ? 2 : (a.rows >> 4) - 1, pmask = (1 << psh) - 1;
    // The next stage: its keys go out once the stage at hand has made its
    // scores, its values once that one has used its own, so one stage of
    // memory keeps one load in flight behind the arithmetic.
    uint32_t n_bytes = 0;
    // flags, list, group, first part (with the batch's half) and first key of that stage
    int n_flags = 0, n_list = 0, n_grp = 0, n_first = 0, n_key = 0;
    auto issue_k = [&]() -> bool {              // false: the range is issued
        const bool fresh = ci == cu_n;
        if (fresh) {
            if (nxt.list < 0) return false;
            ++batch;
            while (nxt.step < 4) more(nxt);
            cu_list = nxt.list;
            cu_grp = nxt.grp;
            cu_s0 = nxt.s0;
            cu_n = nxt.s1 - nxt.s0;
            cu_flags = nxt.flags;
            ci = 0;
        }
        const int first = ci * a.pps;
        const Place at = places[warp][min(31, first + lane)];
        const bool live = lane < a.pps && at.nk > 0;
        n_bytes = part_bytes * __popc(__ballot_sync(~0u, live));
        n_first = 32 * (batch & 1) + first;
        n_list = cu_list;
        n_grp = cu_grp;
        if (a.cu) {
            // every block in order: where the stage's keys lie, and whether
            // the unit's first row sees them all
            const int c = (cu_s0 + ci) * a.pps;
            n_key = c / a.sub * s.bs + c % a.sub * a.rows;
        }
        n_flags = (cu_flags & (F_WHOLE | F_CUT)) | (ci == 0 ? cu_flags & F_NEW : 0) |
                  (ci == cu_n - 1 ? cu_flags & F_LAST : 0) |
                  (__any_sync(~0u, lane < a.pps && at.nk < (kSingle ? 64 : a.rows)) ? F_TAIL : 0);
        if (lane == 0) {
            if (n_bytes) mbar_expect_tx(bar_k, n_bytes);
            else mbar_arrive(bar_k);
        }
        __syncwarp();
        if (live) tma_load_2d(kb + lane * part_bytes, &tmK, bar_k, 0, at.y);
        if (fresh) {
            // the records go where the batch before the last one had its own
            parts[warp][batch & 1][lane] = Part{nxt.ks, nxt.vs, nxt.gate, nxt.nk};
            open(nxt);
            __syncwarp();
        }
        return true;
    };
    auto issue_v = [&]() {
        if (lane == 0) {
            if (n_bytes) mbar_expect_tx(bar_v, n_bytes);
            else mbar_arrive(bar_v);
        }
        __syncwarp();
        const Place at = places[warp][min(31, ci * a.pps + lane)];
        if (lane < a.pps && at.nk > 0) tma_load_2d(vb + lane * part_bytes, &tmV, bar_v, 0, at.y);
        ++ci;
        if (nxt.list >= 0 && nxt.step < 3) more(nxt);
    };
    open(nxt);

    // ---- consumer side -------------------------------------------------------
    Acc<kD, kNT> acc;
    uint32_t qb[kD / 16][kNT][2];
    float qf[2 * kNT];
    int lim[2 * kNT], lim0 = 0;        // chunk: keys that the lane's rows see, that the unit's first row sees
    int done = 0;
    // v_out: this stage's values are on their way; k_next: the next one's keys
    bool ok = true, have = issue_k(), v_out = have, k_next = false;
    if (have) issue_v();
    for (; have; ++done) {
        const int flags = n_flags, list = n_list, grp = n_grp, key0 = n_key;
        const Part *part = &parts[warp][0][n_first];
        if (flags & F_NEW) {
            // the unit's queries: dimensions 16 k + 4 tq + {0, 1}, {2, 3} of head 8 n + gq
            const UnitAt w = unit_at(a, list, grp);
            acc.reset();
            if (a.cu) {
                lim0 = sees(a, w.l, w.r0);
#pragma unroll
                for (int i = 0; i < 2 * kNT; ++i) lim[i] = sees(a, w.l, w.r0 + 8 * (i >> 1) + 2 * tq + (i & 1));
            }
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
                const int h = 8 * n + gq;
                const __nv_bfloat16 *src = a.q + row_at(a, w, h < w.rn ? h : 0) * kD + 4 * tq;
                uint2 x[kD / 16];
                unsigned big = 0;      // largest magnitude's bits
#pragma unroll
                for (int k = 0; k < kD / 16; ++k) {
                    x[k] = h < w.rn ? *reinterpret_cast<const uint2 *>(src + 16 * k) : make_uint2(0, 0);
                    const unsigned y = __vmaxu2(x[k].x & 0x7fff7fffu, x[k].y & 0x7fff7fffu);
                    big = __vmaxu2(big, y);
                }
                big = max(big & 0xffffu, big >> 16);
                big = max(big, __shfl_xor_sync(~0u, big, 1));
                big = max(big, __shfl_xor_sync(~0u, big, 2));
                // 2^(14 - exponent), within fp32's normal powers
                const int e = (int)(big >> 7) - 127;
                const int up = max(-113, min(126, 14 - e));
                const float f = __uint_as_float((unsigned)(up + 127) << 23);
#pragma unroll
                for (int k = 0; k < kD / 16; ++k) {
                    const float2 lo = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&x[k].x));
                    const float2 hi = __bfloat1622float2(*reinterpret_cast<__nv_bfloat162 *>(&x[k].y));
                    qb[k][n][0] = pack_h2(lo.x * f, lo.y * f);
                    qb[k][n][1] = pack_h2(hi.x * f, hi.y * f);
                }
                // logit factor of the heads this lane's S columns hold
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int up2 = __shfl_sync(~0u, up, (2 * tq + i) * 4);
                    qf[2 * n + i] = s.scale * kLog2e * __uint_as_float((unsigned)(127 - up2) << 23);
                }
            }
        }
        ok = mbar_wait_lazy(bar_k, done & 1, &abort_s, a.status);
        if (!__all_sync(~0u, ok)) break;
        const int mrow = (lane & 7) + (lane & 8), mch = lane >> 4;   // row and chunk of the lane's ldmatrix address
        // S^T = K q^T: 16 keys x 8 heads per tile
        float z[4][kNT][4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int n = 0; n < kNT; ++n) z[t][n][0] = z[t][n][1] = z[t][n][2] = z[t][n][3] = 0.f;
#pragma unroll
        for (int k = 0; k < kD / 32; ++k) {
            uint32_t kr[4][4];
#pragma unroll
            for (int t = 0; t < 4; ++t)
                ldsm4(kb + swz<kD>(16 * t + mrow, 2 * k + mch), kr[t]);
#pragma unroll
            for (int half = 0; half < 2; ++half)
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint32_t *r = kr[t] + 2 * half;
                    uint32_t p0, q0, p1, q1;
                    to_h2<kCode, false>(r[0], p0, q0);
                    to_h2<kCode, false>(r[1], p1, q1);
#pragma unroll
                    for (int n = 0; n < kNT; ++n)
                        mma_f16(z[t][n], p0, p1, q0, q1, qb[2 * k + half][n][0], qb[2 * k + half][n][1]);
                }
        }
        __syncwarp();
        k_next = issue_k();
        // logits in log2 units, -inf where there is no key
        float top[2 * kNT];
#pragma unroll
        for (int i = 0; i < 2 * kNT; ++i) top[i] = -CUDART_INF_F;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            const Part pt = part[t >> psh];
#pragma unroll
            for (int n = 0; n < kNT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    z[t][n][e] = fmaf(z[t][n][e], qf[2 * n + (e & 1)] * pt.ks, hier ? 0.f : pt.gate);
        }
        if ((flags & F_TAIL) || (a.cu && key0 + 64 > lim0)) {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int nk = part[t >> psh].nk - 16 * (t & pmask), k0 = key0 + 16 * t;
#pragma unroll
                for (int n = 0; n < kNT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int k = gq + 8 * (e >> 1);
                        const bool on = k < nk && (!a.cu || k0 + k < lim[2 * n + (e & 1)]);
                        z[t][n][e] = on ? z[t][n][e] : -CUDART_INF_F;
                    }
            }
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int n = 0; n < kNT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) top[2 * n + (e & 1)] = fmaxf(top[2 * n + (e & 1)], z[t][n][e]);
        float pf[2 * kNT];     // hierarchical: weight of the block over its sum
        if (!hier) {
            bool high = false;
#pragma unroll
            for (int i = 0; i < 2 * kNT; ++i) high |= top[i] > acc.m[i] + (kWeightLift + kWeightSlack);
            if (__any_sync(~0u, high)) {
                float f[2 * kNT];
#pragma unroll
                for (int i = 0; i < 2 * kNT; ++i) {
                    float x = top[i];
                    x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
                    x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
                    x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
                    x = fmaxf(x - kWeightLift, acc.m[i]);
                    f[i] = acc.m[i] == -CUDART_INF_F ? 0.f : ex2(acc.m[i] - x);
                    acc.m[i] = x;
                    acc.l[i] *= f[i];
                }
                acc.scale(f);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2 * kNT; ++i) {
                float x = top[i];
                x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
                x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
                top[i] = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
            }
        }
        float sum[2 * kNT];
#pragma unroll
        for (int i = 0; i < 2 * kNT; ++i) sum[i] = 0.f;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int n = 0; n < kNT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int i = 2 * n + (e & 1);
                    const float ref = hier ? top[i] : acc.m[i];
                    const float p = ex2(z[t][n][e] - (ref == -CUDART_INF_F ? 0.f : ref));
                    z[t][n][e] = p;
                    sum[i] += p;
                }
        if (hier) {
            const float score = part[0].gate;
            float f[2 * kNT];
#pragma unroll
            for (int i = 0; i < 2 * kNT; ++i) {
                float lb = sum[i];
                lb += __shfl_xor_sync(~0u, lb, 4);
                lb += __shfl_xor_sync(~0u, lb, 8);
                lb += __shfl_xor_sync(~0u, lb, 16);
                f[i] = 1.f;
                pf[i] = 0.f;
                // 0: no key (a query that is not a number goes on); -inf: no weight
                if (lb != 0.f && score != -CUDART_INF_F) {
                    // nothing is held back here: the weights get all the room
                    const float M = fmaxf(acc.m[i], score - (kWeightLift + kWeightSlack));
                    f[i] = acc.m[i] == -CUDART_INF_F ? 0.f : ex2(acc.m[i] - M);
                    const float w = ex2(score - M);
                    acc.m[i] = M;
                    // the sum over lanes at the end counts it once
                    acc.l[i] = acc.l[i] * f[i] + (gq == 0 ? w : 0.f);
                    pf[i] = w / lb;
                }
            }
            acc.scale(f);
        } else {
#pragma unroll
            for (int i = 0; i < 2 * kNT; ++i) acc.l[i] += sum[i];
        }
        // P^T as the second operand: keys 16 t + 2 tq + {0, 1} (+ 8), head 8 n + gq
        uint32_t pb[4][kNT][2];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int n = 0; n < kNT; ++n) {
                const float f0 = hier ? pf[2 * n] : 1.f, f1 = hier ? pf[2 * n + 1] : 1.f;
                pb[t][n][0] = transpose8(pack_h2(z[t][n][0] * f0, z[t][n][1] * f1));
                pb[t][n][1] = transpose8(pack_h2(z[t][n][2] * f0, z[t][n][3] * f1));
            }
        // O^T += V^T P^T, 32 dimensions at a time
        ok = mbar_wait_lazy(bar_v, done & 1, &abort_s, a.status);
        if (!__all_sync(~0u, ok)) break;
        const float vs0 = part[0].vs;
        const bool blank = kCode == SA_E4M3 && (flags & F_TAIL);   // what is not a key may hold NaN codes
#pragma unroll
        for (int np = 0; np < kD / 32; ++np) {
            uint32_t vr[4][4];
#pragma unroll
            for (int t = 0; t < 4; ++t)
                ldsm4t(vb + swz<kD>(16 * t + mrow, 2 * np + mch), vr[t]);
            float d[2][kNT][4];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int n = 0; n < kNT; ++n) d[h][n][0] = d[h][n][1] = d[h][n][2] = d[h][n][3] = 0.f;
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                uint32_t *r = vr[t];
                if (blank) {
                    const int nk = part[t >> psh].nk - 16 * (t & pmask);
                    const uint32_t m0 = (2 * tq < nk ? 0xffffu : 0u) | (2 * tq + 1 < nk ? 0xffff0000u : 0u);
                    const uint32_t m1 = (2 * tq + 8 < nk ? 0xffffu : 0u) | (2 * tq + 9 < nk ? 0xffff0000u : 0u);
                    r[0] &= m0;
                    r[1] &= m1;
                    r[2] &= m0;
                    r[3] &= m1;
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t a0, a1, a2, a3;
                    to_h2<kCode, true>(r[2 * h], a0, a1);
                    to_h2<kCode, true>(r[2 * h + 1], a2, a3);
#pragma unroll
                    for (int n = 0; n < kNT; ++n) mma_f16(d[h][n], a0, a1, a2, a3, pb[t][n][0], pb[t][n][1]);
                }
                if constexpr (!kSingle) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int n = 0; n < kNT; ++n)
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                acc.o[2 * np + h][n][e] = fmaf(part[t >> psh].vs, d[h][n][e], acc.o[2 * np + h][n][e]);
                                d[h][n][e] = 0.f;
                            }
                }
            }
            if constexpr (kSingle) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int n = 0; n < kNT; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            acc.o[2 * np + h][n][e] = fmaf(vs0, d[h][n][e], acc.o[2 * np + h][n][e]);
            }
        }
        __syncwarp();
        have = v_out = k_next;
        k_next = false;
        if (have) issue_v();
        if (flags & F_LAST) {
#pragma unroll
            for (int i = 0; i < 2 * kNT; ++i) {
                acc.l[i] += __shfl_xor_sync(~0u, acc.l[i], 4);
                acc.l[i] += __shfl_xor_sync(~0u, acc.l[i], 8);
                acc.l[i] += __shfl_xor_sync(~0u, acc.l[i], 16);
            }
            if (flags & F_WHOLE) acc.store(a, unit_at(a, list, grp), lane);
            else acc.save(a.rec + ((size_t)range * 2 + (flags & F_CUT ? 0 : 1)) * rec_floats<kD, kNT>(), lane);
        }
    }
    if (!ok) {
        // a wait ran out: let the copies in flight land before the CTA exits
        // (the keys of this stage or of the next, the values of this stage)
        volatile int never = 0;
        if (v_out) mbar_wait_lazy(bar_v, done & 1, &never, a.status);
        mbar_wait_lazy(bar_k, done & 1, &never, a.status);
        if (k_next) mbar_wait_lazy(bar_k, (done + 1) & 1, &never, a.status);
    }
}

// Joins the records of the units that several ranges shared, in their order.
// A warp takes an eighth of the lanes' values (and every row's max and sum) of
// its group's share of the records, four records at a time; groups meet in
// shared memory.  One group of 256 threads while there are more units than
// SMs (few records each), three where few units have many records.
constexpr int kSlices = 8, kBatch = 4;
template <int kD, int kNT, int kGroups>
__global__ void __launch_bounds__(32 * kSlices * kGroups)
paged_merge_kernel(DecArgs a) {
    constexpr int NO = kD / 16 * kNT * 4, K = NO / kSlices, H = 2 * kNT;
    __shared__ float part[kGroups > 1 ? kGroups - 1 : 1][kSlices][K + 2 * H][32];
    const int u = blockIdx.x, lane = threadIdx.x & 31, slice = (threadIdx.x >> 5) % kSlices;
    const int grp = threadIdx.x / (32 * kSlices), i0 = slice * K;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int4 in = a.info[u];
    // a range whose wait ran out may have left the entry of another call
    if (in.y < 2 || in.x < 0 || in.y > a.ranges - in.x || in.z < 0 || in.z >= a.lists || in.w < 0 ||
        in.w >= a.units)
        return;
    // the entry of the lane's rows that value k of the slice belongs to (a
    // slice is whole tiles of 4 kNT values, or at d = 64 a part of one)
    auto pick = [&](const float *f, int k) {
        if constexpr (K >= 4 * kNT || kNT == 1) return f[2 * (k / 4 % kNT) + (k & 1)];
        else return (slice * K / 4) % kNT ? f[2 + (k & 1)] : f[k & 1];
    };
    float m[H], l[H], o[K];
#pragma unroll
    for (int h = 0; h < H; ++h) {
        m[h] = -CUDART_INF_F;
        l[h] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < K; ++k) o[k] = 0.f;
    const int share = (in.y + kGroups - 1) / kGroups, r0 = grp * share, r1 = min(in.y, r0 + share);
    for (int r = r0; r < r1; r += kBatch) {
        float xm[kBatch][H], xl[kBatch][H], xo[kBatch][K];
#pragma unroll
        for (int c = 0; c < kBatch; ++c) {
            if (r + c >= r1) continue;
            const float *p = a.rec + ((size_t)(in.x + r + c) * 2 + (r + c == 0 ? 1 : 0)) * rec_floats<kD, kNT>() + lane;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                xm[c][h] = p[32 * (NO + 2 * h)];
                xl[c][h] = p[32 * (NO + 2 * h + 1)];
            }
#pragma unroll
            for (int k = 0; k < K; ++k) xo[c][k] = p[32 * (i0 + k)];
        }
        float f[H];
#pragma unroll
        for (int h = 0; h < H; ++h) {
            float M = m[h];
#pragma unroll
            for (int c = 0; c < kBatch; ++c)
                if (r + c < r1) M = fmaxf(M, xm[c][h]);
            f[h] = m[h] == -CUDART_INF_F ? 0.f : ex2(m[h] - M);
            m[h] = M;
            l[h] *= f[h];
        }
#pragma unroll
        for (int k = 0; k < K; ++k) o[k] *= pick(f, k);
#pragma unroll
        for (int c = 0; c < kBatch; ++c) {
            if (r + c >= r1) continue;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                f[h] = xm[c][h] == -CUDART_INF_F ? 0.f : ex2(xm[c][h] - m[h]);
                l[h] += xl[c][h] * f[h];
            }
#pragma unroll
            for (int k = 0; k < K; ++k) o[k] += xo[c][k] * pick(f, k);
        }
    }
    if constexpr (kGroups > 1) {
        if (grp) {
            float(*p)[32] = part[grp - 1][slice];
#pragma unroll
            for (int k = 0; k < K; ++k) p[k][lane] = o[k];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                p[K + 2 * h][lane] = m[h];
                p[K + 2 * h + 1][lane] = l[h];
            }
        }
        __syncthreads();
        if (grp) return;
#pragma unroll
        for (int c = 0; c < kGroups - 1; ++c) {
            const float(*p)[32] = part[c][slice];
            float fa[H], fb[H];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float m2 = p[K + 2 * h][lane], l2 = p[K + 2 * h + 1][lane], M = fmaxf(m[h], m2);
                fa[h] = m[h] == -CUDART_INF_F ? 0.f : ex2(m[h] - M);
                fb[h] = m2 == -CUDART_INF_F ? 0.f : ex2(m2 - M);
                l[h] = l[h] * fa[h] + l2 * fb[h];
                m[h] = M;
            }
#pragma unroll
            for (int k = 0; k < K; ++k) o[k] = o[k] * pick(fa, k) + p[k][lane] * pick(fb, k);
        }
    }
    const UnitAt w = unit_at(a, in.z, in.w);
    const int gq = lane >> 2, tq = lane & 3;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int i = i0 + k, row = 8 * (i / 4 % kNT) + 2 * tq + (i & 1);
        const float lk = pick(l, k);
        if (row < w.rn)
            a.o[row_at(a, w, row) * kD + 16 * (i / (4 * kNT)) + 2 * gq + (i >> 1 & 1)] =
                __float2bfloat16_rn(lk == 0.f ? 0.f : o[k] / lk);
    }
    if (slice == 0 && gq == 0) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
            const int row = 8 * (h >> 1) + 2 * tq + (h & 1);
            if (row < w.rn) a.lse[row_at(a, w, row)] = l[h] == 0.f ? -CUDART_INF_F : (m[h] + log2f(l[h])) * kLn2;
        }
    }
}

// Rows of codes [rows][d], one byte each, read in boxes of box_rows rows.
bool code_map(CUtensorMap *map, const uint8_t *base, uint64_t rows, int d, int box_rows) {
    auto enc = tensor_map_encoder();
    if (!enc) return false;
    cuuint64_t dims[2] = {(cuuint64_t)d, rows};
    cuuint64_t strides[1] = {(cuuint64_t)d};
    cuuint32_t box[2] = {(cuuint32_t)d, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Rows that read one list: the heads of a decode, or on average those of a
// chunk (the packed rows know no more on the host).
long long rows_per_list(const PagedShape &s, bool chunk) {
    return chunk ? ((long long)s.tokens * s.G + s.B - 1) / s.B : s.heads_per;
}
int head_tiles(const PagedShape &s, bool chunk) { return rows_per_list(s, chunk) <= 8 ? 1 : 2; }
int rows_per_group(const PagedShape &s, bool chunk) { return chunk ? 8 * head_tiles(s, true) : 16; }
// A chunk call of few rows, on average (16 a sequence) and in all (1024).
bool few_in_all(const PagedShape &s) {
    return (long long)s.tokens * s.G <= max(256, min(16 * s.B, 1024));
}
// The most units a call can have: a chunk's rows are shared out over the
// sequences on the device.
long long units_of(const PagedShape &s, bool chunk) {
    const int group = rows_per_group(s, chunk);
    if (!chunk) return (long long)s.B * s.Hsel * ((s.heads_per + group - 1) / group);
    const long long any = (long long)s.tokens * s.G / group + s.B;
    const int limit = few_in_all(s) ? INT_MAX : paged_rows_limit(s, true);
    return min(any, limit == INT_MAX ? any : (long long)s.B * ((limit + group - 1) / group)) * s.Hkv;
}
size_t rec_bytes(const PagedShape &s, bool chunk) {
    return (size_t)(s.d / 16 * 4 + 4) * head_tiles(s, chunk) * 32 * sizeof(float);
}
// Without lists a kv-head's rows go together, whoever would select: with
// SA_SELECT_PER_QHEAD left on, every query head read the cache for itself (4
// heads a kv-head, 32 ragged sequences up to 32K: 655 us against 190).
PagedShape without_lists(PagedShape s, bool chunk) {
    s.flags &= chunk ? SA_CAUSAL : ~SA_SELECT_PER_QHEAD;
    s.Hsel = s.Hkv;
    s.heads_per = s.G;
    return s;
}
// The workspace counts the 148 SMs of a B200; the grid follows the device.
constexpr int kMaxGrid = 148;

template <int kD, int kCode, int kNT>
cudaError_t run(DecArgs a, int grid, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t st) {
    a.ranges = grid * warps_of<kNT>();
    constexpr int smem = warps_of<kNT>() * 2 * 64 * kD + 1024;
    auto kern = a.pps == 1 ? paged_decode_kernel<kD, kCode, kNT, true> : paged_decode_kernel<kD, kCode, kNT, false>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kern, dim3((unsigned)grid), dim3(32 * warps_of<kNT>()), smem, st, mk, mv, a);
    note_launch();
    if (e != cudaSuccess) return e;
    e = a.units > grid ? launch_pdl(paged_merge_kernel<kD, kNT, 1>, dim3((unsigned)a.units), dim3(32 * kSlices), 0, st, a)
                       : launch_pdl(paged_merge_kernel<kD, kNT, 3>, dim3((unsigned)a.units), dim3(96 * kSlices), 0, st, a);
    note_launch();
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// bf16; a hierarchical block's softmax needs the block in one stage.
bool paged_decode_supported(const PagedShape &s) {
    return s.dtype == SA_BF16 && !((s.flags & SA_HIER) && s.bs > 64);
}

// A sequence of few rows is read once per 16 of them here, at the decode's
// rate; the tiles of paged_prefill.cu take 256 rows in about twice the time of
// one such pass, so up to some 40 rows a kv-head are better off here (8
// sequences of 5000 keys with 20 rows: 42 us against 56; 64 of 4000 with 40:
// 306 against 412).  How the rows are shared out is known on the device only.
// Most calls run both kernels, each over its own sequences: 512 + 63 x 1 tokens
// over 64 x 16K keys take 542 us, all of them here 1090, all in tiles 1685.  The
// tile kernel's three launches cost up to 20 us when no sequence is theirs (64 x
// 4 tokens at 4000 keys 146 us with, 131 without), so a call of few rows runs
// here as a whole, as long as a chunk that hides in it cannot read too much
// again: all the rows may be one sequence's, and that as long as its table, so
// the bytes of those passes are held to 512 MB, about 80 us, four times what
// the launches cost.  With tables for 128K keys, as a whole and by both kernels:
// 63 + 1 tokens at 128K 755 and 304 us, 192 at 128K + 64 x 1 at 2K 2138 and 533,
// 897 + 127 x 1 of one head a kv-head 3328 and 697; where no chunk hides, 64 x 4
// tokens at 4000 keys 131 and 146, 8 x 5 at 5000 62 and 76.
// `least`: as with the longest tables.
int paged_rows_limit(const PagedShape &s, bool least) {
    constexpr int kFew = 40;
    constexpr long long kHidden = 512ll << 20;
    const long long rows = (long long)s.tokens * s.G;
    if (s.dtype != SA_BF16 || s.tokens <= 0 || rows >= (1ll << 30)) return 0;
    if (s.G > 128) return INT_MAX;
    if (rows <= kFew) return INT_MAX;
    if (s.B == 1) return 0;
    const int group = rows_per_group(s, true);
    const long long pass = 2ll * s.maxb * s.bs * s.Hkv * s.d;    // bytes of the longest sequence
    return few_in_all(s) && !least && (rows + group - 1) / group <= kHidden / pass ? INT_MAX : kFew;
}

size_t paged_decode_scratch(const PagedShape &shape, bool chunk) {
    auto need = [&](const PagedShape &s) {
        return ((units_of(s, chunk) * sizeof(int4) + 255) & ~(size_t)255) +
               (size_t)kMaxGrid * kMaxWarps * 2 * rec_bytes(s, chunk);
    };
    return max(need(shape), need(without_lists(shape, chunk)));
}

cudaError_t launch_paged_decode(const PagedShape &shape, const void *q, const int32_t *cu, const PagedCache &c,
                                const PagedLists &l, void *o, float *lse, unsigned *status, void *scratch,
                                cudaStream_t st) {
    const bool chunk = cu != nullptr;
    const PagedShape s = l.idx ? shape : without_lists(shape, chunk);
    DecArgs a{};
    a.s = s;
    a.c = c;
    a.l = l;
    a.cu = cu;
    a.limit = chunk ? paged_rows_limit(s) : INT_MAX;
    a.q = (const __nv_bfloat16 *)q;
    a.o = (__nv_bfloat16 *)o;
    a.lse = lse;
    a.status = status;
    a.lists = s.B * s.Hsel;
    a.group = rows_per_group(s, chunk);
    a.units = (int)units_of(s, chunk);
    a.info = (int4 *)scratch;
    a.rec = (float *)((unsigned char *)scratch + (((size_t)a.units * sizeof(int4) + 255) & ~(size_t)255));
    // a page of up to 64 tokens is one part, a longer one two; small pages
    // share a stage (not in hierarchical mode, where a stage is one block)
    a.sub = s.bs > 64 ? 2 : 1;
    a.rows = s.bs > 64 ? (s.bs + 31) / 32 * 16 : s.bs;
    a.pps = (s.flags & SA_HIER) ? 1 : 64 / a.rows;
    const int sms = sm_count();
    if (sms <= 0) return cudaErrorNoDevice;
    CUtensorMap mk, mv;
    const uint64_t rows = (uint64_t)s.pages * s.Hkv * s.bs;
    if (!code_map(&mk, c.K, rows, s.d, a.rows) || !code_map(&mv, c.V, rows, s.d, a.rows))
        return cudaErrorInvalidValue;
    const int grid = min(sms, kMaxGrid);
    const int key = (s.d == 128 ? 4 : 0) | (s.code == SA_E4M3 ? 2 : 0) | (head_tiles(s, chunk) == 2 ? 1 : 0);
    switch (key) {
        case 0: return run<64, SA_INT8, 1>(a, grid, mk, mv, st);
        case 1: return run<64, SA_INT8, 2>(a, grid, mk, mv, st);
        case 2: return run<64, SA_E4M3, 1>(a, grid, mk, mv, st);
        case 3: return run<64, SA_E4M3, 2>(a, grid, mk, mv, st);
        case 4: return run<128, SA_INT8, 1>(a, grid, mk, mv, st);
        case 5: return run<128, SA_INT8, 2>(a, grid, mk, mv, st);
        case 6: return run<128, SA_E4M3, 1>(a, grid, mk, mv, st);
        default: return run<128, SA_E4M3, 2>(a, grid, mk, mv, st);
    }
}

}  // namespace sa
