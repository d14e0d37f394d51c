// paged_cache.cu -- block tables and slot maps, the quantising append and the
// read-back of the paged 8-bit key/value cache.
#include "paged.cuh"

namespace sa {
namespace {

// ---------------------------------------------------------------------------
// Block tables and slot maps
//
// Sequence b grows or shrinks from cur[b] to want[b] tokens.  With nb(x) =
// ceil(x / bs): a shrinking sequence gives back its blocks nb(want) ..
// nb(cur) - 1, pushed in order of (sequence, block) on the free stack; a
// growing one takes nb(want) - nb(cur) pages, popped in the same order.  Pop
// number a is therefore the released page R - 1 - a while a < R, then
// free[n_free - 1 - (a - R)]: a function of the inputs alone, so one launch
// does it all without a word between its CTAs.  Every CTA scans the B
// lengths into shared memory (a few bytes a sequence, from L2) and takes its
// share of the slots and of the new table entries, each found by a binary
// search in the scanned offsets.  Latency bound: 7 us for 256 sequences that
// grow by a token; with many slots a thread has four or five, one after the
// other, each a search and two dependent reads (334K slots 13 us).
// ---------------------------------------------------------------------------
constexpr int kTabThreads = 512;

struct Sum3 {
    long long t;   // new tokens (a call whose sum passes 32 bits is refused)
    int a, r;      // pages wanted, pages released
};
__device__ __forceinline__ Sum3 add3(Sum3 x, Sum3 y) { return {x.t + y.t, x.a + y.a, x.r + y.r}; }

// Last index b in [0, n) with off[b] <= x (off ascending, off[0] = 0).
__device__ __forceinline__ int owner(const int *off, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (off[m] <= x) lo = m;
        else hi = m;
    }
    return lo;
}

__global__ void __launch_bounds__(kTabThreads)
paged_tables_kernel(PagedShape s, const int32_t *__restrict__ cur, const int32_t *__restrict__ want,
                    int32_t *free_pages, const int32_t *__restrict__ n_free_in, int32_t *n_free_out, int32_t *table,
                    int32_t *cu, int64_t *slot, unsigned *status) {
    extern __shared__ int sm_tab[];
    const int B = s.B, bs = s.bs, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int *offT = sm_tab, *offA = offT + B + 1, *offR = offA + B + 1;
    __shared__ Sum3 wsum[kTabThreads / 32];
    __shared__ int bad_s;
    if (tid == 0) bad_s = 0;
    __syncthreads();
    const int per = (B + kTabThreads - 1) / kTabThreads;
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    const int most = s.maxb * bs;
    Sum3 mine{0, 0, 0};
    int bad = 0;
    for (int b = b0; b < b1; ++b) {
        const int c = cur[b], w = want[b];
        if (c < 0 || c > most || w < 0 || w > most) {
            bad = 1;
            continue;
        }
        const int oc = (c + bs - 1) / bs, ow = (w + bs - 1) / bs;
        mine = add3(mine, {max(0, w - c), max(0, ow - oc), max(0, oc - ow)});
    }
    if (bad) bad_s = 1;
    Sum3 inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sum3 y{__shfl_up_sync(~0u, inc.t, o), __shfl_up_sync(~0u, inc.a, o), __shfl_up_sync(~0u, inc.r, o)};
        if (lane >= o) inc = add3(inc, y);
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    Sum3 base{0, 0, 0}, tot{0, 0, 0};
    for (int w = 0; w < kTabThreads / 32; ++w) {
        if (w < warp) base = add3(base, wsum[w]);
        tot = add3(tot, wsum[w]);
    }
    Sum3 at = add3(base, {inc.t - mine.t, inc.a - mine.a, inc.r - mine.r});
    const int nf = n_free_in[0];
    const bool wrong = bad_s || nf < 0 || nf > s.pages;
    const bool out = !wrong && (tot.t > s.tokens || tot.a > (long long)nf + tot.r || nf + (long long)tot.r - tot.a > s.pages);
    const bool refuse = wrong || out;   // nothing changes: no slots, the same free pages
    for (int b = b0; b < b1; ++b) {
        const int c = refuse ? 0 : cur[b], w = refuse ? 0 : want[b];
        const int oc = (c + bs - 1) / bs, ow = (w + bs - 1) / bs;
        offT[b] = refuse ? 0 : (int)at.t;
        offA[b] = refuse ? 0 : at.a;
        offR[b] = refuse ? 0 : at.r;
        at = add3(at, {max(0, w - c), max(0, ow - oc), max(0, oc - ow)});
    }
    const int T = refuse ? 0 : (int)tot.t, A = refuse ? 0 : tot.a, R = refuse ? 0 : tot.r;
    if (tid == 0) {
        offT[B] = T;
        offA[B] = A;
        offR[B] = R;
        if (blockIdx.x == 0) {
            n_free_out[0] = refuse ? nf : nf + R - A;
            if (wrong) set_status(status, kStatusBadIndex);
            if (out) set_status(status, kStatusPool);
        }
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int b = tid; b <= B; b += kTabThreads) cu[b] = offT[b];

    // the i-th page given back, in order of (sequence, block)
    auto released = [&](int i) {
        const int b = owner(offR, B, i);
        return table[(size_t)b * s.maxb + (want[b] + bs - 1) / bs + (i - offR[b])];
    };
    // the page of pop number a (-1, with a status, if the list holds none there)
    auto popped = [&](int a) {
        const int pg = a < R ? released(R - 1 - a) : free_pages[nf - 1 - (a - R)];
        if (pg >= 0 && pg < s.pages) return pg;
        set_status(status, kStatusBadIndex);
        return -1;
    };
    const long long step = (long long)gridDim.x * kTabThreads, first = (long long)blockIdx.x * kTabThreads + tid;
    for (long long i = first; i < A; i += step) {
        const int b = owner(offA, B, (int)i);
        table[(size_t)b * s.maxb + (cur[b] + bs - 1) / bs + ((int)i - offA[b])] = popped((int)i);
    }
    // what stays released goes on the stack (above every entry that is popped)
    for (long long i = first; i < R - A; i += step) {
        const int pg = released((int)i);
        if (pg < 0 || pg >= s.pages) set_status(status, kStatusBadIndex);
        free_pages[nf + i] = pg;
    }
    for (long long i = first; i < s.tokens; i += step) {
        long long out_slot = -1;
        if (i < T) {
            const int b = owner(offT, B, (int)i);
            const int c = cur[b], pos = c + ((int)i - offT[b]), j = pos / bs, oc = (c + bs - 1) / bs;
            int pg;
            if (j < oc) {
                pg = table[(size_t)b * s.maxb + j];
                if (pg < 0 || pg >= s.pages) {
                    set_status(status, kStatusBadIndex);
                    pg = -1;
                }
            } else {
                pg = popped(offA[b] + j - oc);
            }
            if (pg >= 0) out_slot = (long long)pg * bs + pos % bs;
        }
        slot[i] = out_slot;
    }
}

// ---------------------------------------------------------------------------
// Append
// ---------------------------------------------------------------------------

// The smallest power of two s >= 2^-126 with amax <= M s (M = 448 or 127), from
// the bits of the finite amax: amax = 1.f * 2^x fits M 2^e exactly when
// 1.f <= 1.75 (e4m3; 1.984375 for int8) at e = x - 8 (x - 6), else one more.
template <int kCode>
__device__ __forceinline__ float scale_for(float amax) {
    const unsigned u = __float_as_uint(amax);
    const int x = (int)(u >> 23) - 127;
    const unsigned frac = u & 0x7fffffu;
    int e = kCode == SA_E4M3 ? x - 8 + (frac > 0x600000u) : x - 6 + (frac > 0x7e0000u);
    e = max(e, -126);
    return __uint_as_float((unsigned)(e + 127) << 23);
}

constexpr int kAppThreads = 128;
constexpr int kWinMax = 64;        // tokens whose runs one CTA looks for

// Eight elements as they lie in memory.
template <typename T> struct Raw8;
template <> struct Raw8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = *reinterpret_cast<const uint4 *>(p); }
    // eight codes in the same registers
    __device__ __forceinline__ void hold(uint2 c) { a.x = c.x, a.y = c.y; }
    __device__ __forceinline__ uint2 held() const { return make_uint2(a.x, a.y); }
    // bits of the largest magnitude, as fp32 (a NaN's are above infinity's)
    __device__ __forceinline__ unsigned top() const {
        const unsigned m = 0x7fff7fffu;
        const unsigned x = __vmaxu2(__vmaxu2(a.x & m, a.y & m), __vmaxu2(a.z & m, a.w & m));
        return max(x << 16, x & 0xffff0000u);
    }
    __device__ __forceinline__ void get(float *f) const {
        const unsigned w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <> struct Raw8<float> {
    float4 a, b;
    __device__ __forceinline__ void hold(uint2 c) { a.x = __uint_as_float(c.x), a.y = __uint_as_float(c.y); }
    __device__ __forceinline__ uint2 held() const { return make_uint2(__float_as_uint(a.x), __float_as_uint(a.y)); }
    __device__ __forceinline__ void load(const float *p) {
        a = *reinterpret_cast<const float4 *>(p);
        b = *reinterpret_cast<const float4 *>(p + 4);
    }
    __device__ __forceinline__ unsigned top() const {
        float f[8];
        get(f);
        unsigned x = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) x = max(x, __float_as_uint(f[i]) & 0x7fffffffu);
        return x;
    }
    __device__ __forceinline__ void get(float *f) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
};

// Sum of eight columns' codes: as fp32 (e4m3) or as whole numbers (int8).
template <int kCode> struct Sum8;
template <> struct Sum8<SA_E4M3> {
    float v[8];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
    }
    __device__ __forceinline__ void add(uint2 c) {
        float f[8];
        code_values4<SA_E4M3>(c.x, f);
        code_values4<SA_E4M3>(c.y, f + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += f[e];
    }
    __device__ __forceinline__ float get(int e) const { return v[e]; }
};
template <> struct Sum8<SA_INT8> {
    unsigned v[4];
    int n;
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = 0;
        n = 0;
    }
    // bytes 0, 2 and 1, 3 of a word in 16 bits each, 128 too large every time
    // (at most 128 rows of 255)
    __device__ __forceinline__ void add(uint2 c) {
        c.x ^= 0x80808080u;
        c.y ^= 0x80808080u;
        v[0] += c.x & 0x00ff00ffu;
        v[1] += (c.x >> 8) & 0x00ff00ffu;
        v[2] += c.y & 0x00ff00ffu;
        v[3] += (c.y >> 8) & 0x00ff00ffu;
        ++n;
    }
    __device__ __forceinline__ float get(int e) const {
        const unsigned w = v[(e >> 2) * 2 + (e & 1)];
        return (float)((int)(e & 2 ? w >> 16 : w & 0xffffu) - 128 * n);
    }
};

// Eight finite values with |y inv| <= M to codes, inv a power of two.
template <int kCode>
__device__ __forceinline__ uint2 encode8(const float *y, float inv) {
    uint2 c;
    if (kCode == SA_E4M3) {
        c.x = codes_of2<kCode>(y[0] * inv, y[1] * inv) | codes_of2<kCode>(y[2] * inv, y[3] * inv) << 16;
        c.y = codes_of2<kCode>(y[4] * inv, y[5] * inv) | codes_of2<kCode>(y[6] * inv, y[7] * inv) << 16;
    } else {
        // adding 1.5 * 2^23 rounds to a whole number whose low byte is the code
        unsigned b[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = __float_as_uint(fmaf(y[i], inv, 12582912.f));
        c.x = __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
        c.y = __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410);
    }
    return c;
}
// A value rounded to odd: v, rounded towards 0, with its last bit set where
// something is left (`rest`, exact value minus v).  Rounding on to a code's few
// bits is then one rounding of the exact value; from a v rounded to nearest it
// is not, where that lies on the border between two codes.
__device__ __forceinline__ float to_odd(float v, float rest) {
    return __uint_as_float(__float_as_uint(v) | (rest != 0.f ? 1u : 0u));
}
// The same for any values and any scale: NaN becomes 0, what is beyond M (an
// infinity) the largest code.  Out of line, as it is rare and its division
// takes registers from the path that is not.
template <int kCode>
__device__ __noinline__ uint2 encode8_any(const float *y, float scale) {
    constexpr float kMost = kCode == SA_E4M3 ? 448.f : 127.f;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float x = y[2 * i + e], q = __fdiv_rz(x, scale);
            v[e] = isnan(q) ? 0.f : fabsf(q) >= kMost ? copysignf(kMost, q) : to_odd(q, fmaf(-q, scale, x));
        }
        w[i] = codes_of2<kCode>(v[0], v[1]);
    }
    return make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
}
// Codes at a scale of `ratio` times the new one to codes at the new one.
template <int kCode>
__device__ __forceinline__ uint2 recode8(uint2 c, float ratio) {
    if constexpr (kCode == SA_INT8) {
        float y[8];
        code_values4<kCode>(c.x, y);
        code_values4<kCode>(c.y, y + 4);
        return encode8<kCode>(y, ratio);        // multiplies and rounds at once
    } else {
        auto word = [&](uint32_t w) {
            float y[4];
            code_values4<kCode>(w, y);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float p = __fmul_rz(y[e], ratio);
                y[e] = to_odd(p, fmaf(y[e], ratio, -p));
            }
            return codes_of2<kCode>(y[0], y[1]) | codes_of2<kCode>(y[2], y[3]) << 16;
        };
        return make_uint2(word(c.x), word(c.y));
    }
}

// Last index b in [0, n) with off[b] <= x, found by a whole warp, 32 probes a
// round (off ascending, off[0] <= x).
__device__ __forceinline__ int warp_owner(const int *off, int n, int x) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5, i = lo + lane * step;
        const unsigned le = __ballot_sync(~0u, i < hi && off[i] <= x) | 1u;
        lo += (31 - __clz((int)le)) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// A run: consecutive slots of one page.  The CTA of (window, head, keys or
// values) takes the runs that begin in its window.  A run's new rows, and for
// the landmark the codes already in the block, are read into registers once:
// their largest magnitude decides the scale (kept when the rows fit, else the
// power of two that holds them, and the codes already there are rounded anew;
// a power of two divides exactly, so a code is one rounding of the value, and a
// scale of another kind, kept from elsewhere, is divided by so that it stays
// one), then the codes are written and the mean of the block's cached keys
// becomes its landmark.  A prompt's 30.6K tokens of 8 heads, int8:
// 54 us, 29 at the copy rate (two bytes in, one out per value); bound by issue
// slots (73 % used by eight CTAs an SM).
template <typename T, int kCode, int kD, int kRows>
__global__ void __launch_bounds__(kAppThreads, sizeof(T) == 2 ? (kRows == 64 ? 8 : 5) : kRows == 64 ? 4 : 2)
paged_append_kernel(PagedShape s, const T *__restrict__ K, const T *__restrict__ V, long long ts, long long hs,
                    const int64_t *__restrict__ slot, const int32_t *__restrict__ cu,
                    const int32_t *__restrict__ new_len, uint8_t *K8, uint8_t *V8, float *ks, float *vs, T *L,
                    int window, unsigned *status) {
    constexpr int VPR = kD / 8;           // vectors of eight per row
    constexpr int RS = 128 / VPR;         // rows per step of a half
    constexpr int NV = kRows / RS;        // steps per block
    constexpr float kMost = kCode == SA_E4M3 ? 448.f : 127.f;
    constexpr int kSpan = kWinMax + 128;  // tokens looked at: the window and the end of its last run
    __shared__ int sl[kSpan + 1];         // slots from the token before the window on
    __shared__ unsigned brk[kSpan / 32 + 1], lead[kWinMax / 32];
    __shared__ unsigned red[4];
    __shared__ float lsum[4][kD];
    const int t = threadIdx.x, lane = t & 31, w4 = t >> 5;
    const int cv = t % VPR, rs = t / VPR;
    // keys and values of every head of a window are neighbours in the grid:
    // they read the same rows of their tensors
    const bool half = blockIdx.x & 1;
    const int h = (blockIdx.x >> 1) % s.Hkv, bs = s.bs;
    const long long w0 = (long long)((blockIdx.x >> 1) / s.Hkv) * window;
    const int span = (int)min((long long)window + bs, (long long)s.tokens - w0);   // tokens w0 .. w0 + span - 1
    // sl[j + 1] = slot of token w0 + j, -1 when there is none or it is out of range
    for (int j = t; j <= span; j += kAppThreads) {
        const long long i = w0 + j - 1;
        const long long x = i >= 0 ? slot[i] : -1;
        const bool good = x >= 0 && x < (long long)s.pages * bs;
        if (x >= 0 && !good) set_status(status, kStatusBadIndex);
        sl[j] = good ? (int)x : -1;
    }
    __syncthreads();
    for (int j = t; j < kSpan + 32; j += kAppThreads) {
        // bit j of brk: a run ends before token w0 + j
        const bool b = j >= span || sl[j + 1] < 0 || sl[j + 1] != sl[j] + 1 || sl[j] < 0 || sl[j + 1] % bs == 0;
        const unsigned m = __ballot_sync(~0u, b);
        const unsigned f = __ballot_sync(~0u, b && j < min(window, span) && sl[j + 1] >= 0);   // a run begins here
        if (lane == 0) {
            brk[j >> 5] = m;
            if (j < kWinMax) lead[j >> 5] = f;
        }
    }
    __syncthreads();
    const T *src = half ? V : K;
    uint8_t *codes = half ? V8 : K8;
    float *scales = half ? vs : ks;
    const bool mean = !half && L;
    unsigned left = lead[0];
    for (int w = 0;; left &= left - 1) {
        while (!left && ++w < kWinMax / 32) left = lead[w];
        if (!left) break;
        const int j = 32 * w + __ffs(left) - 1, first = sl[j + 1];
        int end = j + 1;                  // next break (a set bit always follows: bits from span on are set)
        while (!((brk[end >> 5] >> (end & 31)) & 1u)) {
            const unsigned rest = brk[end >> 5] >> (end & 31);
            end = rest ? end + __ffs(rest) - 1 : (end | 31) + 1;
        }
        const int n = end - j, page = first / bs, off = first - page * bs;
        const T *x0 = src + (w0 + j - off) * ts + (long long)h * hs + cv * 8;   // row r of the block: x0 + r ts
        uint8_t *blk = codes + ((size_t)page * s.Hkv + h) * bs * kD + cv * 8;
        float *scale_at = scales + (size_t)page * s.Hkv + h;
        const float was = off > 0 ? *scale_at : 0.f;
        // block rows rs, rs + RS, ...: codes already there, or new rows
        Raw8<T> x[NV];
        unsigned top = 0;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int r = rs + RS * k;
            if (r >= off && r < off + n) x[k].load(x0 + r * ts);
            else if (mean && r < off) x[k].hold(*reinterpret_cast<const uint2 *>(blk + (size_t)r * kD));
        }
        // the landmark's place
        int b = 0, pos = -1;
        if (mean) {
            const int i = (int)(w0 + j), last = cu[s.B];
            b = warp_owner(cu, s.B, min(i, last - 1));
            if (i < last) pos = new_len[b] - cu[b + 1] + i;
            if (pos < 0 || pos % bs != off || pos / bs >= s.maxb) {
                if (t == 0) set_status(status, kStatusBadIndex);
                pos = -1;
            }
        }
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int r = rs + RS * k;
            if (r >= off && r < off + n) top = max(top, x[k].top());
        }
        top = __reduce_max_sync(~0u, top);
        if (lane == 0) red[w4] = top;
        __syncthreads();
        top = max(max(red[0], red[1]), max(red[2], red[3]));
        const bool odd = top >= 0x7f800000u;
        if (odd) {
            // not all finite: the largest of those that are
            if (t == 0) set_status(status, kStatusNaN);
            top = 0;
#pragma unroll 1
            for (int r = rs; r < off + n; r += RS) {
                if (r < off) continue;
                Raw8<T> z;
                z.load(x0 + r * ts);
                float f[8];
                z.get(f);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const unsigned u = __float_as_uint(f[e]) & 0x7fffffffu;
                    top = max(top, u < 0x7f800000u ? u : 0u);
                }
            }
            top = __reduce_max_sync(~0u, top);
            __syncthreads();   // red was read by all
            if (lane == 0) red[w4] = top;
            __syncthreads();
            top = max(max(red[0], red[1]), max(red[2], red[3]));
        }
        const float am = __uint_as_float(top);
        const bool usable = was > 0.f && was <= 3.402823466e38f;
        const bool fits = off > 0 && usable && am <= kMost * was;
        const float now = fits ? was : scale_for<kCode>(am);
        Sum8<kCode> sum;
        sum.zero();
        // codes already there: as they are, or rounded anew to the grown scale
        if (!fits) {
            const float ratio = off > 0 && usable ? __fdiv_rn(was, now) : 0.f;
#pragma unroll 1
            for (int r = rs; r < off; r += RS) {
                uint2 *at = reinterpret_cast<uint2 *>(blk + (size_t)r * kD);
                const uint2 c = recode8<kCode>(*at, ratio);
                *at = c;
                if (mean) sum.add(c);
            }
        } else if (mean) {
#pragma unroll
            for (int k = 0; k < NV; ++k)
                if (rs + RS * k < off) sum.add(x[k].held());
        }
        // the new rows: a power of two divides exactly by its reciprocal; a
        // kept scale may be any number
        if (!odd && (__float_as_uint(now) & 0x7fffffu) == 0) {
            const float inv = __fdiv_rn(1.f, now);
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                const int r = rs + RS * k;
                if (r < off || r >= off + n) continue;
                float y[8];
                x[k].get(y);
                const uint2 c = encode8<kCode>(y, inv);
                *reinterpret_cast<uint2 *>(blk + (size_t)r * kD) = c;
                if (mean) sum.add(c);
            }
        } else {
#pragma unroll 1
            for (int r = rs; r < off + n; r += RS) {
                if (r < off) continue;
                Raw8<T> z;
                z.load(x0 + r * ts);
                float y[8];
                z.get(y);
                const uint2 c = encode8_any<kCode>(y, now);
                *reinterpret_cast<uint2 *>(blk + (size_t)r * kD) = c;
                if (mean) sum.add(c);
            }
        }
        if (t == 0) *scale_at = now;
        if (mean) {
            // sums of e4m3 codes are exact in fp32 up to 2^24 steps of 2^-9
            // (one rounding at most in a full block of 128 extreme codes)
            float acc[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = sum.get(e);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
#pragma unroll
                for (int o = VPR; o < 32; o <<= 1) acc[e] += __shfl_xor_sync(~0u, acc[e], o);
            }
            if (lane < VPR) {
#pragma unroll
                for (int e = 0; e < 8; ++e) lsum[w4][cv * 8 + e] = acc[e];
            }
            __syncthreads();
            if (pos >= 0 && t < kD) {
                const float all = (lsum[0][t] + lsum[1][t]) + (lsum[2][t] + lsum[3][t]);
                from_f(L[(((size_t)b * s.Hkv + h) * s.maxb + pos / bs) * kD + t],
                       __fdiv_rn(all * now, (float)(off + n)));
            }
        }
        __syncthreads();
    }
}

// The same for few tokens (a step of single tokens): one warp per (token,
// head, keys or values), the run's first token leading.  Every read of a warp
// that does not need another is sent off at once -- slots, then scale, new
// rows, eight steps of the block's codes and the landmark's place -- and nothing
// is shared between warps.  Bound by that chain of reads (63 old rows are four
// rounds of codes): 256 tokens of 8 heads 11 us where the bytes take 1.6, half
// of a warp's time between two instructions spent on loads.
template <typename T, int kCode, int kD>
__global__ void __launch_bounds__(128)
paged_append_step_kernel(PagedShape s, const T *__restrict__ K, const T *__restrict__ V, long long ts, long long hs,
                         const int64_t *__restrict__ slot, const int32_t *__restrict__ cu,
                         const int32_t *__restrict__ new_len, uint8_t *K8, uint8_t *V8, float *ks, float *vs, T *L,
                         unsigned *status) {
    constexpr int VPR = kD / 8;           // lanes per row, eight columns each
    constexpr int RS = 32 / VPR;          // rows per step
    constexpr int NB = 8;                 // steps in flight
    constexpr float kMost = kCode == SA_E4M3 ? 448.f : 127.f;
    const int lane = threadIdx.x & 31, cv = lane % VPR, rs = lane / VPR;
    const long long unit = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    const bool val = unit & 1;
    const int h = (int)((unit >> 1) % s.Hkv), bs = s.bs;
    const long long i0 = (unit >> 1) / s.Hkv;
    if (i0 >= s.tokens) return;
    const long long most = (long long)s.pages * bs;
    // slots of the tokens before, of and after i0: lane l holds i0 - 1 + l
    auto slot_at = [&](long long i) { return i >= 0 && i < s.tokens ? slot[i] : -1ll; };
    const long long mine = slot_at(i0 - 1 + lane);
    const long long x = __shfl_sync(~0u, mine, 1), before = __shfl_sync(~0u, mine, 0);
    if (x < 0) return;
    if (x >= most) {
        if (lane == 0) set_status(status, kStatusBadIndex);
        return;
    }
    const int first = (int)x, page = first / bs, off = first - page * bs;
    if (off > 0 && before >= 0 && before + 1 == x) return;      // inside a run
    // rows of the run: slots go on by one within the page
    int n = 0;
    for (int base = 0;; base += 30) {
        const long long v = base == 0 ? mine : slot_at(i0 - 1 + base + lane);
        const bool on = lane > 0 && v == x + base + lane - 1 && off + base + lane - 1 < bs;
        const unsigned stop = ~__ballot_sync(~0u, on) & 0xfffffffeu;
        n = base + (stop ? __ffs((int)stop) - 2 : 31);
        if (stop || base + 30 >= bs) break;
    }
    n = min(n, bs - off);
    const T *src = (val ? V : K) + (i0 - off) * ts + (long long)h * hs + cv * 8;      // row r of the block: src + r ts
    uint8_t *blk = (val ? V8 : K8) + ((size_t)page * s.Hkv + h) * bs * kD + cv * 8;
    float *scale_at = (val ? vs : ks) + (size_t)page * s.Hkv + h;
    const float was = off > 0 ? *scale_at : 0.f;
    const bool mean = !val && L;
    unsigned top = 0;
    Raw8<T> x0;                            // the run's first rows, kept
    const bool has0 = rs < n;
    if (has0) x0.load(src + (off + rs) * ts);
    uint2 old[NB];
    if (mean) {
#pragma unroll
        for (int k = 0; k < NB; ++k)
            if (rs + RS * k < off) old[k] = *reinterpret_cast<const uint2 *>(blk + (size_t)(rs + RS * k) * kD);
    }
    int b = 0, pos = -1;
    if (mean) {
        const int i = (int)i0, last = cu[s.B];
        b = warp_owner(cu, s.B, min(i, last - 1));
        if (i < last) pos = new_len[b] - cu[b + 1] + i;
        if (pos < 0 || pos % bs != off || pos / bs >= s.maxb) {
            if (lane == 0) set_status(status, kStatusBadIndex);
            pos = -1;
        }
    }
    if (has0) top = x0.top();
#pragma unroll 4
    for (int r = rs + RS; r < n; r += RS) {
        Raw8<T> z;
        z.load(src + (off + r) * ts);
        top = max(top, z.top());
    }
    top = __reduce_max_sync(~0u, top);
    const bool odd = top >= 0x7f800000u;
    if (odd) {
        // not all finite: the largest of those that are
        if (lane == 0) set_status(status, kStatusNaN);
        top = 0;
        for (int r = rs; r < n; r += RS) {
            Raw8<T> z;
            z.load(src + (off + r) * ts);
            float f[8];
            z.get(f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const unsigned u = __float_as_uint(f[e]) & 0x7fffffffu;
                top = max(top, u < 0x7f800000u ? u : 0u);
            }
        }
        top = __reduce_max_sync(~0u, top);
    }
    const float am = __uint_as_float(top);
    const bool usable = was > 0.f && was <= 3.402823466e38f;
    const bool fits = off > 0 && usable && am <= kMost * was;
    const float now = fits ? was : scale_for<kCode>(am);
    Sum8<kCode> sum;
    sum.zero();
    if (!fits) {
        const float ratio = off > 0 && usable ? __fdiv_rn(was, now) : 0.f;
#pragma unroll 1
        for (int r = rs; r < off; r += RS) {
            uint2 *at = reinterpret_cast<uint2 *>(blk + (size_t)r * kD);
            const uint2 c = recode8<kCode>(*at, ratio);
            *at = c;
            if (mean) sum.add(c);
        }
    } else if (mean) {
        for (int k0 = 0; k0 * RS < off; k0 += NB) {
            uint2 nx[NB];
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                const int r = rs + RS * (k0 + NB + k);
                if (r < off) nx[k] = *reinterpret_cast<const uint2 *>(blk + (size_t)r * kD);
            }
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                if (rs + RS * (k0 + k) < off) sum.add(old[k]);
                old[k] = nx[k];
            }
        }
    }
    const bool pow2 = !odd && (__float_as_uint(now) & 0x7fffffu) == 0;
    const float inv = __fdiv_rn(1.f, now);
#pragma unroll 4
    for (int r = rs; r < n; r += RS) {
        Raw8<T> z = x0;
        if (r >= RS) z.load(src + (off + r) * ts);
        float y[8];
        z.get(y);
        const uint2 c = pow2 ? encode8<kCode>(y, inv) : encode8_any<kCode>(y, now);
        *reinterpret_cast<uint2 *>(blk + (size_t)(off + r) * kD) = c;
        if (mean) sum.add(c);
    }
    if (lane == 0) *scale_at = now;
    if (mean) {
        float acc[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            acc[e] = sum.get(e);
#pragma unroll
            for (int o = VPR; o < 32; o <<= 1) acc[e] += __shfl_xor_sync(~0u, acc[e], o);
            acc[e] = __fdiv_rn(acc[e] * now, (float)(off + n));
        }
        if (pos >= 0 && lane < VPR) {
            T *to = L + (((size_t)b * s.Hkv + h) * s.maxb + pos / bs) * kD + cv * 8;
#pragma unroll
            for (int e = 0; e < 8; e += Vec<T>::n) store16(to + e, acc + e);
        }
    }
}

// ---------------------------------------------------------------------------
// Read-back: row i = the cached keys and values at slot[i] (zeros where the
// slot is negative or out of range).  One thread per 16 codes of K and of V.
// ---------------------------------------------------------------------------
template <typename T, int kCode>
__global__ void __launch_bounds__(256)
paged_gather_kernel(PagedShape s, const int64_t *__restrict__ slot, const uint8_t *__restrict__ K8,
                    const uint8_t *__restrict__ V8, const float *__restrict__ ks, const float *__restrict__ vs, T *K,
                    T *V, long long ts, long long hs, unsigned *status) {
    const int vpr = s.d / 16;
    const long long total = (long long)s.tokens * s.Hkv * vpr;
    for (long long x = (long long)blockIdx.x * 256 + threadIdx.x; x < total; x += (long long)gridDim.x * 256) {
        const int c = (int)(x % vpr);
        const long long y = x / vpr;
        const int h = (int)(y % s.Hkv);
        const long long i = y / s.Hkv;
        const long long sl = slot[i];
        const bool good = sl >= 0 && sl < (long long)s.pages * s.bs;
        if (sl >= 0 && !good) set_status(status, kStatusBadIndex);
        uint4 k = make_uint4(0, 0, 0, 0), v = k;
        float sk = 0.f, sv = 0.f;
        if (good) {
            const int page = (int)(sl / s.bs), off = (int)(sl - (long long)page * s.bs);
            const size_t ph = (size_t)page * s.Hkv + h;
            const size_t at = (ph * s.bs + off) * s.d + c * 16;
            k = *reinterpret_cast<const uint4 *>(K8 + at);
            v = *reinterpret_cast<const uint4 *>(V8 + at);
            sk = ks[ph];
            sv = vs[ph];
        }
        T *ok = K + i * ts + h * hs + c * 16, *ov = V + i * ts + h * hs + c * 16;
        float f[16];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const uint4 u = half ? v : k;
            const float sc = half ? sv : sk;
            code_values4<kCode>(u.x, f);
            code_values4<kCode>(u.y, f + 4);
            code_values4<kCode>(u.z, f + 8);
            code_values4<kCode>(u.w, f + 12);
#pragma unroll
            for (int e = 0; e < 16; ++e) f[e] *= sc;
            T *o = half ? ov : ok;
#pragma unroll
            for (int e = 0; e < 16; e += Vec<T>::n) store16(o + e, f + e);
        }
    }
}

template <typename T, int kCode>
cudaError_t append_t(const PagedShape &s, const void *K, const void *V, long long ts, long long hs,
                     const int64_t *slot, const int32_t *cu, const int32_t *nl, uint8_t *K8, uint8_t *V8, float *ks,
                     float *vs, void *L, unsigned *status, cudaStream_t st) {
    // While a warp per (token, head, keys or values) fits the GPU at once (64
    // an SM), a call is a step of single tokens or as short as one: a warp
    // each takes 256 tokens of 8 heads in 11 us, the windows below in 20.
    if ((long long)s.tokens * s.Hkv * 2 <= 64ll * max(1, sm_count())) {
        auto k = s.d == 128 ? paged_append_step_kernel<T, kCode, 128> : paged_append_step_kernel<T, kCode, 64>;
        k<<<(unsigned)(((long long)s.tokens * s.Hkv * 2 + 3) / 4), 128, 0, st>>>(
            s, (const T *)K, (const T *)V, ts, hs, slot, cu, nl, K8, V8, ks, vs, (T *)L, status);
        note_launch();
        return cudaGetLastError();
    }
    // Windows as long as leaves about a wave of eight CTAs per SM, so that a
    // prompt's tokens, of which one in `block` begins a run, do not cost a CTA
    // each.
    int window = 1;
    while (window < kWinMax && (long long)s.tokens * s.Hkv > (long long)window * 8 * max(1, sm_count())) window <<= 1;
    const unsigned grid = (unsigned)((s.tokens + window - 1) / window * s.Hkv * 2);
    auto k = s.d == 128 ? (s.bs <= 64 ? paged_append_kernel<T, kCode, 128, 64> : paged_append_kernel<T, kCode, 128, 128>)
                        : (s.bs <= 64 ? paged_append_kernel<T, kCode, 64, 64> : paged_append_kernel<T, kCode, 64, 128>);
    k<<<grid, kAppThreads, 0, st>>>(s, (const T *)K, (const T *)V, ts, hs, slot, cu, nl, K8, V8, ks, vs, (T *)L,
                                    window, status);
    note_launch();
    return cudaGetLastError();
}

template <typename T, int kCode>
cudaError_t gather_t(const PagedShape &s, const int64_t *slot, const uint8_t *K8, const uint8_t *V8, const float *ks,
                     const float *vs, void *K, void *V, long long ts, long long hs, unsigned *status,
                     cudaStream_t st) {
    const long long total = (long long)s.tokens * s.Hkv * (s.d / 16);
    const unsigned grid = (unsigned)min((total + 255) / 256, 64ll * max(1, sm_count()));
    paged_gather_kernel<T, kCode><<<grid, 256, 0, st>>>(s, slot, K8, V8, ks, vs, (T *)K, (T *)V, ts, hs, status);
    note_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_paged_tables(const PagedShape &s, const int32_t *cur, const int32_t *want, int32_t *free_pages,
                                const int32_t *n_free, int32_t *n_free_out, int32_t *table, int32_t *cu,
                                int64_t *slot, unsigned *status, cudaStream_t st) {
    const size_t smem = 3 * (size_t)(s.B + 1) * sizeof(int);
    if (smem > 40 * 1024) {
        const cudaError_t e =
            cudaFuncSetAttribute(paged_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    // every CTA repeats the scan, so one per 2,048 slots or sequences is enough
    const long long work = max((long long)s.tokens, (long long)s.B);
    const unsigned grid = (unsigned)max(1ll, min((work + 2047) / 2048, (long long)max(1, sm_count())));
    paged_tables_kernel<<<grid, kTabThreads, smem, st>>>(s, cur, want, free_pages, n_free, n_free_out, table, cu,
                                                         slot, status);
    note_launch();
    return cudaGetLastError();
}

cudaError_t launch_paged_append(const PagedShape &s, const void *K, const void *V, long long ts, long long hs,
                                const int64_t *slot, const int32_t *cu, const int32_t *nl, uint8_t *K8, uint8_t *V8,
                                float *ks, float *vs, void *L, unsigned *status, cudaStream_t st) {
    if (s.tokens == 0) return cudaSuccess;
    auto f = s.dtype == SA_BF16 ? (s.code == SA_E4M3 ? append_t<__nv_bfloat16, SA_E4M3> : append_t<__nv_bfloat16, SA_INT8>)
                                : (s.code == SA_E4M3 ? append_t<float, SA_E4M3> : append_t<float, SA_INT8>);
    return f(s, K, V, ts, hs, slot, cu, nl, K8, V8, ks, vs, L, status, st);
}

cudaError_t launch_paged_gather(const PagedShape &s, const int64_t *slot, const uint8_t *K8, const uint8_t *V8,
                                const float *ks, const float *vs, void *K, void *V, long long ts, long long hs,
                                unsigned *status, cudaStream_t st) {
    if (s.tokens == 0) return cudaSuccess;
    auto f = s.dtype == SA_BF16 ? (s.code == SA_E4M3 ? gather_t<__nv_bfloat16, SA_E4M3> : gather_t<__nv_bfloat16, SA_INT8>)
                                : (s.code == SA_E4M3 ? gather_t<float, SA_E4M3> : gather_t<float, SA_INT8>);
    return f(s, slot, K8, V8, ks, vs, K, V, ts, hs, status, st);
}

}  // namespace sa
