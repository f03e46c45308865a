// Tokens sampled from logits (er_sample): temperature, top-k, top-p, min-p and a given random number.
//
// Mathematics.  Over a row's logits x with largest M: mass w_i = exp((x_i - M) / T).  In the order of falling logit, ties by
// index, kept are the first top_k; of those the ones before which the masses' sum is below top_p times their sum; of those the
// ones with w >= min_p.  With W the kept masses' sum, the token is the first in the vocabulary's order at which their running
// sum passes u W.
//
// Masses are whole numbers of 2^-44, each within 5 of its 64-bit value (sm_mass), so that sums are exact in any order:
// the kernel's choice next to a border is that of the definition in 64 bits but where a border lies within some 2^-40 of the sum.
//
// Work.  A cluster of CTAs takes a row and keeps it in shared memory; a thread's elements follow one another, so that running
// sums of threads are running sums of the vocabulary.  After the row's largest value:
//   nothing but a temperature or min-p   masses' sums of every thread, then the thread and the element that u W falls to
//   few elements can be kept             these (at least as large as a bound, below) go to the first CTA, which sorts them
//   else                                 counts and masses of 1024 ranges of the logit; the range with the border is looked
//                                        into: its elements are sorted if they are few, split into 1024 ranges again if not
// Bounds for what can be kept: mass 2^-45 (less counts as none); top-k: a value that at least top_k groups of elements reach;
// top-p alone: mass (1 - p) / V, as what lies below sums to at most 1 - p; min-p's mass.
//
// What bounds it.  Rows are read once (512 x 128256 fp32: 263 MB, 39 us at a copy's rate).  Few rows: the cluster's meetings and the
// first CTA's steps one after another: a row of 128256 with top-k and top-p 13 us, 16 rows with other parameters each 51 us (the
// slowest, a flat row with top-p, takes the ranges twice), issue 20 %.  Many rows: 512 with top-k and top-p 238 us; two CTAs an
// SM, each a row's eighth, wait for one another (issue 28 %, barriers first among the stalls).  Temperature alone: masses, some 95
// instructions each for what is within 2^-24 of the largest (128 x 128256 91 us, issue 62 %); half of them were the terms of a
// longer series before the table of 256.
#include <cooperative_groups.h>

#include "pages.cuh"
#include "requests.h"
#include "sample_table.cuh"

namespace er {
namespace cg = cooperative_groups;

constexpr int SM_THREADS = 512, SM_WARPS = 16;
constexpr int SM_LIST = 2048;   // elements that the first CTA sorts
constexpr int SM_BINS = 1024;
constexpr int SM_FEW = 128;     // kept elements that are put in order by counting
constexpr int SM_MAX_CTAS = 8;
constexpr int SM_Q = 44;        // masses are whole numbers of 2^-SM_Q
constexpr unsigned long long SM_ONE = 1ull << SM_Q;
constexpr float SM_LOG2E_HI = 1.44269502162933349609375f, SM_LOG2E_LO = 1.92596299e-8f;
constexpr float SM_LN2_HI = 0.693147182464599609375f, SM_LN2_LO = -1.904654299e-9f;

struct SampleArgs {
    int rows, V, E;  // E: elements of a thread, odd (neighbouring threads' elements then lie in different banks)
    const void *logits;
    long long stride;
    const float *temperature, *top_p, *min_p, *uniform;
    const int32_t *top_k;
    const int64_t *top_k64;  // (in its place)
    int32_t *tokens;
    float *logprobs;
};

// a row's masses: M, 1 / (T ln 2) as two floats
struct SmScale {
    float M, ch, cl;
};
ER_DEV SmScale sm_scale(float T) {
    SmScale s;
    s.M = 0.f;
    const float q = 1.f / T;
    float q2 = q * fmaf(-q, T, 1.f);
    if (!isfinite(q2)) q2 = 0.f;  // T is infinite, or so small that only M has a mass
    s.ch = q * SM_LOG2E_HI;
    s.cl = fmaf(q, SM_LOG2E_HI, -s.ch) + fmaf(q, SM_LOG2E_LO, q2 * SM_LOG2E_HI);
    if (!isfinite(s.cl)) s.cl = 0.f;
    return s;
}
// At temperatures above SM_WIDE logits further apart than float32's largest number have a mass.  A row and its temperature then count
// times 2^-40: differences are numbers, and so is the temperature's reciprocal.  (Only logits below 2^-86 lose bits by it.)
constexpr float SM_WIDE = 1e30f, SM_WIDE_BY = 0x1p-40f;

// M - x for finite M, at most float32's largest number (where it is cut off, the mass is none)
ER_DEV float sm_dist(float x, float M) { return fminf(M - x, 3.402823466e38f); }

// (M - x) / (T ln 2) as two floats: the exact difference (Knuth's sum) times 1 / (T ln 2)
ER_DEV void sm_octaves(float x, const SmScale &s, float &th, float &tl) {
    const float d = sm_dist(x, s.M);
    const float bb = d - s.M;
    const float dl = (s.M - (d - bb)) - (x + bb);
    th = d * s.ch;
    tl = fmaf(d, s.ch, -th) + fmaf(d, s.cl, dl * s.ch);
}

// x's mass in units of 2^-44: 2^-t, t = n + i / 256 + r, |r| <= 1 / 512: 2^-n times the table's entry times e^y, y = -r ln 2,
//   e^y - 1 = y + y^2 (1 / 2 + y / 6 + y^2 / 24)   (the next term is below 2^-54), y as two floats.
// Masses below 2^-24 need no more than 21 bits: one ex2.  (-infinity: th is infinite or, at an infinite T, 0: the caller's.)
ER_DEV unsigned long long sm_mass(float x, const SmScale &s, const float2 *table) {
    float th, tl;
    sm_octaves(x, s, th, tl);
    if (!(th < SM_Q + 2.f)) return 0;
    if (th > 24.f) return (unsigned long long)__float2uint_rn(pg_ex2(SM_Q - th - tl));
    const float k = fmaf(th, 256.f, 12582912.f);  // 1.5 2^23: the nearest whole number of 256 th in its low bits
    const uint32_t ki = __float_as_uint(k);
    const float r = fmaf(k - 12582912.f, -1.f / 256.f, th);  // exact
    const float2 T = table[ki & 255];
    const float y0 = -r * SM_LN2_HI, y1 = fmaf(-r, SM_LN2_HI, -y0) - fmaf(r, SM_LN2_LO, tl * SM_LN2_HI);
    const float yh = y0 + y1, yl = y1 - (yh - y0);
    const float low = fmaf(yh * yh, fmaf(yh, fmaf(yh, 1.f / 24.f, 1.f / 6.f), 0.5f), yl);
    // (1 + yh + low) * (T.x + T.y) = h + l, h = T.x + T.x yh rounded
    const float m = T.x * yh, h = T.x + m;
    const float l = ((T.x - h) + m) + (fmaf(T.x, yh, -m) + fmaf(T.y, yh, fmaf(T.x, low, T.y)));
    const float unit = __uint_as_float((uint32_t)(127 + SM_Q) * 0x800000u - ((ki << 15) & 0x1F800000u));  // 2^(44 - n)
    return (unsigned long long)(__float2ll_rn(h * unit) + (long long)__float2int_rn(l * unit));
}

// floor (UP: ceiling) of f w for 0 <= f <= 1, w < 2^63
template <bool UP>
ER_DEV unsigned long long sm_times(float f, unsigned long long w) {
    const uint32_t b = __float_as_uint(f);
    int s = 150 - (int)(b >> 23);  // f = m 2^-s
    unsigned long long m = b & 0x7FFFFFu;
    if (b >> 23) m |= 0x800000u;
    else s = 149;
    const unsigned long long hi = __umul64hi(m, w), lo = m * w;
    unsigned long long v, cut;  // (s is 23 at least)
    if (s >= 128) v = 0, cut = hi | lo;
    else if (s >= 64) v = hi >> (s - 64), cut = lo | (s == 64 ? 0 : hi << (128 - s));
    else v = (hi << (64 - s)) | (lo >> s), cut = lo << (64 - s);
    return v + (UP && cut ? 1 : 0);
}

struct alignas(16) SmShared {
    // what the cluster's CTAs read of one another, a field a phase
    unsigned long long top;   // the largest element: (order key, ~index)
    uint32_t group;           // an order key that the largest elements of q groups reach
    float least;              // the least candidate
    unsigned long long sum;   // masses' sum
    unsigned long long pad;   // (where the fields behind it lie decides spills: 16 bytes with it, 48 without, 128 x 128256 91 and 99 us)
    unsigned listed;          // elements for `list`
    uint32_t kmin, kmax;      // of a range that is split again
    unsigned ties;
    unsigned long long kept;  // kept masses' sum
    // the first CTA's word to all
    struct {
        int bin;
        unsigned count, r, ties;
        uint32_t thr;
        unsigned long long above, sum;
    } word;
    // inside a CTA
    unsigned long long w64[SM_WARPS];
    unsigned w32[SM_WARPS], v32[SM_WARPS];
    float wg[SM_WARPS];
    uint32_t group_top[SM_THREADS];
    unsigned long long pick;  // kept elements' sum and number, a count
    int keeps;
    unsigned fits;
    float2 table[256];
    unsigned bin_n[SM_BINS], bin_lo[SM_BINS], bin_hi[SM_BINS];  // this CTA's
    unsigned all_n[SM_BINS];                                    // the cluster's (first CTA)
    unsigned long long all_m[SM_BINS];
    unsigned long long list[SM_LIST];
};

ER_DEV float sm_value(unsigned long long key) {  // the logit of an element's key
    const uint32_t k = (uint32_t)(key >> 32);
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// inclusive sums over the CTA's threads; *total: of all
template <class T>
ER_DEV T sm_scan(T v, T *part, T *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();
    if (lane == 31) part[warp] = v;
    __syncthreads();
    T before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < SM_WARPS; ++w) {
        const T s = part[w];
        if (w < warp) before += s;
        all += s;
    }
    *total = all;
    return v + before;
}

// Falling order of the list's n keys; whole CTA.  Bitonic: partners 64 and more apart meet in shared memory, nearer ones in a warp's
// registers (64 keys, two a lane): for 1024 keys 10 steps with a barrier each, and 5 passes in registers, instead of 55 steps.
ER_DEV void sm_order(unsigned long long &a, unsigned long long &b, bool falling) {  // a before b
    if ((a < b) == falling) {
        const unsigned long long t = a;
        a = b;
        b = t;
    }
}
ER_DEV void sm_sort(SmShared &S, int n) {
    unsigned long long *const list = S.list;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (n <= SM_THREADS / 2) {
        // few: an element's place is the number of larger ones, counted by a thread or several (no two keys are equal)
        const int parts = n <= SM_THREADS / 8 ? 8 : n <= SM_THREADS / 4 ? 4 : 2;
        const int i = threadIdx.x / parts, part = threadIdx.x % parts;
        __syncthreads();
        const unsigned long long key = i < n ? list[i] : 0;
        int place = 0;
#pragma unroll 4
        for (int j = part; j < n; j += parts) place += list[j] > key;
        for (int o = 1; o < parts; o <<= 1) place += __shfl_xor_sync(0xffffffffu, place, o);
        __syncthreads();
        if (i < n && part == 0) list[place] = key;
        __syncthreads();
        return;
    }
    int size = 64;
    while (size < n) size <<= 1;
    for (int i = n + threadIdx.x; i < size; i += SM_THREADS) list[i] = 0;
    __syncthreads();
    for (int k = 64; k <= size; k <<= 1) {
        for (int j = k >> 1; j >= 64; j >>= 1) {
            for (int i = threadIdx.x; i < size / 2; i += SM_THREADS) {
                const int a = 2 * i - (i & (j - 1)), b = a + j;
                unsigned long long x = list[a], y = list[b];
                sm_order(x, y, (a & k) == 0);
                list[a] = x;
                list[b] = y;
            }
            __syncthreads();
        }
        for (int c = 64 * warp; c < size; c += 64 * SM_WARPS) {
            unsigned long long x = list[c + lane], y = list[c + 32 + lane];
            // runs of kk up to 64 in the first pass, of k in the others
            for (int kk = k == 64 ? 2 : k; kk <= k; kk <<= 1) {
                const bool fx = ((c + lane) & kk) == 0, fy = ((c + 32 + lane) & kk) == 0;
                if (kk >= 64) sm_order(x, y, fx);
                for (int j = kk >= 64 ? 16 : kk >> 1; j; j >>= 1) {
                    const unsigned long long px = __shfl_xor_sync(0xffffffffu, x, j), py = __shfl_xor_sync(0xffffffffu, y, j);
                    const bool first = (lane & j) == 0;
                    x = (first == fx) == (x > px) ? x : px;
                    y = (first == fy) == (y > py) ? y : py;
                }
            }
            list[c + lane] = x;
            list[c + 32 + lane] = y;
        }
        __syncthreads();
    }
}

// The list's n keys without those below the least of 16 groups' q-th largest, 16 q >= kk: at least the kk largest stay, in any
// order; their number.  Warp w's group is every 16th key.
ER_DEV int sm_prune(SmShared &S, int n, int kk) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, q = (kk + SM_WARPS - 1) / SM_WARPS;
    constexpr int PL = SM_LIST / SM_THREADS;
    unsigned long long key[PL];
#pragma unroll
    for (int j = 0; j < PL; ++j) {
        const int i = (32 * j + lane) * SM_WARPS + warp;
        key[j] = i < n ? S.list[i] : 0;
    }
    // the q-th largest order key (or smaller): the largest is taken away q - 1 times
    uint32_t top = 0;
    unsigned long long last = ~0ull;
    for (int t = 0; t < q; ++t) {
        uint32_t best = 0;
#pragma unroll
        for (int j = 0; j < PL; ++j)
            if (key[j] < last) best = max(best, (uint32_t)(key[j] >> 32));
        top = __reduce_max_sync(0xffffffffu, best);
        // of equal ones the largest
        uint32_t low = 0;
#pragma unroll
        for (int j = 0; j < PL; ++j)
            if (key[j] < last && (uint32_t)(key[j] >> 32) == top) low = max(low, (uint32_t)key[j]);
        low = __reduce_max_sync(0xffffffffu, low);
        last = (unsigned long long)top << 32 | low;
    }
    if (lane == 0) S.w32[warp] = top;
    if (threadIdx.x == 0) S.fits = 0;
    __syncthreads();
    uint32_t least = S.w32[0];
#pragma unroll
    for (int w = 1; w < SM_WARPS; ++w) least = min(least, S.w32[w]);
#pragma unroll
    for (int j = 0; j < PL; ++j)
        if (key[j] && (uint32_t)(key[j] >> 32) >= least) S.list[atomicAdd(&S.fits, 1u)] = key[j];
    __syncthreads();
    return (int)S.fits;
}

template <class T>
__global__ void __launch_bounds__(SM_THREADS, 2) sample_kernel(const SampleArgs a) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    SmShared &S = *reinterpret_cast<SmShared *>(smem_raw);
    float *xs = reinterpret_cast<float *>(smem_raw + sizeof(SmShared));
    static_assert(sizeof(SmShared) % 16 == 0, "rows are stored by 16 bytes");
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int row = blockIdx.x / C, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int E = a.E, L = SM_THREADS * E, first = rank * L, n = max(0, min(L, a.V - first));
    auto of = [&](int r) { return cluster.map_shared_rank(&S, r); };

    float temp = a.temperature ? a.temperature[row] : 1.f;
    if (temp > 0.f) temp = fmaxf(temp, 0x1p-120f);  // (1 / (T ln 2) stays a number)
    const bool wide = temp > SM_WIDE;
    if (wide) temp *= SM_WIDE_BY;
    const long long k = a.top_k ? a.top_k[row] : a.top_k64 ? a.top_k64[row] : 0;
    const int kk = k <= 0 || k >= a.V ? a.V : (int)k;
    const float p = a.top_p ? a.top_p[row] : 1.f, mp = a.min_p ? a.min_p[row] : 0.f;
    float u = a.uniform[row];
    u = u > 0.f ? fminf(u, 1.f) : 0.f;

    // ---- the row, its largest element, and a bound for top-k: of the largest elements of every CTA's groups (what 8 or fewer
    // threads load, a power of two) the q-th largest, the least of these over the CTAs: with q = kk / CTAs at least kk elements reach it
    constexpr int PER = 16 / (int)sizeof(T);
    const T *const src = reinterpret_cast<const T *>(a.logits) + (long long)row * a.stride + first;
    const bool vec = ((uintptr_t)src & 15) == 0;  // (CTAs' parts are multiples of 16 bytes apart)
    int size = 8, q = 0;
    bool bounded = false;
    {
        // groups of threads that load anything, of a CTA with m elements
        auto groups = [&](int m, int z) {
            return ((vec ? min(SM_THREADS, max(m / PER, m % PER)) : min(SM_THREADS, m)) + z - 1) / z;
        };
        const int parts = (a.V + L - 1) / L, last = a.V - (parts - 1) * L;  // CTAs with elements; the last one's
        q = (kk + parts - 1) / parts;
        while (size > 1 && groups(last, size) < q) size >>= 1;
        bounded = kk < a.V && groups(last, size) >= q;
    }
    for (int i = tid; i < 256; i += SM_THREADS) S.table[i] = sm_table[i];
    if (tid == 0) S.listed = 0;
    {
        float best = -INFINITY;
        int where = 0;
        bool any = false;
        auto take = [&](float x, int i) {
            x = fmaxf(x, -INFINITY) + 0.f;  // NaN: never chosen; -0 is 0, a tie that goes by index
            if (x > best) best = x, where = i;
            return x;
        };
        int done = 0;
        if (vec) {
            done = n / PER * PER;
#pragma unroll 8
            for (int i = tid; i < n / PER; i += SM_THREADS) {
                const uint4 w = __ldg(reinterpret_cast<const uint4 *>(src) + i);
                const T *v = reinterpret_cast<const T *>(&w);
                __align__(16) float f[PER];
#pragma unroll
                for (int e = 0; e < PER; ++e) f[e] = take(pg_ld<T>(v + e), PER * i + e);
#pragma unroll
                for (int e = 0; e < PER; e += 4)
                    *reinterpret_cast<float4 *>(xs + PER * i + e) = *reinterpret_cast<const float4 *>(f + e);
                any = true;
            }
        }
#pragma unroll 8
        for (int i = done + tid; i < n; i += SM_THREADS) xs[i] = take(pg_ld<T>(src + i), i), any = true;
        unsigned long long key = any ? (unsigned long long)float_order_key(best) << 32 | (0xFFFFFFFFu - (uint32_t)(first + where)) : 0;
        if (bounded) {
            float g = any ? best : -INFINITY;
            for (int o = 1; o < size; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
            if (tid % size == 0) S.group_top[tid / size] = any ? float_order_key(g) : 0;  // (0: a group without elements)
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
        if (lane == 0) S.w64[warp] = key;
        __syncthreads();
        if (tid == 32) {
            for (int w = 0; w < SM_WARPS; ++w) key = max(key, S.w64[w]);
            S.top = key;
        }
        if (bounded && warp == 0) {  // the largest number of 24 bits that q groups reach
            const int count = SM_THREADS / size;
            uint32_t v[SM_THREADS / 32], reached = 0;
#pragma unroll
            for (int i = 0; i < SM_THREADS / 32; ++i) v[i] = 32 * i + lane < count ? S.group_top[32 * i + lane] : 0;
            for (uint32_t bit = 1u << 31; bit >= 1u << 8; bit >>= 1) {
                const uint32_t next = reached | bit;
                int c = 0;
#pragma unroll
                for (int i = 0; i < SM_THREADS / 32; ++i)
                    if (32 * i < count) c += v[i] >= next;
                if (__reduce_add_sync(0xffffffffu, c) >= q) reached = next;
            }
            if (lane == 0) S.group = n > 0 ? reached : 0xFFFFFFFFu;
        }
        __syncthreads();
    }
    const int at = tid * E, mine = max(0, min(E, n - at));  // this thread's elements: xs[at .. at + mine - 1]
    float *const my = xs + at;
    // what does not need the others, while they come
    const bool has_k = kk < a.V, has_p = p < 1.f;
    SmScale sc = sm_scale(temp);
    const unsigned long long least_mass = mp > 0.f ? max(1ull, sm_times<true>(fminf(mp, 1.f), SM_ONE)) : 1;
    float R = 46.f;  // octaves below M that can be kept
    if (has_p && !has_k) R = fminf(R, log2f((float)a.V) - log2f(1.f - p) + 0.01f);
    if (mp > 0.f && !(has_k && has_p)) R = fminf(R, 0.01f - log2f(fminf(mp, 1.f)));
    R *= temp * SM_LN2_HI * 1.0001f;
    cluster.sync();
    unsigned long long top = 0;
    uint32_t group = 0xFFFFFFFFu;
#pragma unroll
    for (int r = 0; r < SM_MAX_CTAS; ++r)
        if (r < C) {
            top = max(top, of(r)->top);
            if (bounded) group = min(group, of(r)->group);
        }
    float M = sm_value(top);
    const bool none = M == -INFINITY, greedy = !(temp > 0.f) || kk == 1 || p <= 0.f;
    if (none || greedy) {
        if (rank == 0 && tid == 0) {
            a.tokens[row] = none ? -1 : (int32_t)(0xFFFFFFFFu - (uint32_t)top);
            if (a.logprobs) a.logprobs[row] = none ? -INFINITY : 0.f;
        }
        cluster.sync();  // (others may still be reading this CTA's fields)
        return;
    }
    if (M == INFINITY) {  // the infinite ones share everything
        __syncthreads();
        for (int i = tid; i < n; i += SM_THREADS) xs[i] = xs[i] == INFINITY ? 0.f : -INFINITY;
        __syncthreads();
        M = 0.f;
        bounded = false;
    } else if (wide) {
        __syncthreads();
        for (int i = tid; i < n; i += SM_THREADS) xs[i] *= SM_WIDE_BY;
        __syncthreads();
        M *= SM_WIDE_BY;
    }
    sc.M = M;
    // (-infinity may be no octave away from M at an infinite temperature)
    auto mass = [&](float x) { return wide && x == -INFINITY ? 0ull : sm_mass(x, sc, S.table); };
    // the answer: element x, index i, of kept masses' sum W (which is at least the largest element's mass, 1)
    auto answer = [&](float x, int i, unsigned long long W) {
        a.tokens[row] = i;
        if (a.logprobs) {
            float th, tl;
            sm_octaves(x, sc, th, tl);
            a.logprobs[row] = -fmaf(th, SM_LN2_HI, fmaf(th, SM_LN2_LO, tl * SM_LN2_HI)) - log1pf((float)(W - SM_ONE) * 0x1p-44f);
        }
    };
    auto target = [&](unsigned long long W) { return min(sm_times<false>(u, W), W - 1); };

    uint32_t thr = 0;  // kept: order keys above, and of those equal to it the first r of `ties`
    unsigned r = 0, ties = 0;
    if (has_k || has_p) {
        // ---- what can be kept is at least X: within R, or the groups' bound
        float X = M - R;
        X = fmaxf(X - (fabsf(X) + fabsf(M)) * 0x1p-22f, -3.402823466e38f);  // (rounding, of M - R's terms too)
        if (has_k && bounded) X = fmaxf(X, sm_value((unsigned long long)group << 32) * (wide ? SM_WIDE_BY : 1.f));
        auto candidate = [&](float x) { return x >= X; };
        // f(element, its place) for all elements of this CTA, in some order
        auto each = [&](auto f) {
            const float4 *v = reinterpret_cast<const float4 *>(xs);
#pragma unroll 4
            for (int i = tid; i < n / 4; i += SM_THREADS) {
                const float4 w = v[i];
                f(w.x, 4 * i);
                f(w.y, 4 * i + 1);
                f(w.z, 4 * i + 2);
                f(w.w, 4 * i + 3);
            }
            for (int i = n / 4 * 4 + tid; i < n; i += SM_THREADS) f(xs[i], i);
        };
        // this CTA's elements with in(x) into its list (as many as fit); their number in S.listed
        auto collect = [&](float x, int i) {
            const unsigned to = atomicAdd(&S.listed, 1u);
            if (to < SM_LIST) S.list[to] = (unsigned long long)float_order_key(x) << 32 | (0xFFFFFFFFu - (uint32_t)(first + i));
        };
        int ends = 0, counts = 0;  // of the CTAs' lists: lane q knows the number of CTA q's elements, and where they end
        auto listed_all = [&]() {
            ends = counts = lane < C ? (int)of(lane)->listed : 0;
#pragma unroll
            for (int o = 1; o < SM_MAX_CTAS; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, ends, o);
                if (lane >= o) ends += u;
            }
            return (unsigned)__shfl_sync(0xffffffffu, ends, SM_MAX_CTAS - 1);
        };
        // all CTAs' lists (listed_all has been called) into the first's; the lists start anew
        auto gather = [&](int total) {
            if (rank == 0)
                for (int i0 = warp * 32; i0 < total; i0 += SM_THREADS) {
                    const int i = i0 + lane;
                    int q = 0;
#pragma unroll
                    for (int w = 0; w < SM_MAX_CTAS - 1; ++w) q += i >= __shfl_sync(0xffffffffu, ends, w);
                    const int start = __shfl_sync(0xffffffffu, ends - counts, q);
                    if (i < total && q) S.list[i] = of(q)->list[i - start];
                }
            cluster.sync();
            if (tid == 0) S.listed = 0;
            __syncthreads();
        };
        {
            const float4 *v = reinterpret_cast<const float4 *>(xs);
#pragma unroll 4
            for (int i = tid; i < n / 4; i += SM_THREADS) {
                const float4 w = v[i];
                if (fmaxf(fmaxf(w.x, w.y), fmaxf(w.z, w.w)) >= X) {
                    const float f[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (candidate(f[e])) collect(f[e], 4 * i + e);
                }
            }
            for (int i = n / 4 * 4 + tid; i < n; i += SM_THREADS)
                if (candidate(xs[i])) collect(xs[i], i);
        }
        cluster.sync();
        const unsigned nc = listed_all();
        // the cluster's sum of v
        auto total_of = [&](unsigned long long v) {
            unsigned long long all = 0;
            sm_scan(v, S.w64, &all);
            if (tid == 0) S.sum = all;
            cluster.sync();
            all = 0;
#pragma unroll
            for (int q = 0; q < SM_MAX_CTAS; ++q)
                if (q < C) all += of(q)->sum;
            return all;
        };
        unsigned long long sum = 0;  // what top-p's share is of
        constexpr int PL = SM_LIST / SM_THREADS;  // list elements of a thread, one after another

        if (nc <= SM_LIST) {
            // ---- few: sorted by the first CTA
            if (!has_k) {
                each([&](float x, int) { sum += mass(x); });
                sum = total_of(sum);
            }
            int m = (int)nc;
            gather(m);
            if (rank) return;
            // top-k of more: what is below the least of the warps' q-th largest, 16 q >= kk, is none of the first kk
            if (has_k && m > 2 * kk + 64) m = sm_prune(S, m, kk);
            sm_sort(S, m);
            unsigned long long ms[PL], total = 0, incl = 0;
#pragma unroll
            for (int j = 0; j < PL; ++j) {
                const int i = PL * tid + j;
                ms[j] = i < m ? mass(sm_value(S.list[i])) : 0;
                incl += ms[j];
            }
            if (tid == 0) S.keeps = SM_LIST, S.pick = ~0ull;
            const unsigned long long before = sm_scan(incl, S.w64, &total) - incl;
            const int nk = min(kk, m);
            if (has_k && has_p) {  // the sum over the first kk
                unsigned long long b = before;
#pragma unroll
                for (int j = 0; j < PL; ++j) {
                    b += ms[j];
                    if (PL * tid + j == nk - 1) S.sum = b;
                }
                __syncthreads();
                sum = S.sum;
            }
            const unsigned long long most = has_p ? sm_times<true>(p, sum) : ~0ull;
            {  // what is kept is the order's beginning: its end tells its number and its sum.  (Masses of logits next to each other may
               // rise by some units, so min-p's may come to an end several times: the first counts, which has the least sum too)
                unsigned long long b = before, next = 0;
                bool kept[PL + 1];
                auto keep = [&](int i, unsigned long long b, unsigned long long m) {
                    return i < nk && (i == 0 || (b < most && m >= least_mass));
                };
                if (PL * tid + PL < nk) next = mass(sm_value(S.list[PL * tid + PL]));
#pragma unroll
                for (int j = 0; j <= PL; ++j) {
                    kept[j] = keep(PL * tid + j, b, j < PL ? ms[j < PL ? j : 0] : next);
                    if (j < PL) b += ms[j];
                }
                b = before;
#pragma unroll
                for (int j = 0; j < PL; ++j) {
                    b += ms[j];
                    if (kept[j] && !kept[j + 1]) atomicMin(&S.keeps, PL * tid + j + 1), atomicMin(&S.pick, b);
                }
            }
            __syncthreads();
            const int keeps = S.keeps;
            const unsigned long long W = S.pick, to = target(W);
            if (keeps <= SM_FEW) {
                // in the vocabulary's order: each counts what comes before it
#pragma unroll
                for (int j = 0; j < PL; ++j)
                    if (PL * tid + j < keeps) S.all_m[PL * tid + j] = ms[j];
                __syncthreads();
                if (tid < keeps) {
                    const unsigned long long key = S.list[tid];
                    unsigned long long b = 0;
#pragma unroll 4
                    for (int i = 0; i < keeps; ++i)
                        if ((uint32_t)S.list[i] > (uint32_t)key) b += S.all_m[i];
                    if (b <= to && to < b + S.all_m[tid]) answer(sm_value(key), (int)(0xFFFFFFFFu - (uint32_t)key), W);
                }
                return;
            }
            // sorted by the vocabulary
#pragma unroll
            for (int j = 0; j < PL; ++j) {
                const int i = PL * tid + j;
                if (i < keeps) S.list[i] = S.list[i] << 32 | S.list[i] >> 32;
            }
            __syncthreads();
            sm_sort(S, keeps);
            incl = 0;
#pragma unroll
            for (int j = 0; j < PL; ++j) {
                const int i = PL * tid + j;
                ms[j] = i < keeps ? mass(sm_value(S.list[i] << 32)) : 0;
                incl += ms[j];
            }
            unsigned long long b = sm_scan(incl, S.w64, &total) - incl;
#pragma unroll
            for (int j = 0; j < PL; ++j) {
                if (b <= to && to < b + ms[j]) {
                    const unsigned long long w = S.list[PL * tid + j];
                    answer(sm_value(w << 32), (int)(0xFFFFFFFFu - (uint32_t)(w >> 32)), W);
                }
                b += ms[j];
            }
            return;
        }
        cluster.sync();  // (all have read it)
        if (tid == 0) S.listed = 0;

        // ---- many: counts and masses of ranges
        float least = INFINITY;  // the least candidate
        each([&](float x, int) {
            if (candidate(x)) least = fminf(least, x);
        });
#pragma unroll
        for (int o = 16; o; o >>= 1) least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
        __syncthreads();
        if (lane == 0) S.wg[warp] = least;
        __syncthreads();
        if (tid == 0) {
            for (int w = 1; w < SM_WARPS; ++w) least = fminf(least, S.wg[w]);
            S.least = least;
        }
        cluster.sync();
        for (int q = 0; q < C; ++q) least = fminf(least, of(q)->least);
        const float range = sm_dist(least, M), per = range > 0.f ? (float)SM_BINS / range : 0.f;
        auto bin_of = [&](float x) { return min(SM_BINS - 1, (int)(sm_dist(x, M) * per)); };
        unsigned long long outside = 0;  // masses without a bin, this thread's
        // sums of every bin into the first CTA's; bin(x) < 0: none (with `rest` its mass counts as outside)
        auto histogram = [&](auto bin, bool rest) {
            outside = 0;
            for (int i = tid; i < SM_BINS; i += SM_THREADS) S.bin_n[i] = S.bin_lo[i] = S.bin_hi[i] = 0;
            __syncthreads();
            each([&](float x, int) {
                const int i = bin(x);
                if (i < 0 && !rest) return;
                const unsigned long long m = mass(x);
                if (i < 0) {
                    outside += m;
                    return;
                }
                atomicAdd(S.bin_n + i, 1u);
                const unsigned lo = (unsigned)m, old = atomicAdd(S.bin_lo + i, lo);
                const unsigned hi = (unsigned)(m >> 32) + (old + lo < old);
                if (hi) atomicAdd(S.bin_hi + i, hi);
            });
            cluster.sync();
            for (int i = tid + rank * (SM_BINS / C); i < (rank + 1) * (SM_BINS / C); i += SM_THREADS) {
                unsigned c = 0;
                unsigned long long m = 0;
                for (int q = 0; q < C; ++q) {
                    const SmShared *o = of(q);
                    c += o->bin_n[i];
                    m += ((unsigned long long)o->bin_hi[i] << 32) + o->bin_lo[i];
                }
                of(0)->all_n[i] = c;
                of(0)->all_m[i] = m;
            }
            cluster.sync();
        };
        bool fresh = false;  // the first CTA has the bins of the whole range
        auto whole = [&]() {
            if (!fresh) histogram([&](float x) { return candidate(x) ? bin_of(x) : -1; }, !has_k);
            fresh = true;
        };
        // Where the order of falling logits comes to `want` elements (by_mass: at least that sum): thr, r, ties; returns the
        // sum up to there.  All CTAs together.
        auto search = [&](bool by_mass, unsigned long long want) -> unsigned long long {
            whole();
            unsigned long long above = 0, sum_above = 0;  // elements and masses before the range that is looked into
            uint32_t lo = 0, hi = 0;                      // its keys, once it has been split
            int bin = -1;
            const SmShared *o = of(0);
            cluster.sync();  // (all have read the last word)
            for (uint32_t kmin = 0, kmax = 0, shift = 0;;) {
                if (rank == 0) {  // the bin with the border
                    const int i = 2 * tid;
                    unsigned all;
                    unsigned long long alls;
                    const unsigned c0 = S.all_n[i], c1 = S.all_n[i + 1];
                    const unsigned long long m0 = S.all_m[i], m1 = S.all_m[i + 1];
                    unsigned long long cb = above + sm_scan(c0 + c1, S.w32, &all) - (c0 + c1);
                    unsigned long long mb = sum_above + sm_scan(m0 + m1, S.w64, &alls) - (m0 + m1);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const unsigned c = j ? c1 : c0;
                        const unsigned long long m = j ? m1 : m0;
                        if (by_mass ? mb < want && want <= mb + m : cb < want && want <= cb + c) {
                            S.word.bin = i + j;
                            S.word.count = c;
                            S.word.above = cb;
                            S.word.sum = mb;
                        }
                        cb += c;
                        mb += m;
                    }
                }
                cluster.sync();
                const unsigned c = o->word.count;
                above = o->word.above;
                sum_above = o->word.sum;
                const bool split = bin >= 0;
                if (!split) {
                    bin = o->word.bin;
                } else {  // keys kmax - (b << shift) and 2^shift - 1 below it, down to kmin
                    hi = kmax - ((uint32_t)o->word.bin << shift);
                    lo = hi - kmin < (1u << shift) ? kmin : hi - (1u << shift) + 1u;
                }
                auto in = [&](float x) {
                    if (!split) return candidate(x) && bin_of(x) == bin;
                    const uint32_t q = float_order_key(x);
                    return q >= lo && q <= hi;
                };
                if (c <= SM_LIST) {
                    each([&](float x, int i) {
                        if (in(x)) collect(x, i);
                    });
                    cluster.sync();
                    const int m = (int)listed_all();
                    gather(m);
                    if (rank == 0) {
                        sm_sort(S, m);
                        unsigned long long ms[PL], incl = 0, total, b;
#pragma unroll
                        for (int j = 0; j < PL; ++j) {
                            const int i = PL * tid + j;
                            ms[j] = i < m ? mass(sm_value(S.list[i])) : 0;
                            incl += ms[j];
                        }
                        b = sum_above + sm_scan(incl, S.w64, &total) - incl;
#pragma unroll
                        for (int j = 0; j < PL; ++j) {
                            const int i = PL * tid + j;
                            if (i < m && (by_mass ? b < want && want <= b + ms[j] : above + i + 1 == want)) {  // the last one kept
                                const uint32_t q = (uint32_t)(S.list[i] >> 32);
                                int f = i, g = i;
                                while (f > 0 && (uint32_t)(S.list[f - 1] >> 32) == q) --f;
                                while (g + 1 < m && (uint32_t)(S.list[g + 1] >> 32) == q) ++g;
                                S.word.thr = q;
                                S.word.r = i - f + 1;
                                S.word.ties = g - f + 1;
                                S.word.sum = b + ms[j];
                            }
                            b += ms[j];
                        }
                    }
                    cluster.sync();
                    thr = o->word.thr;
                    r = o->word.r;
                    ties = o->word.ties;
                    return o->word.sum;
                }
                // too many: the range between its least and its largest key again
                uint32_t a0 = ~0u, a1 = 0;
                each([&](float x, int) {
                    if (!in(x)) return;
                    const uint32_t q = float_order_key(x);
                    a0 = min(a0, q);
                    a1 = max(a1, q);
                });
                a0 = __reduce_min_sync(0xffffffffu, a0);
                a1 = __reduce_max_sync(0xffffffffu, a1);
                if (lane == 0) S.w32[warp] = a0, S.v32[warp] = a1;
                __syncthreads();
                if (tid == 0) {
                    for (int w = 1; w < SM_WARPS; ++w) a0 = min(a0, S.w32[w]), a1 = max(a1, S.v32[w]);
                    S.kmin = a0;
                    S.kmax = a1;
                }
                cluster.sync();
                kmin = ~0u, kmax = 0;
                for (int q = 0; q < C; ++q) kmin = min(kmin, of(q)->kmin), kmax = max(kmax, of(q)->kmax);
                if (kmin == kmax) {  // one value
                    const unsigned long long m = mass(sm_value((unsigned long long)kmin << 32));
                    thr = kmin;
                    ties = c;
                    r = (unsigned)(by_mass ? (want - sum_above + m - 1) / m : want - above);
                    return sum_above + r * m;
                }
                shift = (uint32_t)max(0, 22 - __clz((int)(kmax - kmin)));
                const uint32_t k0 = kmin, k1 = kmax, sh = shift;
                histogram([&](float x) {
                    const uint32_t q = float_order_key(x);
                    return q >= k0 && q <= k1 ? (int)((k1 - q) >> sh) : -1;
                }, false);
                fresh = false;
            }
        };
        // (fewer than kk candidates: their sum, as what is no candidate then has no mass; as many: X may be the groups' bound, and what
        // is below it is left out.  Without top-k all masses' sum.  Candidates' masses are in the bins, the others' outside)
        unsigned long long inside = 0;
        if (has_k && kk <= (int)nc) {
            inside = sum = search(false, kk);
        } else {
            whole();
            unsigned long long in = 0;
            for (int i = tid; i < SM_BINS; i += SM_THREADS) in += ((unsigned long long)S.bin_hi[i] << 32) + S.bin_lo[i];
            inside = total_of(in);
            sum = inside;
            cluster.sync();  // (all have read it)
            if (!has_k) sum += total_of(outside);
        }
        // (what min-p leaves may sum to less than top-p asks for: then top-p drops none of it)
        const unsigned long long most = max(1ull, sm_times<true>(p, sum));
        if (has_p && most <= inside) search(true, most);
    }

    // ---- masses' sums in the vocabulary's order
    const bool partial = r < ties;
    unsigned tie = 0;  // ties before this thread's
    if (partial) {
        unsigned c = 0, all;
        for (int e = 0; e < mine; ++e) c += float_order_key(my[e]) == thr;
        tie = sm_scan(c, S.w32, &all) - c;
        if (tid == 0) S.ties = all;
        cluster.sync();
        for (int q = 0; q < rank; ++q) tie += of(q)->ties;
    }
    unsigned long long incl = 0, W = 0, before = 0;
    {
        unsigned t = tie;
        for (int e = 0; e < mine; ++e) {
            const float x = my[e];
            const uint32_t q = float_order_key(x);
            if (q < thr || (q == thr && partial && t++ >= r)) continue;
            const unsigned long long m = mass(x);
            if (m >= least_mass) incl += m;
        }
    }
    const unsigned long long own = incl;
    incl = sm_scan(incl, S.w64, &W);
    if (tid == 0) S.kept = W;
    cluster.sync();
    W = 0;
    for (int q = 0; q < C; ++q) {
        const unsigned long long v = of(q)->kept;
        if (q < rank) before += v;
        W += v;
    }
    cluster.sync();  // (all have read; nothing of another CTA is needed from here on)
    const unsigned long long to = target(W);
    const bool found = before + incl - own <= to && to < before + incl;
    const unsigned who = __ballot_sync(0xffffffffu, found);
    if (!who) return;
    // the element: the warp takes the found thread's, 32 at a time
    const int from = __ffs(who) - 1;
    unsigned long long b = __shfl_sync(0xffffffffu, before + incl - own, from);
    unsigned t = __shfl_sync(0xffffffffu, tie, from);
    const int a0 = __shfl_sync(0xffffffffu, at, from), count = __shfl_sync(0xffffffffu, mine, from);
    for (int e0 = 0; e0 < count; e0 += 32) {
        const int e = e0 + lane;
        const float x = e < count ? xs[a0 + e] : -INFINITY;
        const uint32_t q = float_order_key(x);
        const unsigned tied = __ballot_sync(0xffffffffu, e < count && q == thr);
        unsigned long long m = e < count ? mass(x) : 0;
        if (q < thr || (q == thr && partial && t + __popc(tied & ((1u << lane) - 1)) >= r) || m < least_mass) m = 0;
        unsigned long long s = m;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const unsigned long long v = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += v;
        }
        if (b + s - m <= to && to < b + s) answer(x, first + a0 + e, W);
        b += __shfl_sync(0xffffffffu, s, 31);
        t += __popc(tied);
    }
}

// A row's CTAs: as many as leave a thread some 16 elements, up to 8.
static int sm_ctas(int V) {
    int c = 1;
    while (c < SM_MAX_CTAS && V > c * SM_THREADS * 16) c *= 2;
    return c;
}
static int sm_elements(int V) {
    const int per = SM_THREADS * sm_ctas(V);
    return ((V + per - 1) / per) | 1;
}
static size_t sm_smem(int E) { return sizeof(SmShared) + (size_t)SM_THREADS * E * sizeof(float); }
static_assert(ER_SAMPLE_MAX_VOCAB / SM_MAX_CTAS * 4 + SM_THREADS * 4 + sizeof(SmShared) <= 232448, "shared memory");

template <class T>
static cudaError_t sm_launch(const SampleArgs &a, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    const int c = sm_ctas(a.V);
    cfg.gridDim = dim3((unsigned)(a.rows * c));
    cfg.blockDim = dim3(SM_THREADS);
    cfg.dynamicSmemBytes = sm_smem(a.E);
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = c;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // (more than 48 KB of shared memory: an attribute of the device's kernel, set on every call as devices may differ, and to the
    // same number by every call: other host threads' vocabularies are larger)
    static const int most = (int)sm_smem(sm_elements(ER_SAMPLE_MAX_VOCAB));
    cudaError_t e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, sample_kernel<T>, a) : e;
}

cudaError_t launch_sample(const er_sample_args &s, cudaStream_t st) {
    SampleArgs a = {};
    a.rows = s.n_rows;
    a.V = s.vocab;
    a.E = sm_elements(s.vocab);
    a.logits = s.logits_dev;
    a.stride = s.stride;
    a.temperature = s.temperature_dev;
    a.top_p = s.top_p_dev;
    a.min_p = s.min_p_dev;
    a.uniform = s.uniform_dev;
    a.top_k = s.top_k_dev;
    a.top_k64 = s.top_k64_dev;
    a.tokens = s.tokens_dev;
    a.logprobs = s.logprobs_dev;
    return s.type == ER_F32 ? sm_launch<float>(a, st) : s.type == ER_F16 ? sm_launch<__half>(a, st) : sm_launch<__nv_bfloat16>(a, st);
}

}  // namespace er
