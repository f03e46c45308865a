// The paged 4-bit K/V cache's calls other than attention: block tables and slot
// maps from request lengths, release, rows in (norm, rotation, quantiser) and out.
// Layout and quantiser: pages.cuh.
#include "pages.cuh"
#include "pages.h"

#include <type_traits>

namespace er {

// ---------------------------------------------------------------------------
// block tables and slot maps
// ---------------------------------------------------------------------------
// need_b = ceil((len_b + new_b) / R) - ceil(len_b / R) pages; the first page given to b is number
// P_b = sum_{i<b} need_i, its first token row T_b = sum_{i<b} new_i, both over the admitted prefix.  Every block scans all the
// requests (4 ints each) and writes its share of tables and slots, so one launch does.  A few KB: latency bounds it (two
// dependent global reads, a scan, a search; 16 requests as 512 prompts about 8.5 us).
constexpr int PL_THREADS = 512;

struct PlanShared {
    int tok[ER_PAGES_MAX_SEQS + 1];   // first row of each request
    int page[ER_PAGES_MAX_SEQS + 1];  // first page number given to each
    long long wsum[2][PL_THREADS / 32];
    int last;
};

// exclusive prefix sums of (a, b) over the block's threads; total in ta, tb
ER_DEV void plan_scan(long long &a, long long &b, long long (&ws)[2][PL_THREADS / 32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long ia = a, ib = b;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long xa = __shfl_up_sync(0xffffffffu, ia, o), xb = __shfl_up_sync(0xffffffffu, ib, o);
        if (lane >= o) {
            ia += xa;
            ib += xb;
        }
    }
    if (lane == 31) {
        ws[0][warp] = ia;
        ws[1][warp] = ib;
    }
    __syncthreads();
    long long oa = 0, ob = 0;
    for (int w = 0; w < warp; ++w) {
        oa += ws[0][w];
        ob += ws[1][w];
    }
    a = ia - a + oa;
    b = ib - b + ob;
}

__global__ void __launch_bounds__(PL_THREADS) pages_plan_kernel(PagesView p, er_pages_plan_args a, int *ticket) {
    __shared__ PlanShared s;
    const int tid = threadIdx.x, R = p.page_rows;
    const long long rows_max = pg_max_len(a.table_stride, R);
    const int free_count = min(max(*a.free_count_dev, 0), p.n_pages);
    constexpr int PER = ER_PAGES_MAX_SEQS / PL_THREADS;
    int flag = 0;
    long long nn[PER], nd[PER], st = 0, sp = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = tid * PER + i;
        nn[i] = nd[i] = 0;
        if (b < a.n_seqs) {
            const long long len = a.lens_dev[b], nw = a.new_dev[b];
            if (len < 0 || nw < 0 || len + nw > rows_max) {
                flag |= ER_PAGES_FLAG_RANGE;
            } else {
                nn[i] = nw;
                nd[i] = (len + nw + R - 1) / R - (len + R - 1) / R;
            }
        }
        st += nn[i];
        sp += nd[i];
    }
    plan_scan(st, sp, s.wsum);
    // admitted: the inclusive sums fit.  Sums never fall, so the admitted requests are a prefix and the first
    // row and page of any later one are the prefix's totals.
    int at[PER], ap[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const bool fits = st + nn[i] <= a.max_tokens && sp + nd[i] <= free_count;
        if (!fits && tid * PER + i < a.n_seqs) flag |= ER_PAGES_FLAG_FULL;
        at[i] = fits ? (int)st : -1;
        ap[i] = (int)sp;
        st += nn[i];
        sp += nd[i];
    }
    if (tid == 0) {
        s.tok[a.n_seqs] = 0;
        s.page[a.n_seqs] = 0;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = tid * PER + i;
        if (b < a.n_seqs) {
            s.tok[b] = at[i];
            s.page[b] = ap[i];
            if (at[i] >= 0) {
                atomicMax(&s.tok[a.n_seqs], at[i] + (int)nn[i]);
                atomicMax(&s.page[a.n_seqs], ap[i] + (int)nd[i]);
            }
        }
    }
    __syncthreads();
    const int total = s.tok[a.n_seqs], pages = s.page[a.n_seqs];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = tid * PER + i;
        if (b < a.n_seqs && at[i] < 0) {
            s.tok[b] = total;
            s.page[b] = pages;
        }
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        for (int b = tid; b <= a.n_seqs; b += PL_THREADS) a.q_start_dev[b] = s.tok[b];
        if (flag) atomicOr(p.flags, flag);
    }
    const long long gtid = (long long)blockIdx.x * PL_THREADS + tid, step = (long long)gridDim.x * PL_THREADS;
    // new table entries: page number i of the step is entry ceil(len / R) + i - P_b of its request's table
    for (long long i = gtid; i < pages; i += step) {
        int lo = 0, hi = a.n_seqs - 1;  // the last request whose first page number is <= i
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s.page[mid] <= (int)i) lo = mid;
            else hi = mid - 1;
        }
        const int have = (a.lens_dev[lo] + R - 1) / R;
        a.tables_dev[(size_t)lo * a.table_stride + have + ((int)i - s.page[lo])] = a.free_dev[free_count - 1 - (int)i];
    }
    for (long long r = gtid; r < a.max_tokens; r += step) {
        int pos = 0, slot = -1, seq = -1;
        if (r < total) {
            int lo = 0, hi = a.n_seqs - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s.tok[mid] <= (int)r) lo = mid;
                else hi = mid - 1;
            }
            seq = lo;
            const int len = a.lens_dev[lo];
            pos = len + (int)r - s.tok[lo];
            const int have = (len + R - 1) / R, blk = pos / R;
            // a page of this step comes from the free list, not from the table another block may be writing
            const int page = blk >= have ? a.free_dev[free_count - 1 - (s.page[lo] + blk - have)]
                                         : a.tables_dev[(size_t)lo * a.table_stride + blk];
            if (page >= 0 && page < p.n_pages) slot = page * R + (pos - blk * R);
            else atomicOr(p.flags, ER_PAGES_FLAG_RANGE);
        }
        a.positions_dev[r] = pos;
        a.slots_dev[r] = slot;
        a.seqs_dev[r] = seq;
    }
    // lens_out and free_count_out may be the inputs themselves: the last block to finish writes them
    __syncthreads();
    if (tid == 0) s.last = atom_add_acq_rel_gpu(ticket, 1) == (int)gridDim.x - 1;
    __syncthreads();
    if (s.last) {
        for (int b = tid; b < a.n_seqs; b += PL_THREADS) a.lens_out_dev[b] = a.lens_dev[b] + (s.tok[b + 1] - s.tok[b]);
        if (tid == 0) {
            *a.free_count_out_dev = free_count - pages;
            *ticket = 0;
        }
    }
}

cudaError_t launch_pages_plan(const PagesView &p, const er_pages_plan_args &a, int *ticket, int num_sms,
                              cudaStream_t st) {
    long long blocks = ((long long)a.max_tokens + PL_THREADS - 1) / PL_THREADS;
    if (blocks < 1) blocks = 1;
    if (blocks > num_sms) blocks = num_sms;
    pages_plan_kernel<<<(unsigned)blocks, PL_THREADS, 0, st>>>(p, a, ticket);
    return cudaGetLastError();
}

// One block: pages of the done requests in order of request and block.
__global__ void __launch_bounds__(PL_THREADS) pages_release_kernel(PagesView p, int n_seqs, const int32_t *done,
                                                                   int32_t *lens, int32_t *tables, int table_stride,
                                                                   int32_t *free_list, int32_t *free_count) {
    __shared__ long long ws[2][PL_THREADS / 32];
    __shared__ int first[ER_PAGES_MAX_SEQS];
    __shared__ int cnt[PL_THREADS / 32];
    __shared__ int base;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, R = p.page_rows;
    constexpr int PER = ER_PAGES_MAX_SEQS / PL_THREADS;
    long long np[PER], sum = 0, zero = 0;
    int flag = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = tid * PER + i;
        np[i] = 0;
        if (b < n_seqs && done[b]) {
            const long long len = lens[b];
            np[i] = len < 0 ? 0 : (len + R - 1) / R;
            if (len < 0 || np[i] > table_stride) {
                flag |= ER_PAGES_FLAG_RANGE;
                np[i] = len < 0 ? 0 : table_stride;
            }
        }
        sum += np[i];
    }
    const long long mine = sum;
    plan_scan(sum, zero, ws);
    long long at = sum;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = tid * PER + i;
        if (b < n_seqs) first[b] = (int)min(at, 2147483647ll);
        at += np[i];
    }
    __shared__ int total_s;
    if (tid == PL_THREADS - 1) total_s = (int)min(sum + mine, 2147483647ll);
    if (tid == 0) base = min(max(*free_count, 0), p.n_pages);
    __syncthreads();
    const int total = total_s;
    // chunks of PL_THREADS entries in order; bad entries leave no gap
    for (int c = 0; c < total; c += PL_THREADS) {
        const int i = c + tid;
        int page = -1;
        if (i < total) {
            int lo = 0, hi = n_seqs - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (first[mid] <= i) lo = mid;
                else hi = mid - 1;
            }
            int32_t *e = tables + (size_t)lo * table_stride + (i - first[lo]);
            page = *e;
            *e = -1;
            if (page < 0 || page >= p.n_pages) {
                page = -1;
                flag |= ER_PAGES_FLAG_RANGE;
            }
        }
        const unsigned m = __ballot_sync(0xffffffffu, page >= 0);
        if (lane == 0) cnt[warp] = __popc(m);
        __syncthreads();
        int before = base + __popc(m & ((1u << lane) - 1u));
        for (int w = 0; w < warp; ++w) before += cnt[w];
        if (page >= 0) {
            if (before < p.n_pages) free_list[before] = page;
            else flag |= ER_PAGES_FLAG_RANGE;
        }
        __syncthreads();
        if (tid == 0) {
            int all = 0;
            for (int w = 0; w < PL_THREADS / 32; ++w) all += cnt[w];
            base = min(base + all, p.n_pages);
        }
        __syncthreads();
    }
    for (int b = tid; b < n_seqs; b += PL_THREADS)
        if (done[b]) lens[b] = 0;
    if (tid == 0) *free_count = base;
    if (flag) atomicOr(p.flags, flag);
}

cudaError_t launch_pages_release(const PagesView &p, int n_seqs, const int32_t *done, int32_t *lens, int32_t *tables,
                                 int table_stride, int32_t *free_list, int32_t *free_count, cudaStream_t st) {
    pages_release_kernel<<<1, PL_THREADS, 0, st>>>(p, n_seqs, done, lens, tables, table_stride, free_list, free_count);
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// rotation table
// ---------------------------------------------------------------------------
__global__ void rope_table_kernel(int hd, double base, int n, float *out) {
    const long long total = (long long)n * (hd / 2);
    for (long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x; i < total;
         i += (long long)gridDim.x * blockDim.x) {
        const long long pos = i / (hd / 2);
        const double th = (double)pos * pow(base, -2.0 * (double)(i % (hd / 2)) / hd);
        double sn, cs;
        sincos(th, &sn, &cs);
        out[2 * i] = (float)cs;
        out[2 * i + 1] = (float)sn;
    }
}

cudaError_t launch_rope_table(int hd, double base, int n, float *out, cudaStream_t st) {
    long long blocks = ((long long)n * (hd / 2) + 255) / 256;
    if (blocks > 8192) blocks = 8192;
    if (blocks < 1) return cudaSuccess;
    rope_table_kernel<<<(unsigned)blocks, 256, 0, st>>>(hd, base, n, out);
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// append and read.  A row is worked by a group of HD / 8 lanes, 8 values a lane: lane c holds the dims 8 c .. + 7 or,
// for the "halves" rotation, 4 c .. + 3 of each half of the head, so that a pair is in one lane.
//
// What bounds append: the bytes of the rows (a token's queries are read and written once, keys and values read
// once and leave in 18 / 32 byte a value).  Queries and keys: a group keeps its token's gain times (cos, sin) in
// registers over several heads, four heads' loads in flight; a key row is quantised from float32 steps, and again from
// float64 ones where those leave a code in doubt (about one warp in a hundred).  Values: a warp takes a run of tokens whose
// slots follow one another inside a tile, so that a prompt's tiles leave as whole 16-byte words although a V word
// mixes four rows; a lone row leaves as bytes.
// ---------------------------------------------------------------------------
// append + read of 8192 bf16 tokens, 32 query and 8 K/V heads of 128: 72 us (33.6 for the bytes alone at the copy rate).
// What costs is instructions and latency, so warps count before registers: blocks of 8 warps 2 an SM 139 us, 3 104, 4 97;
// then with the factors joined, 16-bit values kept as words and the unsure rows done after the others (few spills) 73,
// and 71 in blocks of 4 warps.
constexpr int AP_WARPS = 4;
constexpr int AP_BLOCKS = 8;  // an SM

// N consecutive values as they are, in 32-bit words (kept as words: 16-bit values alone would take a register each)
template <class T, int N>
ER_DEV void ld_raw(const T *p, bool vec, uint32_t *w) {
    constexpr int W = N * sizeof(T) / 4;
    if (!vec) {
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int e = 0; e < N; ++e) w[e] = reinterpret_cast<const uint32_t *>(p)[e];
        } else {
#pragma unroll
            for (int e = 0; e < W; ++e)
                w[e] = (uint32_t) reinterpret_cast<const unsigned short *>(p)[2 * e] |
                       (uint32_t) reinterpret_cast<const unsigned short *>(p)[2 * e + 1] << 16;
        }
    } else if constexpr (W % 4 == 0) {
#pragma unroll
        for (int k = 0; k < W / 4; ++k) {
            const uint4 x = reinterpret_cast<const uint4 *>(p)[k];
            w[4 * k] = x.x, w[4 * k + 1] = x.y, w[4 * k + 2] = x.z, w[4 * k + 3] = x.w;
        }
    } else {
        const uint2 x = *reinterpret_cast<const uint2 *>(p);
        w[0] = x.x, w[1] = x.y;
    }
}
// those words' 8 values
template <class T>
ER_DEV void raw_f32(const uint32_t (&w)[2 * sizeof(T)], float (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        if constexpr (std::is_same<T, float>::value) {
            x[e] = __uint_as_float(w[e]);
        } else if constexpr (std::is_same<T, __half>::value) {
            x[e] = __half2float(__ushort_as_half((unsigned short)(w[e >> 1] >> (16 * (e & 1)))));
        } else {
            x[e] = __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
        }
    }
}
template <class T>
ER_DEV void st8(T *p, bool vec, const float (&x)[8]) {
    __align__(16) T v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = pg_cvt<T>(x[e]);
    if (vec) {
#pragma unroll
        for (int k = 0; k < (int)(8 * sizeof(T)) / 16; ++k) reinterpret_cast<uint4 *>(p)[k] = reinterpret_cast<uint4 *>(v)[k];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = v[e];
    }
}
// 4 consecutive values (8 or 16 bytes)
template <class T>
ER_DEV void st4(T *p, bool vec, const float *x) {
    __align__(16) T v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = pg_cvt<T>(x[e]);
    if (vec) {
        if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<uint4 *>(v);
        else *reinterpret_cast<uint2 *>(p) = *reinterpret_cast<uint2 *>(v);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = v[e];
    }
}
// a row in lane c's order (see above)
template <class T, int HD, bool HALVES>
ER_DEV void ld_row(const T *row, int c, bool vec, uint32_t (&v)[2 * sizeof(T)]) {
    if constexpr (HALVES) {
        ld_raw<T, 4>(row + 4 * c, vec, v);
        ld_raw<T, 4>(row + HD / 2 + 4 * c, vec, v + sizeof(T));
    } else {
        ld_raw<T, 8>(row + 8 * c, vec, v);
    }
}
template <class T, int HD, bool HALVES>
ER_DEV void st_row(T *row, int c, bool vec, const float (&x)[8]) {
    if constexpr (HALVES) {
        st4<T>(row + 4 * c, vec, x);
        st4<T>(row + HD / 2 + 4 * c, vec, x + 4);
    } else {
        st8<T>(row + 8 * c, vec, x);
    }
}

// Codes of a row's blocks, 4 bits each in lane order (value e at bits 4 e), and their scales: d[s] of block
// s of the lane (HALVES: one in each half of the head, else d[0]).  The lanes of a block are neighbours; whole warps call
// this.  A quotient comes from the scale's reciprocal where that leaves no doubt about its code, else from the division.
//
// CHECK: y is off the exact row by at most E = 2 AP_ERR max |m| over the blocks that hold the lane's pairs (that block and,
// for halves, its counterpart in the other half, which the same lanes hold).  Returns whether some code or scale is
// not certain within E.
// In steps of u = 2^-24, relative to |a c| + |b s| of a pair (a, b) times its gains: the sum of HD squares takes 8 fused steps
// and 3 or 4 additions, eps 1 more, together 13, of which the root keeps 6.5; the reciprocal root 4 (2 ulp); gain times
// cosine 1, the rotation 2, the last product 1: 14.5.  (c, s) turn and scale the pair, so |a c| + |b s| is at most sqrt(2) times
// the larger of the two results: 20.5.  The exact value's own rounding to float32 and that of |m| +- E below: 22.5.  E counts
// 2 * 14 = 28.
constexpr float AP_ERR = 14.f * 5.9604645e-8f;
// A mean square (and eps) between these is as exact as that counts: no square that matters has underflowed or overflowed.
constexpr float AP_SMALL = 0x1p-90f, AP_LARGE = 0x1p120f;

template <bool HALVES, bool CHECK>
ER_DEV bool ap_quant(const float (&y)[8], uint32_t &codes, float (&d)[2], int lane) {
    constexpr int S = HALVES ? 2 : 1, EP = 8 / S, LANES = 32 / EP;  // a block: EP values of LANES lanes
    float mx[S], mn[S], m[S];
    bool odd = false;  // NaN, or (exact rows) two values of the largest size and different signs
#pragma unroll
    for (int s = 0; s < S; ++s) {
        mx[s] = mn[s] = y[s * EP];
#pragma unroll
        for (int e = 0; e < EP; ++e) {
            mx[s] = fmaxf(mx[s], y[s * EP + e]);
            mn[s] = fminf(mn[s], y[s * EP + e]);
            odd |= isnan(y[s * EP + e]);
        }
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) {
            mx[s] = fmaxf(mx[s], __shfl_xor_sync(0xffffffffu, mx[s], o));
            mn[s] = fminf(mn[s], __shfl_xor_sync(0xffffffffu, mn[s], o));
        }
        m[s] = mx[s] > -mn[s] ? mx[s] : mn[s];
        if (!CHECK) odd |= mx[s] == -mn[s] && mx[s] != 0.f;
    }
    bool unsure = CHECK && odd;
    if (!CHECK && __any_sync(0xffffffffu, odd)) {
        // the first value of the largest size decides; NaN counts as the largest of all (its bits are above infinity's)
#pragma unroll
        for (int s = 0; s < S; ++s) {
            unsigned big = 0, key = 0xffffu;
#pragma unroll
            for (int e = 0; e < EP; ++e) big = max(big, __float_as_uint(y[s * EP + e]) & 0x7fffffffu);
#pragma unroll
            for (int o = 1; o < LANES; o <<= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
#pragma unroll
            for (int e = EP - 1; e >= 0; --e) {
                const unsigned u = __float_as_uint(y[s * EP + e]);
                if ((u & 0x7fffffffu) == big) key = (unsigned)((EP * (lane & (LANES - 1)) + e) * 2) | (u >> 31);
            }
#pragma unroll
            for (int o = 1; o < LANES; o <<= 1) key = min(key, __shfl_xor_sync(0xffffffffu, key, o));
            m[s] = __uint_as_float(big | (key << 31));
        }
    }
    float E = 0.f;
    if (CHECK) {
#pragma unroll
        for (int s = 0; s < S; ++s) E = fmaxf(E, fabsf(m[s]));
        E *= 2.f * AP_ERR;
    }
    // 1.5 * 2^23 + 8: adding it to a quotient leaves the code in the sum's last bits, rounded to nearest
    constexpr float MAGIC = 12582920.f;
    constexpr uint32_t BITS = 0x4B400000u;  // of 1.5 * 2^23
    codes = 0;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const float dd = pg_scale(m[s]), inv = 1.f / dd;
        d[s] = dd;
        // within this of a border between codes the quotient is in doubt: the reciprocal's and the product's rounding of at most
        // 8.1, and the row's own error
        const float sure = 0.5f - 3e-6f - (CHECK ? E * fabsf(inv) : 0.f);
        if (CHECK) unsure |= pg_scale(fabsf(m[s]) + E) != pg_scale(fabsf(m[s]) - E) || fabsf(mx[s] + mn[s]) <= 2.f * E;
        const bool none = dd == 0.f || isnan(dd);
        float off = 0.f;  // the largest distance of a quotient from its code
        uint32_t acc = 0;
#pragma unroll
        for (int e = 0; e < EP; ++e) {
            const float u = fmaf(y[s * EP + e], inv, MAGIC);
            off = fmaxf(off, fabsf(fmaf(y[s * EP + e], inv, MAGIC - u)));
            acc += (__float_as_uint(fminf(u, MAGIC + 7.f)) - BITS) << (4 * (s * EP + e));
        }
        // (a limited or subnormal scale lets quotients pass 8 (1 + 2^-8); then the fields below would spill over)
        const bool doubt = !none && !(off < sure && fabsf(m[s]) < 21600.f && fabsf(dd) >= 6.2e-5f);
        if (CHECK) {
            unsure |= doubt || none;
        } else if (__any_sync(0xffffffffu, doubt)) {
            if (doubt) {
                acc = 0;
#pragma unroll
                for (int e = 0; e < EP; ++e)
                    acc |= (uint32_t)fminf(fmaxf(roundf(y[s * EP + e] / dd) + 8.f, 0.f), 15.f) << (4 * (s * EP + e));
            }
        }
        codes |= none ? (S == 1 ? 0x88888888u : s ? 0x88880000u : 0x8888u) : acc;
    }
    return unsure;
}

// 8 codes of consecutive dims (dim j at bits 4 j) -> K's word: dim 2 i + e at bits 4 i + 16 e
ER_DEV uint32_t ap_kword(uint32_t c) {
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) w |= ((c >> (4 * j)) & 15u) << (4 * (j >> 1) + 16 * (j & 1));
    return w;
}

struct AppendArgs {
    PagesView p;
    er_pages_append_args a;
    int parts;      // groups that share a token's queries and keys
    int v_blocks;   // blocks that take the values, first because a run takes longest; those after them take the others
    int chunk;      // tokens of a value warp's chunk (1 or 16)
};

// whether token t has a row to write; flags what is out of range
ER_DEV bool ap_there(const AppendArgs &A, int t, int slot, int pos) {
    if (slot < 0) return false;
    if ((long long)slot >= (long long)A.p.n_pages * A.p.page_rows || (A.a.rope_dev && (pos < 0 || pos >= A.a.rope_positions))) {
        atomicOr(A.p.flags, ER_PAGES_FLAG_RANGE);
        return false;
    }
    return true;
}

template <class T, int HD, bool HALVES>
ER_DEV void append_qk(const AppendArgs &A) {
    constexpr int LG = HD / 8, GPW = 32 / LG;  // lanes of a group, groups of a warp
    const er_pages_append_args &a = A.a;
    const PagesView &p = A.p;
    const int lane = threadIdx.x & 31, c = lane % LG;
    const long long grp = ((long long)(blockIdx.x - A.v_blocks) * AP_WARPS + (threadIdx.x >> 5)) * GPW + lane / LG;
    const int t = (int)(grp / A.parts), part = (int)(grp - (long long)t * A.parts);
    const bool in = t < a.n_tokens;
    const int slot = in ? a.slots_dev[t] : -1;
    const int pos = in && a.rope_dev && slot >= 0 ? a.positions_dev[t] : 0;
    const bool there = ap_there(A, t, slot, pos);
    if (!__any_sync(0xffffffffu, there)) return;
    auto aligned = [](const void *x, int64_t stride) { return ((uintptr_t)x & 15) == 0 && (stride * sizeof(T)) % 16 == 0; };
    const bool vq = aligned(a.q_dev, a.q_stride), vk = aligned(a.k_dev, a.k_stride), vo = aligned(a.q_out_dev, a.q_out_stride);
    // The lane's pair i is values (2 i, 2 i + 1), or (i, i + 4) for halves.  Gain, cosine and sine go together once a token:
    //   (a, b) -> rs (a ga c - b gb s, b gb c + a ga s)
    const bool turn = a.rope_dev != nullptr;
    auto dim = [&](int e) { return HALVES ? (e >> 2) * (HD / 2) + 4 * c + (e & 3) : 8 * c + e; };
    auto table = [&](int i) {
        return turn && there ? __ldg(reinterpret_cast<const float2 *>(a.rope_dev) + (size_t)pos * (HD / 2) + 4 * c + i)
                             : make_float2(1.f, 0.f);
    };
    float co[8], si[8];  // ga c, gb c of each pair; ga s, gb s
    auto factors = [&](const float *gain) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = table(i);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int e = HALVES ? i + 4 * k : 2 * i + k;
                const float g = gain ? __ldg(gain + dim(e)) : 1.f;
                co[e] = g * t.x;
                si[e] = g * t.y;
            }
        }
    };
    // returns false where the sum of squares may have left fp32's range on its way
    auto row_of = [&](const float (&x)[8], bool norm, float eps, float (&y)[8]) {
        float rs = 1.f;
        bool in_range = true;
        if (norm) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int o = 1; o < LG; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float ms = ss * (1.f / HD) + eps;
            in_range = ms > AP_SMALL && ms < AP_LARGE;
            rs = rsqrtf(ms);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e0 = HALVES ? i : 2 * i, e1 = HALVES ? i + 4 : 2 * i + 1;
            y[e0] = (x[e0] * co[e0] - x[e1] * si[e1]) * rs;
            y[e1] = (x[e1] * co[e1] + x[e0] * si[e0]) * rs;
        }
        return in_range;
    };
    // Whole warps go round together (its groups' tokens and parts may differ), U rows of a group at a time: their loads are
    // in flight together.  work returns whether the row is to be done again by the exact steps, after the others of its U.
    constexpr int U = sizeof(T) == 2 ? 4 : 2;  // (8 with 3 / 4 of the warps: 78 us for 73; 2: 79 for 75)
    auto rows_of = [&](const T *base, int64_t stride, bool vec, int n, auto work, auto again) {
        const T *src = base + t * stride + (size_t)part * HD;
        for (int r = part; r - part < n; r += U * A.parts) {
            uint32_t v[U][2 * sizeof(T)];
#pragma unroll
            for (int u = 0; u < U; ++u) {
#pragma unroll
                for (int e = 0; e < (int)(2 * sizeof(T)); ++e) v[u][e] = 0;
                if (there && r + u * A.parts < n) ld_row<T, HD, HALVES>(src + (size_t)u * A.parts * HD, c, vec, v[u]);
            }
            unsigned redo = 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (r - part + u * A.parts >= n) break;  // (the same in the whole warp)
                float x[8];
                raw_f32<T>(v[u], x);
                redo |= (work(r + u * A.parts, there && r + u * A.parts < n, x) ? 1u : 0u) << u;
            }
            for (redo = __reduce_or_sync(0xffffffffu, redo); redo; redo &= redo - 1) {
                const int u = __ffs(redo) - 1;
                const bool live = there && r + u * A.parts < n;
                uint32_t w[2 * sizeof(T)] = {};
                if (live) ld_row<T, HD, HALVES>(src + (size_t)u * A.parts * HD, c, vec, w);
                float x[8];
                raw_f32<T>(w, x);
                again(r + u * A.parts, live, x);
            }
            src += (size_t)U * A.parts * HD;
        }
    };
    auto never = [](int, bool, const float (&)[8]) {};
    if (a.n_heads) {
        factors(a.q_gain_dev);
        T *dst = (T *)a.q_out_dev + t * a.q_out_stride;
        auto put = [&](int r, bool live, const float (&y)[8]) {
            if (live) st_row<T, HD, HALVES>(dst + (size_t)r * HD, c, vo, y);
            return false;
        };
        if (a.q_gain_dev && a.eps <= AP_SMALL) {
            // eps keeps no mean square in range: the row and eps times the power of two that brings the larger to [1, 2)
            rows_of((const T *)a.q_dev, a.q_stride, vq, a.n_heads, [&](int r, bool live, const float (&x)[8]) {
                unsigned top = __float_as_uint(sqrtf(a.eps));
#pragma unroll
                for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
#pragma unroll
                for (int o = 1; o < LG; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                const float up = __uint_as_float((254u - min(max(top >> 23, 1u), 253u)) << 23);
                float z[8], y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) z[e] = x[e] * up;
                row_of(z, true, a.eps * up * up, y);
                return put(r, live, y);
            }, never);
        } else {
            rows_of((const T *)a.q_dev, a.q_stride, vq, a.n_heads, [&](int r, bool live, const float (&x)[8]) {
                float y[8];
                row_of(x, a.q_gain_dev != nullptr, a.eps, y);
                return put(r, live, y);
            }, never);
        }
    }
    const bool norm = a.k_gain_dev != nullptr;
    factors(a.k_gain_dev);
    auto store = [&](int r, bool live, uint32_t codes, const float (&d)[2]) {
        const uint32_t mate = __shfl_xor_sync(0xffffffffu, codes, 1);
        if (!live) return;
        uint8_t *tile = pg_tile(p.pool, p.page_rows, p.KV, HD, slot, r);
        const int in16 = (slot % p.page_rows) & 15;
        __half *ks = reinterpret_cast<__half *>(tile + pg_off_ks(HD)) + in16 * (HD / 32);
        if constexpr (HALVES) {
            // two lanes make a word: the even one that of the first half, the odd one that of the second
            const bool odd = c & 1;
            const uint32_t lo = odd ? mate >> 16 : codes & 0xFFFFu, hi = odd ? codes >> 16 : mate & 0xFFFFu;
            const int dim = (odd ? HD / 2 : 0) + 8 * (c >> 1);
            *reinterpret_cast<uint32_t *>(tile + pg_k_word(in16, ((dim & 31) >> 3) * (HD / 32) + (dim >> 5), HD)) =
                ap_kword(lo | hi << 16);
            if ((c & 7) == 0) {
                ks[c >> 3] = __float2half_rn(d[0]);
                ks[HD / 64 + (c >> 3)] = __float2half_rn(d[1]);
            }
        } else {
            *reinterpret_cast<uint32_t *>(tile + pg_k_word(in16, (c & 3) * (HD / 32) + (c >> 2), HD)) = ap_kword(codes);
            if ((c & 3) == 0) ks[c >> 2] = __float2half_rn(d[0]);
        }
    };
    auto exact = [&](int r, bool live, const float (&x)[8]) {
        // in float64: the codes are those of the formula whatever the float32 steps were
        double zs = 0.0, rs = 1.0;
#pragma unroll
        for (int e = 0; e < 8; ++e) zs += (double)x[e] * (double)x[e];
#pragma unroll
        for (int o = 1; o < LG; o <<= 1) zs += __shfl_xor_sync(0xffffffffu, zs, o);
        if (norm) rs = 1.0 / sqrt(zs / HD + (double)a.eps);
        float y[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 cs = table(i);
            const int e0 = HALVES ? i : 2 * i, e1 = HALVES ? i + 4 : 2 * i + 1;
            const double za = (double)x[e0] * rs * (norm ? (double)__ldg(a.k_gain_dev + dim(e0)) : 1.0);
            const double zb = (double)x[e1] * rs * (norm ? (double)__ldg(a.k_gain_dev + dim(e1)) : 1.0);
            y[e0] = (float)(za * (double)cs.x - zb * (double)cs.y);
            y[e1] = (float)(zb * (double)cs.x + za * (double)cs.y);
        }
        uint32_t codes;
        float d[2];
        ap_quant<HALVES, false>(y, codes, d, lane);
        store(r, live, codes, d);
    };
    if (!norm && !turn) {  // keys as they are
        rows_of((const T *)a.k_dev, a.k_stride, vk, p.KV, [&](int r, bool live, const float (&x)[8]) {
            uint32_t codes;
            float d[2];
            ap_quant<HALVES, false>(x, codes, d, lane);
            store(r, live, codes, d);
            return false;
        }, never);
    } else {
        rows_of((const T *)a.k_dev, a.k_stride, vk, p.KV, [&](int r, bool live, const float (&x)[8]) {
            uint32_t codes;
            float d[2], y[8];
            const bool in_range = row_of(x, norm, a.eps, y);
            const bool unsure = ap_quant<HALVES, true>(y, codes, d, lane) || !in_range;
            store(r, live, codes, d);
            return unsure && live;
        }, exact);
    }
}

template <class T, int HD>
ER_DEV void append_v(const AppendArgs &A, uint32_t (&cw)[16][HD / 8 + 2], unsigned short (&sc)[16][HD / 32]) {
    constexpr int LG = HD / 8, GPW = 32 / LG;
    const er_pages_append_args &a = A.a;
    const PagesView &p = A.p;
    const int lane = threadIdx.x & 31, c = lane % LG, gi = lane / LG;
    const long long item = (long long)blockIdx.x * AP_WARPS + (threadIdx.x >> 5);
    const int chunk = (int)(item / p.KV), h = (int)(item - (long long)chunk * p.KV);
    const int t0 = chunk * A.chunk;
    if (t0 >= a.n_tokens) return;
    const bool vec = ((uintptr_t)a.v_dev & 15) == 0 && (a.v_stride * sizeof(T)) % 16 == 0;
    // lane i: token t0 + i; a run starts where a token does not follow the one before it inside a tile
    const int ti = t0 + lane;
    const int slot = ti < a.n_tokens ? a.slots_dev[ti] : -1;
    const int prev = ti < a.n_tokens && ti > 0 ? a.slots_dev[ti - 1] : -2;
    const int pos = ti < a.n_tokens && a.rope_dev && slot >= 0 ? a.positions_dev[ti] : 0;
    const int ppos = ti < a.n_tokens && a.rope_dev && ti > 0 && prev >= 0 ? a.positions_dev[ti - 1] : 0;
    const bool there = ap_there(A, ti, slot, pos);
    auto good = [&](int s, int q) {
        return s >= 0 && (long long)s < (long long)p.n_pages * p.page_rows && (!a.rope_dev || (q >= 0 && q < a.rope_positions));
    };
    const bool starts = there && (slot % 16 == 0 || slot != prev + 1 || !good(prev, ppos));
    const unsigned sm = __ballot_sync(0xffffffffu, starts), tm = __ballot_sync(0xffffffffu, there);
    // the runs that start among the chunk's tokens (one may reach past it, up to 15 tokens on)
    for (unsigned left = sm & ((1u << A.chunk) - 1u); left; left &= left - 1) {
        const int first = __ffs(left) - 1;
        const unsigned stop = (sm | ~tm) & ~((2u << first) - 1u);  // the next start, or the next token without a row
        const int n = min((stop ? __ffs(stop) - 1 : 32) - first, 16);
        const int s0 = __shfl_sync(0xffffffffu, slot, first), r0 = (s0 % p.page_rows) & 15;
        // rows k = gi, gi + GPW, ... of the run: codes and scales to shared memory
        const T *src = (const T *)a.v_dev + (t0 + first) * a.v_stride + (size_t)h * HD + 8 * c;
#pragma unroll 4
        for (int k0 = 0; k0 < n; k0 += GPW) {
            const int k = k0 + gi;
            uint32_t v[2 * sizeof(T)] = {};
            if (k < n) ld_raw<T, 8>(src + k * a.v_stride, vec, v);
            float x[8];
            raw_f32<T>(v, x);
            uint32_t codes;
            float d[2];
            ap_quant<false, false>(x, codes, d, lane);
            if (k < n) {
                cw[r0 + k][c] = codes;
                if ((c & 3) == 0) sc[r0 + k][c >> 2] = __half_as_ushort(__float2half_rn(d[0]));
            }
        }
        __syncwarp();
        uint8_t *tile = pg_tile(p.pool, p.page_rows, p.KV, HD, s0, h);
        // lane (g, t): words u of run q: dims 64 q + 16 u + g and + 8 of rows 2 t, 2 t + 8, 2 t + 1, 2 t + 9
        const int g = lane >> 2, t = lane & 3;
        auto has = [&](int r) { return r >= r0 && r < r0 + n; };
        const bool all = has(2 * t) && has(2 * t + 1) && has(2 * t + 8) && has(2 * t + 9);
#pragma unroll
        for (int q = 0; q < HD / 64; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                w[u] = 0;
#pragma unroll
                for (int b = 0; b < 4; ++b) {  // byte b: row 2 t + (b >> 1) + 8 (b & 1)
                    const uint2 y = *reinterpret_cast<const uint2 *>(&cw[2 * t + (b >> 1) + 8 * (b & 1)][8 * q + 2 * u]);
                    w[u] |= (((y.x >> (4 * g)) & 15u) | ((y.y >> (4 * g)) & 15u) << 4) << (8 * b);
                }
            }
            uint8_t *dst = tile + pg_off_v(HD) + q * 512 + lane * 16;
            if (all) {
                *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    if (has(2 * t + (b >> 1) + 8 * (b & 1)))
#pragma unroll
                        for (int u = 0; u < 4; ++u) dst[4 * u + b] = (uint8_t)(w[u] >> (8 * b));
            }
        }
        unsigned short *vs = reinterpret_cast<unsigned short *>(tile + pg_off_vs(HD));
        for (int k = lane; k < n * (HD / 32); k += 32) {
            const int r = r0 + k / (HD / 32), blk = k % (HD / 32);
            vs[pg_vs_half(r, blk, HD)] = sc[r][blk];
        }
        __syncwarp();
    }
}

template <class T, int HD, bool HALVES>
__global__ void __launch_bounds__(AP_WARPS * 32, AP_BLOCKS) pages_append_kernel(const AppendArgs A) {
    __shared__ __align__(16) uint32_t cw[AP_WARPS][16][HD / 8 + 2];
    __shared__ unsigned short sc[AP_WARPS][16][HD / 32];
    if ((int)blockIdx.x < A.v_blocks) append_v<T, HD>(A, cw[threadIdx.x >> 5], sc[threadIdx.x >> 5]);
    else append_qk<T, HD, HALVES>(A);
}

template <class T>
static cudaError_t append_t(const PagesView &p, const er_pages_append_args &a, int num_sms, cudaStream_t st) {
    AppendArgs A = {p, a, 1, 0, 16};
    const int rows = a.n_heads > p.KV ? a.n_heads : p.KV;
    // Groups (of HD / 8 lanes) enough for the threads that the GPU holds at once, and no more than one a row: a step's few
    // tokens are spread row by row, a prompt's groups keep their token's factors for several heads (8192 tokens: two
    // groups a token 71 us, three 75, five 78, nine 88).
    const long long want = (long long)num_sms * AP_BLOCKS * AP_WARPS * 32 / (p.hd / 8);
    const long long parts = (want + a.n_tokens - 1) / a.n_tokens;
    A.parts = (int)(parts < 1 ? 1 : parts > rows ? rows : parts);
    const long long per = AP_WARPS * 32 / (p.hd / 8);
    const long long qk = ((long long)a.n_tokens * A.parts + per - 1) / per;
    // Chunks of 16 tokens where that still makes a warp for every scheduler, else a token each
    A.chunk = (long long)a.n_tokens * p.KV / 16 >= 4ll * num_sms ? 16 : 1;
    const long long chunks = ((long long)a.n_tokens + A.chunk - 1) / A.chunk;
    const long long v = (chunks * p.KV + AP_WARPS - 1) / AP_WARPS;
    if (qk + v > 2147483647ll) return cudaErrorInvalidValue;
    A.v_blocks = (int)v;
    const unsigned blocks = (unsigned)(qk + v);
    const bool halves = a.rope_style == ER_ROPE_HALVES;
    if (p.hd == 128)
        halves ? pages_append_kernel<T, 128, true><<<blocks, AP_WARPS * 32, 0, st>>>(A)
               : pages_append_kernel<T, 128, false><<<blocks, AP_WARPS * 32, 0, st>>>(A);
    else
        halves ? pages_append_kernel<T, 64, true><<<blocks, AP_WARPS * 32, 0, st>>>(A)
               : pages_append_kernel<T, 64, false><<<blocks, AP_WARPS * 32, 0, st>>>(A);
    return cudaGetLastError();
}

cudaError_t launch_pages_append(const PagesView &p, const er_pages_append_args &a, int num_sms, cudaStream_t st) {
    return a.type == ER_F32   ? append_t<float>(p, a, num_sms, st)
           : a.type == ER_F16 ? append_t<__half>(p, a, num_sms, st)
                              : append_t<__nv_bfloat16>(p, a, num_sms, st);
}

// ---------------------------------------------------------------------------
// rows out: a group of HD / 8 lanes per (slot, head), 8 consecutive dims a lane
// ---------------------------------------------------------------------------
template <class T, int HD>
__global__ void __launch_bounds__(256) pages_read_kernel(PagesView p, int n, const int32_t *slots, T *k, T *v, bool vec) {
    constexpr int LG = HD / 8;
    const int c = threadIdx.x % LG;
    const long long it = (long long)blockIdx.x * (256 / LG) + threadIdx.x / LG;
    if (it >= (long long)n * p.KV) return;
    // heads fastest: neighbouring groups write neighbouring rows
    const int t = (int)(it / p.KV), h = (int)(it - (long long)t * p.KV);
    const int slot = slots[t];
    if (slot < 0) return;
    if ((long long)slot >= (long long)p.n_pages * p.page_rows) {
        if (c == 0) atomicOr(p.flags, ER_PAGES_FLAG_RANGE);
        return;
    }
    const uint8_t *tile = pg_tile(p.pool, p.page_rows, p.KV, HD, slot, h);
    const int r = (slot % p.page_rows) & 15;
    const size_t out = (size_t)it * HD + 8 * c;
    float x[8];
    if (k) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(tile + pg_k_word(r, (c & 3) * (HD / 32) + (c >> 2), HD));
        const float d = __half2float(reinterpret_cast<const __half *>(tile + pg_off_ks(HD))[r * (HD / 32) + (c >> 2)]);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = d * (float)((int)((w >> (4 * (j >> 1) + 16 * (j & 1))) & 15u) - 8);
        st8<T>(k + out, vec, x);
    }
    if (v) {
        // dims 8 c .. + 7: nibbles c & 1 of 8 bytes, 64 apart
        const uint8_t *src = tile + pg_off_v(HD) + pg_v_byte(r, 8 * (c >> 1));
        const float d = __half2float(reinterpret_cast<const __half *>(tile + pg_off_vs(HD))[pg_vs_half(r, c >> 2, HD)]);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = d * (float)((int)((src[64 * j] >> (4 * (c & 1))) & 15) - 8);
        st8<T>(v + out, vec, x);
    }
}

template <class T>
static cudaError_t read_t(const PagesView &p, int n, const int32_t *slots, void *k, void *v, cudaStream_t st) {
    const int per = 256 / (p.hd / 8);
    const long long blocks = ((long long)n * p.KV + per - 1) / per;
    if (blocks < 1) return cudaSuccess;
    if (blocks > 2147483647ll) return cudaErrorInvalidValue;
    const bool vec = (((uintptr_t)k | (uintptr_t)v) & 15) == 0;
    if (p.hd == 128) pages_read_kernel<T, 128><<<(unsigned)blocks, 256, 0, st>>>(p, n, slots, (T *)k, (T *)v, vec);
    else pages_read_kernel<T, 64><<<(unsigned)blocks, 256, 0, st>>>(p, n, slots, (T *)k, (T *)v, vec);
    return cudaGetLastError();
}

cudaError_t launch_pages_read(const PagesView &p, int n, const int32_t *slots, int type, void *k, void *v,
                              cudaStream_t st) {
    return type == ER_F32   ? read_t<float>(p, n, slots, k, v, st)
           : type == ER_F16 ? read_t<__half>(p, n, slots, k, v, st)
                            : read_t<__nv_bfloat16>(p, n, slots, k, v, st);
}

}  // namespace er
