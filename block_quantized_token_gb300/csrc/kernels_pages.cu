// The paged 4-bit K/V cache's calls other than attention: block tables and slot
// maps from request lengths, release, rows in (norm, rotation, quantiser) and out.
// Layout and quantiser: pages.cuh.
#include "pages.cuh"
#include "pages.h"

namespace er {

// ---------------------------------------------------------------------------
// block tables and slot maps
// ---------------------------------------------------------------------------
// need_b = ceil((len_b + new_b) / R) - ceil(len_b / R) pages; the first page given to b is number
// P_b = sum_{i<b} need_i, its first token row T_b = sum_{i<b} new_i, both over the admitted prefix.
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
    const long long rows_max = (long long)a.table_stride * R;
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
// append: one warp per (token, head), heads 0 .. H - 1 queries, then KV keys, then KV values
// ---------------------------------------------------------------------------
constexpr int AP_WARPS = 8;

// max / min over the 32 / W lanes that share a block
template <int LANES>
ER_DEV float group_max(float v) {
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Dims of element e of a lane.  PAIRS: HD / 32 consecutive dims; HALVES: half of them in each half of the head,
// so that a pair is in one lane in both styles.
template <int HD, bool HALVES>
ER_DEV constexpr int ap_dim(int lane, int e) {
    constexpr int E = HD / 32;
    return HALVES ? (e / (E / 2)) * (HD / 2) + (E / 2) * lane + e % (E / 2) : E * lane + e;
}

// Codes of a warp's row y (ap_dim order) into cs[HD] (warp's shared memory) and its scales into d[]: element e's
// block scale.  err: bound of |y - exact|; returns whether some code or scale is not certain within it.
template <int HD, bool HALVES, bool CHECK>
ER_DEV bool ap_quant(const float (&y)[HD / 32], const float (&err)[HD / 32], uint8_t *cs, float (&d)[HD / 32],
                     int lane) {
    constexpr int E = HD / 32, S = HALVES ? 2 : 1, EP = E / S, LANES = 32 / EP;  // a block: EP elements of LANES lanes
    bool unsure = false;
#pragma unroll
    for (int s = 0; s < S; ++s) {
        // the largest size: NaN counts as the largest of all (its bits are above infinity's)
        unsigned big = 0;
#pragma unroll
        for (int e = 0; e < EP; ++e) big = max(big, __float_as_uint(y[s * EP + e]) & 0x7fffffffu);
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
        // of those of that size the first one's sign: key = index * 2 + sign
        unsigned key = 0xffffu;
#pragma unroll
        for (int e = EP - 1; e >= 0; --e) {
            const unsigned u = __float_as_uint(y[s * EP + e]);
            if ((u & 0x7fffffffu) == big) key = (unsigned)(((EP * lane + e) & 31) * 2) | (u >> 31);
        }
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) key = min(key, __shfl_xor_sync(0xffffffffu, key, o));
        const float m = __uint_as_float(big | (key << 31));
        const float dd = pg_scale(m);
        if (CHECK) {
            float lo = 0.f, hi = 0.f;  // the exact largest size lies in [lo, hi]
#pragma unroll
            for (int e = 0; e < EP; ++e) {
                lo = fmaxf(lo, fabsf(y[s * EP + e]) - err[s * EP + e]);
                hi = fmaxf(hi, fabsf(y[s * EP + e]) + err[s * EP + e]);
            }
            lo = group_max<LANES>(lo);
            hi = group_max<LANES>(hi);
            unsure |= pg_scale(lo) != pg_scale(hi);
#pragma unroll
            for (int e = 0; e < EP; ++e)  // could a value of the other sign be the largest?
                unsure |= fabsf(y[s * EP + e]) + err[s * EP + e] >= lo && (__float_as_uint(y[s * EP + e]) >> 31) != (key & 1u);
        }
#pragma unroll
        for (int e = 0; e < EP; ++e) {
            const float r = y[s * EP + e] / dd;
            d[s * EP + e] = dd;
            cs[ap_dim<HD, HALVES>(lane, s * EP + e)] =
                (uint8_t)(dd != 0.f && !isnan(dd) ? (int)fminf(fmaxf(roundf(r) + 8.f, 0.f), 15.f) : 8);
            if (CHECK && dd != 0.f) {
                const float t = fabsf(r);
                // distance of |r| from the border between two codes; its own rounding is at most t 2^-24
                unsure |= fabsf(t - (floorf(t) + 0.5f)) <= err[s * EP + e] / fabsf(dd) * 1.0001f + t * 1.2e-7f;
            }
        }
    }
    return unsure;
}

template <class T, int HD, bool HALVES>
__global__ void __launch_bounds__(AP_WARPS * 32) pages_append_kernel(PagesView p, er_pages_append_args a) {
    constexpr int E = HD / 32;
    __shared__ __align__(16) uint8_t codes[AP_WARPS][HD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int heads = a.n_heads + 2 * p.KV;
    const long long items = (long long)a.n_tokens * heads;
    for (long long it = (long long)blockIdx.x * AP_WARPS + warp; it < items; it += (long long)gridDim.x * AP_WARPS) {
        const int t = (int)(it / heads), h = (int)(it - (long long)t * heads);
        const int slot = a.slots_dev[t];
        if (slot < 0) continue;
        const int pos = a.rope_dev ? a.positions_dev[t] : 0;
        if ((long long)slot >= (long long)p.n_pages * p.page_rows ||
            (a.rope_dev && (pos < 0 || pos >= a.rope_positions))) {
            if (lane == 0) atomicOr(p.flags, ER_PAGES_FLAG_RANGE);
            continue;
        }
        const int what = h < a.n_heads ? 0 : h < a.n_heads + p.KV ? 1 : 2;  // query, key, value
        const int hh = what == 0 ? h : what == 1 ? h - a.n_heads : h - a.n_heads - p.KV;
        const T *src = (what == 0   ? (const T *)a.q_dev + t * a.q_stride
                        : what == 1 ? (const T *)a.k_dev + t * a.k_stride
                                    : (const T *)a.v_dev + t * a.v_stride) + (size_t)hh * HD;
        const float *gain = what == 0 ? a.q_gain_dev : what == 1 ? a.k_gain_dev : nullptr;
        const bool turn = a.rope_dev && what < 2;
        float x[E], y[E], err[E], cs_[E], sn_[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            x[e] = pg_ld<T>(src + ap_dim<HD, HALVES>(lane, e));
            y[e] = x[e];
            err[e] = 0.f;
        }
        if (gain) {
            float ss = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
            for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            const float rs = 1.f / sqrtf(ss / HD + a.eps);
#pragma unroll
            for (int e = 0; e < E; ++e) y[e] = x[e] * rs * gain[ap_dim<HD, HALVES>(lane, e)];
        }
        if (turn) {
            const float2 *tab = reinterpret_cast<const float2 *>(a.rope_dev) + (size_t)pos * (HD / 2);
#pragma unroll
            for (int i = 0; i < E / 2; ++i) {
                const int e0 = HALVES ? i : 2 * i, e1 = HALVES ? i + E / 2 : 2 * i + 1;
                const float2 c = tab[HALVES ? ap_dim<HD, true>(lane, i) : (E * lane) / 2 + i];
                cs_[e0] = c.x;
                sn_[e0] = c.y;
                const float ya = y[e0], yb = y[e1];
                y[e0] = ya * c.x - yb * c.y;
                y[e1] = yb * c.x + ya * c.y;
                err[e0] = err[e1] = fabsf(ya) + fabsf(yb);
            }
        } else if (gain) {
#pragma unroll
            for (int e = 0; e < E; ++e) err[e] = fabsf(y[e]);
        }
        if (what == 0) {
            T *dst = (T *)a.q_out_dev + t * a.q_out_stride + (size_t)hh * HD;
#pragma unroll
            for (int e = 0; e < E; ++e) dst[ap_dim<HD, HALVES>(lane, e)] = pg_cvt<T>(y[e]);
            continue;
        }
        float d[E];
        if (what == 1 && (gain || turn)) {
            // float32 rounding of y: the sum of HD squares at most 9 steps of 2^-24 (half of that in its root), the
            // division, the root and two products 4 more, the rotation 3: below 12 * 2^-24 of |a| + |b|
#pragma unroll
            for (int e = 0; e < E; ++e) err[e] *= 12.f * 5.9604645e-8f;
            const bool unsure = ap_quant<HD, HALVES, true>(y, err, codes[warp], d, lane);
            if (__any_sync(0xffffffffu, unsure)) {
                // the row again in float64: its codes are those of the formula whatever the float32 steps were
                double z[E], ss = 0.0;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    z[e] = (double)x[e];
                    ss += z[e] * z[e];
                }
                if (gain) {
#pragma unroll
                    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                    const double rs = sqrt(ss / HD + (double)a.eps);
#pragma unroll
                    for (int e = 0; e < E; ++e) z[e] = z[e] / rs * (double)gain[ap_dim<HD, HALVES>(lane, e)];
                }
                if (turn) {
#pragma unroll
                    for (int i = 0; i < E / 2; ++i) {
                        const int e0 = HALVES ? i : 2 * i, e1 = HALVES ? i + E / 2 : 2 * i + 1;
                        const double za = z[e0], zb = z[e1], c = (double)cs_[e0], sn = (double)sn_[e0];
                        z[e0] = za * c - zb * sn;
                        z[e1] = zb * c + za * sn;
                    }
                }
#pragma unroll
                for (int e = 0; e < E; ++e) y[e] = (float)z[e];
                __syncwarp();
                ap_quant<HD, HALVES, false>(y, err, codes[warp], d, lane);
            }
        } else {
            ap_quant<HD, HALVES, false>(y, err, codes[warp], d, lane);
        }
        __syncwarp();
        uint8_t *tile = pg_tile(p.pool, p.page_rows, p.KV, HD, slot, hh);
        const int r = (slot % p.page_rows) & 15;
        const uint8_t *cs = codes[warp];
        if (what == 1) {
            if (lane < HD / 8) {  // word w: dims 32 b + 8 t .. + 7
                const int tq = lane / (HD / 32), b = lane % (HD / 32);
                const uint2 c8 = *reinterpret_cast<const uint2 *>(cs + 32 * b + 8 * tq);
                uint32_t w = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int j = 2 * i + e;
                        w |= (((j < 4 ? c8.x : c8.y) >> (8 * (j & 3))) & 15u) << (4 * i + 16 * e);
                    }
                *reinterpret_cast<uint32_t *>(tile + pg_k_word(r, lane, HD)) = w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < HD / 64; ++i) {
                const int j = lane + 32 * i, dim = 16 * (j >> 3) + (j & 7);
                tile[pg_off_v(HD) + pg_v_byte(r, j, HD)] = (uint8_t)(cs[dim] | cs[dim + 8] << 4);
            }
        }
        // the lane that holds a block's first dim writes its scale
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int dim = ap_dim<HD, HALVES>(lane, e);
            if ((dim & 31) == 0) {
                __half *sc = reinterpret_cast<__half *>(tile + (what == 1 ? pg_off_ks(HD) : pg_off_vs(HD)));
                sc[what == 1 ? r * (HD / 32) + dim / 32 : pg_vs_half(r, dim / 32, HD)] = __float2half_rn(d[e]);
            }
        }
        __syncwarp();
    }
}

template <class T>
static cudaError_t append_t(const PagesView &p, const er_pages_append_args &a, int num_sms, cudaStream_t st) {
    const long long items = (long long)a.n_tokens * (a.n_heads + 2 * p.KV);
    long long blocks = (items + AP_WARPS - 1) / AP_WARPS;
    if (blocks > 64ll * num_sms) blocks = 64ll * num_sms;
    if (blocks < 1) return cudaSuccess;
    const bool halves = a.rope_style == ER_ROPE_HALVES;
    if (p.hd == 128)
        halves ? pages_append_kernel<T, 128, true><<<(unsigned)blocks, AP_WARPS * 32, 0, st>>>(p, a)
               : pages_append_kernel<T, 128, false><<<(unsigned)blocks, AP_WARPS * 32, 0, st>>>(p, a);
    else
        halves ? pages_append_kernel<T, 64, true><<<(unsigned)blocks, AP_WARPS * 32, 0, st>>>(p, a)
               : pages_append_kernel<T, 64, false><<<(unsigned)blocks, AP_WARPS * 32, 0, st>>>(p, a);
    return cudaGetLastError();
}

cudaError_t launch_pages_append(const PagesView &p, const er_pages_append_args &a, int num_sms, cudaStream_t st) {
    return a.type == ER_F32   ? append_t<float>(p, a, num_sms, st)
           : a.type == ER_F16 ? append_t<__half>(p, a, num_sms, st)
                              : append_t<__nv_bfloat16>(p, a, num_sms, st);
}

// ---------------------------------------------------------------------------
// rows out: one warp per (slot, head), K then V
// ---------------------------------------------------------------------------
template <class T, int HD>
__global__ void __launch_bounds__(256) pages_read_kernel(PagesView p, int n, const int32_t *slots, T *k, T *v) {
    const int lane = threadIdx.x & 31;
    const long long it = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (it >= (long long)n * p.KV) return;
    const int t = (int)(it / p.KV), h = (int)(it - (long long)t * p.KV);
    const int slot = slots[t];
    if (slot < 0) return;
    if ((long long)slot >= (long long)p.n_pages * p.page_rows) {
        if (lane == 0) atomicOr(p.flags, ER_PAGES_FLAG_RANGE);
        return;
    }
    const uint8_t *tile = pg_tile(p.pool, p.page_rows, p.KV, HD, slot, h);
    const int r = (slot % p.page_rows) & 15;
    const size_t out = (size_t)it * HD;
    const __half *ks = reinterpret_cast<const __half *>(tile + pg_off_ks(HD));
    const __half *vs = reinterpret_cast<const __half *>(tile + pg_off_vs(HD));
    if (k && lane < HD / 8) {
        const int tq = lane / (HD / 32), b = lane % (HD / 32);
        const uint32_t w = *reinterpret_cast<const uint32_t *>(tile + pg_k_word(r, lane, HD));
        const float d = __half2float(ks[r * (HD / 32) + b]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                k[out + 32 * b + 8 * tq + 2 * i + e] = pg_cvt<T>(d * (float)((int)((w >> (4 * i + 16 * e)) & 15u) - 8));
    }
    if (v) {
#pragma unroll
        for (int i = 0; i < HD / 64; ++i) {
            const int j = lane + 32 * i, dim = 16 * (j >> 3) + (j & 7);
            const int c = tile[pg_off_v(HD) + pg_v_byte(r, j, HD)];
            const float d = __half2float(vs[pg_vs_half(r, dim / 32, HD)]);
            v[out + dim] = pg_cvt<T>(d * (float)((c & 15) - 8));
            v[out + dim + 8] = pg_cvt<T>(d * (float)((c >> 4) - 8));
        }
    }
}

template <class T>
static cudaError_t read_t(const PagesView &p, int n, const int32_t *slots, void *k, void *v, cudaStream_t st) {
    const long long blocks = ((long long)n * p.KV + 7) / 8;
    if (blocks < 1) return cudaSuccess;
    if (p.hd == 128) pages_read_kernel<T, 128><<<(unsigned)blocks, 256, 0, st>>>(p, n, slots, (T *)k, (T *)v);
    else pages_read_kernel<T, 64><<<(unsigned)blocks, 256, 0, st>>>(p, n, slots, (T *)k, (T *)v);
    return cudaGetLastError();
}

cudaError_t launch_pages_read(const PagesView &p, int n, const int32_t *slots, int type, void *k, void *v,
                              cudaStream_t st) {
    return type == ER_F32   ? read_t<float>(p, n, slots, k, v, st)
           : type == ER_F16 ? read_t<__half>(p, n, slots, k, v, st)
                            : read_t<__nv_bfloat16>(p, n, slots, k, v, st);
}

}  // namespace er
