// Attention over the paged 4-bit K/V cache (pages.cuh) for few query rows a sequence: o = softmax(scale q k^T) v
// over the rows that a token attends, in one pass with a running reference m and sums
//   p_r = 2^(s_r - m + 7),  l = sum p_r,  o = sum p_r v_r   (s in log2 units),
// rescaled by 2^(m - m') when a score passes m by more than 8 (so p <= 2^15, an fp16 number, and most tiles skip the
// rescale).
//
// What bounds it: the cache's bytes (18 / 32 a value); next, instructions: two a value to turn codes into fp16 pairs
// and feed the tensor cores, so a tile's codes are laid out as the fragments take them and a mask and one FMA yield
// a pair.
//
// Work split.  A unit is a (sequence, group of 8 query rows, KV head); a query row is a (token, head of the KV
// head's group).  The 16-row tiles that the units attend form one list in order of unit; CTA c of C takes the
// contiguous range [c N / C, (c + 1) N / C) and its warps contiguous parts of that, so every SM streams the same
// bytes whatever the lengths.  A unit that lies in one warp's part is finished there; otherwise the warps' states
// are joined in shared memory, and a unit of several CTAs by the last of them to arrive, always in list order:
//   M = max m_w,  o = sum 2^(m_w - M) o_w / sum 2^(m_w - M) l_w.
//
// A warp's tiles arrive by bulk copies (one a tile, 18 HD bytes: codes and scales of K and V) in a ring of its own,
// each slot with its mbarrier; the table entries of the next 32 tiles are held a lane each, so no copy waits for a
// table.
//
// Arithmetic per tile (mma.sync m16n8k16, fp32 sums): A = the 8 query rows, rows 0..7 their hi fp16 half and 8..15 the lo
// half (q = hi + lo to 2^-22 of the row's largest); B = K.  The accumulators' hi and lo rows sit in one lane, which adds
// them.  The scores' layout is the A layout of P V; p = hi + lo again; B = V.  Cached values are fp16 numbers
// (pages.cuh), so the only rounding next to fp32's is those 2^-22.
//
// Masks.  Tiles that some row of the unit attends only in part go through a path that masks scores and zeroes the
// scales of rows nobody attends (they may hold anything); a NaN value that only some of the unit's tokens attend
// is carried by their scores instead.
#include "internal.h"
#include "pages.cuh"

namespace er {

constexpr int PD_WARPS = 12;
constexpr int PD_THREADS = PD_WARPS * 32;
constexpr int PD_SLOTS = 5;
constexpr int PD_ROWS = 8;       // query rows of a unit
constexpr int PD_MIN_TILES = 4;  // tiles of a CTA at least
constexpr float PD_UP = 7.f;     // p = 2^(s - m + PD_UP)
constexpr float PD_SLACK = 8.f;  // scores may pass m by this much

template <int HD>
struct PdCfg {
    static constexpr int TILE = pg_tile_bytes(HD);
    static constexpr int NB = HD / 32;               // 32-dim blocks
    static constexpr int NTD = HD / 8;               // n8 tiles of P V
    static constexpr int STATE = PD_ROWS * HD + 16;  // floats of a state: o [8][HD], m [8], l [8]
    static constexpr int RING = PD_SLOTS * TILE;     // a warp's; later its last segment's state
    static constexpr int OFF_FIRST = PD_WARPS * RING;
    static constexpr int OFF_W = OFF_FIRST + PD_WARPS * STATE * 4;
    static constexpr int OFF_NT = OFF_W + (ER_PAGES_MAX_SEQS + 1) * 8;
    static constexpr int OFF_T0 = OFF_NT + ER_PAGES_MAX_SEQS * 4;
    static constexpr int OFF_BARS = OFF_T0 + ER_PAGES_MAX_SEQS * 4 + 8;
    static constexpr int OFF_MISC = OFF_BARS + PD_WARPS * PD_SLOTS * 8;
    static constexpr int SMEM = OFF_MISC + 2048;
    static_assert(RING >= STATE * 4 && OFF_W % 8 == 0 && OFF_BARS % 8 == 0, "shared memory layout");
};

// a piece of a unit that some warp holds as a state
struct PdSeg {
    long long u0, u1;  // the unit's tiles in the list
    int b, rg, h;
    int off;  // byte offset of the state in shared memory, -1: none
};
struct PdMisc {
    PdSeg seg[2 * PD_WARPS];
    long long wsum[PD_WARPS];
    int run[2 * PD_WARPS + 1];
    int n_runs;
    int wait_bad;
    int last[2];
};

ER_DEV float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
ER_DEV uint32_t h2_dup(uint32_t h2, int hi) { return prmt(h2, h2, hi ? 0x3232u : 0x1010u); }
ER_DEV uint32_t h2_mul(uint32_t a, uint32_t b) {
    __half2 r = __hmul2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
    return *reinterpret_cast<uint32_t *>(&r);
}
ER_DEV uint32_t pd_pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
ER_DEV void pd_split(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pd_pack(a, b);
    const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    lo = pd_pack(a - h.x, b - h.y);
}
// nibble n of each half of w (bits 4 n ..) as the fp16 pair 16 + c
template <int N>
ER_DEV uint32_t pd_code(uint32_t w) {
    return lop3_and_or(N == 0 ? w << 6 : N == 1 ? w << 2 : N == 2 ? w >> 2 : w >> 6, 0x03C003C0u, 0x4C004C00u);
}
constexpr uint32_t PD_M24 = 0xCE00CE00u;  // half2(-24, -24)

struct PdArgs {
    PagesView p;
    er_pages_attention_args a;
    float *part;  // [CTAs][2] states of units that several CTAs share
    int *cnt;     // [CTAs] arrivals, zero between launches
};

// query row r of group rg of sequence b, KV head h: its token's row in q / out and its head
ER_DEV void pd_row(int r, int rg, int G, int q0, int h, int &row, int &head, int &i) {
    const int f = rg * PD_ROWS + r;
    i = f / G;
    row = q0 + i;
    head = h * G + (f - i * G);
}

template <class T, int HD>
__global__ void __launch_bounds__(PD_THREADS, 1) pages_decode_kernel(const PdArgs P) {
    using C = PdCfg<HD>;
    extern __shared__ __align__(128) uint8_t smem[];
    long long *W = reinterpret_cast<long long *>(smem + C::OFF_W);
    int *NT = reinterpret_cast<int *>(smem + C::OFF_NT), *T0 = reinterpret_cast<int *>(smem + C::OFF_T0);
    PdMisc &ms = *reinterpret_cast<PdMisc *>(smem + C::OFF_MISC);
    static_assert(sizeof(PdMisc) <= 2048, "misc");
    const er_pages_attention_args &a = P.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int KV = P.p.KV, G = a.n_heads / KV, R = P.p.page_rows;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BARS) + warp * PD_SLOTS;
    uint8_t *ring = smem + warp * C::RING;
    if (lane < PD_SLOTS) mbar_init(bars + lane, 1);
    if (tid == 0) ms.wait_bad = 0;
    if (lane < 2) ms.seg[2 * warp + lane].off = -1;
    fence_mbar_init();

    // ---- the list: tiles of every sequence, prefix sums in W
    {
        constexpr int PER = (ER_PAGES_MAX_SEQS + PD_THREADS - 1) / PD_THREADS;
        const int per = (a.n_seqs + PD_THREADS - 1) / PD_THREADS;
        long long own[PER], sum = 0;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            own[k] = 0;
            const int b = tid * per + k;
            if (k < per && b < a.n_seqs) {
                const int q0 = a.q_start_dev[b], q1 = a.q_start_dev[b + 1], len = a.lens_dev[b];
                int nt = 0, t0 = 0;
                const bool bad = q0 < 0 || q1 < q0 || q1 > a.n_tokens || len < 0 ||
                                 (long long)len > (long long)a.table_stride * R;
                if (bad) {
                    if (blockIdx.x == 0) atomicOr(P.p.flags, ER_PAGES_FLAG_RANGE);
                } else if (q1 > q0 && len > 0) {
                    const int lo = a.window ? max(0, len - (q1 - q0) - a.window + 1) : 0;
                    t0 = lo >> 4;
                    nt = ((len - 1) >> 4) - t0 + 1;
                    own[k] = (long long)nt * ((((long long)(q1 - q0) * G + PD_ROWS - 1) / PD_ROWS) * KV);
                } else if (q1 > q0) {
                    nt = -1;  // rows without anything to attend: zeros, below
                }
                NT[b] = nt;
                T0[b] = t0;
            }
            sum += own[k];
        }
        long long inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += x;
        }
        if (lane == 31) ms.wsum[warp] = inc;
        __syncthreads();
        long long at = inc - sum;
        for (int w = 0; w < warp; ++w) at += ms.wsum[w];
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            const int b = tid * per + k;
            if (k < per && b < a.n_seqs) {
                W[b] = at;
                at += own[k];
                if (b == a.n_seqs - 1) W[a.n_seqs] = at;
            }
        }
        __syncthreads();
    }
    // sequences of length 0: zeros and -infinity
    for (int b = blockIdx.x; b < a.n_seqs; b += gridDim.x) {
        if (NT[b] != -1) continue;
        const int q0 = a.q_start_dev[b];
        const long long n = (long long)(a.q_start_dev[b + 1] - q0) * a.n_heads;
        for (long long i = tid; i < n * HD; i += PD_THREADS) {
            const int row = q0 + (int)(i / HD / a.n_heads), head = (int)(i / HD % a.n_heads);
            ((T *)a.out_dev)[row * a.out_stride + (size_t)head * HD + i % HD] = pg_cvt<T>(0.f);
        }
        if (a.lse_dev)
            for (long long i = tid; i < n; i += PD_THREADS) a.lse_dev[(size_t)q0 * a.n_heads + i] = -INFINITY;
    }
    const long long N = W[a.n_seqs];
    if (N == 0) return;
    const long long C_ = min((long long)gridDim.x, (N + PD_MIN_TILES - 1) / PD_MIN_TILES);
    if ((long long)blockIdx.x >= C_) return;
    const long long c0 = blockIdx.x * N / C_, c1 = (blockIdx.x + 1) * N / C_;
    const long long w0 = c0 + warp * (c1 - c0) / PD_WARPS, w1 = c0 + (warp + 1) * (c1 - c0) / PD_WARPS;

    auto seq_of = [&](long long i) {  // the sequence of list entry i: the last b with W[b] <= i (empty ones are skipped)
        int lo = 0, hi = a.n_seqs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (W[mid] <= i) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    };
    // where list entry i lies in the pool
    auto source = [&](long long i) -> unsigned long long {
        if (i >= w1) return 0;
        const int b = seq_of(i), nt = NT[b];
        const long long rem = i - W[b], unit = rem / nt;
        const int row = (T0[b] + (int)(rem - unit * nt)) << 4, h = (int)(unit % KV);
        const int blk = row / R;
        int page = a.tables_dev[(size_t)b * a.table_stride + blk];
        if (page < 0 || page >= P.p.n_pages) {
            atomicOr(P.p.flags, ER_PAGES_FLAG_RANGE);
            page = 0;
        }
        return (((unsigned long long)page * KV + h) * (R >> 4) + ((row - blk * R) >> 4)) * C::TILE;
    };
    long long ibase = w0, inext = w0;  // entries ibase .. + 31 are in cur, the 32 after them in nxt; next to request
    unsigned long long cur = source(w0 + lane), nxt = source(w0 + 32 + lane);
    auto issue = [&]() {  // requests the next tile (whole warp)
        if (inext >= w1) return;
        if (inext - ibase == 32) {
            ibase += 32;
            cur = nxt;
            nxt = source(ibase + 32 + lane);
        }
        const unsigned long long off = __shfl_sync(0xffffffffu, cur, (int)(inext - ibase));
        if (lane == 0) {
            const int slot = (int)((inext - w0) % PD_SLOTS);
            mbar_arrive_expect_tx(bars + slot, C::TILE);
            bulk_g2s(ring + slot * C::TILE, P.p.pool + off, C::TILE, bars + slot);
        }
        ++inext;
    };
    for (int k = 0; k < PD_SLOTS; ++k) issue();

    const float qscale = (a.scale != 0.f ? a.scale : 1.f / sqrtf((float)HD)) * 1.4426950408889634f;
    const bool vec = ((uintptr_t)a.q_dev & 15) == 0 && (a.q_stride * sizeof(T)) % 16 == 0;
    int wslot = 0;         // ring slot and parity of the next tile to consume
    uint32_t wpar = 0;
    bool bad = false;      // a wait gave up

    for (long long i = w0; i < w1 && !bad;) {
        // ---- the unit of entry i
        const int b = seq_of(i), nt = NT[b], t0 = T0[b];
        const long long unit = (i - W[b]) / nt, u0 = W[b] + unit * nt, u1 = u0 + nt;
        const int h = (int)(unit % KV), rg = (int)(unit / KV);
        const int q0 = a.q_start_dev[b], qn = a.q_start_dev[b + 1] - q0, len = a.lens_dev[b];
        const long long send = min(u1, w1);
        int row, head, tok;
        pd_row(g, rg, G, q0, h, row, head, tok);
        const bool real = tok < qn;
        // rows that this lane's query row attends, and the ranges that all and any of the unit's rows attend
        const int tok0 = rg * PD_ROWS / G, tok1 = min((rg * PD_ROWS + PD_ROWS - 1) / G, qn - 1);
        const int pos = real ? len - qn + tok : -1;
        const int first = a.window ? max(0, pos - a.window + 1) : 0;
        const int any_lo = a.window ? max(0, len - qn + tok0 - a.window + 1) : 0, any_hi = len - qn + tok1;
        const int all_lo = a.window ? max(0, len - qn + tok1 - a.window + 1) : 0, all_hi = len - qn + tok0;

        uint32_t qa[2 * C::NB][4];  // k16 steps: dims 32 b + 8 t + 4 m .. + 3 of step 2 b + m
        float down;
        {
            float x[C::NB][8], top = 0.f;
#pragma unroll
            for (int bb = 0; bb < C::NB; ++bb) {
                const T *src = (const T *)a.q_dev + row * a.q_stride + (size_t)head * HD + 32 * bb + 8 * t;
                if (!real) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[bb][e] = 0.f;
                } else if (vec) {
                    __align__(16) T v[8];
#pragma unroll
                    for (int k = 0; k < (int)(8 * sizeof(T)) / 16; ++k)
                        reinterpret_cast<uint4 *>(v)[k] = reinterpret_cast<const uint4 *>(src)[k];
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[bb][e] = pg_ld<T>(v + e) * qscale;
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[bb][e] = pg_ld<T>(src + e) * qscale;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(x[bb][e]));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            int ex = 0;  // the row's largest goes to [2^14, 2^15), so the lo halves of all that matters are normal
            if (top > 0.f && isfinite(top)) {
                frexpf(top, &ex);
                ex = min(max(15 - ex, -126), 126);
            }
            const float up = ldexpf(1.f, ex);
            down = ldexpf(1.f, -ex);
#pragma unroll
            for (int bb = 0; bb < C::NB; ++bb)
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    pd_split(x[bb][4 * m] * up, x[bb][4 * m + 1] * up, qa[2 * bb + m][0], qa[2 * bb + m][1]);
                    pd_split(x[bb][4 * m + 2] * up, x[bb][4 * m + 3] * up, qa[2 * bb + m][2], qa[2 * bb + m][3]);
                }
        }
        float m = -INFINITY, l = 0.f;
        float o[C::NTD][4];
#pragma unroll
        for (int j = 0; j < C::NTD; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

        for (; i < send; ++i) {
            if (!__all_sync(0xffffffffu, mbar_wait(bars + wslot, wpar))) {
                bad = true;
                break;
            }
            const uint32_t sl = smem_u32(ring + wslot * C::TILE);
            const int r0 = (t0 + (int)(i - u0)) << 4;
            const bool edge = r0 < all_lo || r0 + 15 > all_hi;
            if (!(edge && (r0 > any_hi || r0 + 15 < any_lo))) {
                // ---- scores of rows r0 .. + 15: two n8 tiles
                float s[2][4];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    s[n][0] = s[n][1] = s[n][2] = s[n][3] = 0.f;
                    const int rr = 8 * n + g;
                    uint32_t w[C::NB], ds[C::NB / 2];
                    if constexpr (HD == 128) {
                        const uint4 x = lds128(sl + rr * 64 + t * 16);
                        w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
                        const uint2 y = lds64(sl + pg_off_ks(HD) + rr * 8);
                        ds[0] = y.x; ds[1] = y.y;
                    } else {
                        const uint2 x = lds64(sl + rr * 32 + t * 8);
                        w[0] = x.x; w[1] = x.y;
                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(ds[0]) : "r"(sl + pg_off_ks(HD) + rr * 4));
                    }
#pragma unroll
                    for (int bb = 0; bb < C::NB; ++bb) {
                        const uint32_t d = h2_dup(ds[bb >> 1], bb & 1), z = h2_mul(d, PD_M24);
                        mma_16816(s[n], qa[2 * bb], h2_fma(pd_code<0>(w[bb]), d, z), h2_fma(pd_code<1>(w[bb]), d, z), s[n]);
                        mma_16816(s[n], qa[2 * bb + 1], h2_fma(pd_code<2>(w[bb]), d, z), h2_fma(pd_code<3>(w[bb]), d, z), s[n]);
                    }
                }
                // V scales of rows 2t, 2t + 1 (vd[.][0]) and 2t + 8, 2t + 9 (vd[.][1]), a pair a word
                uint32_t vd[C::NB][2];
#pragma unroll
                for (int k = 0; k < C::NB / 2; ++k) {
                    const uint4 x = lds128(sl + pg_off_vs(HD) + t * (C::NB * 8) + 16 * k);
                    vd[2 * k][0] = x.x; vd[2 * k][1] = x.y; vd[2 * k + 1][0] = x.z; vd[2 * k + 1][1] = x.w;
                }
                // score k: row r0 + 2 t + (k & 1) + 8 (k >> 1)
                float sc[4] = {(s[0][0] + s[0][2]) * down, (s[0][1] + s[0][3]) * down, (s[1][0] + s[1][2]) * down,
                               (s[1][1] + s[1][3]) * down};
                if (edge) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int r = r0 + 2 * t + (k & 1) + 8 * (k >> 1);
                        const uint32_t half = (k & 1) ? 0xFFFF0000u : 0x0000FFFFu;
                        bool nan = false;
#pragma unroll
                        for (int bb = 0; bb < C::NB; ++bb) {
                            const uint32_t x = (vd[bb][k >> 1] & half) & 0x7FFF7FFFu;
                            const bool n = x > (0x7C007C00u & half);
                            nan |= n;
                            if (n || r < any_lo || r > any_hi) vd[bb][k >> 1] &= ~half;
                        }
                        if (nan) sc[k] = NAN;
                        if (r < first || r > pos) sc[k] = -INFINITY;
                    }
                }
                float mt = fmaxf(fmaxf(sc[0], sc[1]), fmaxf(sc[2], sc[3]));
                mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
                mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
                if (__any_sync(0xffffffffu, mt > m + PD_SLACK)) {
                    const float mn = mt > m + PD_SLACK ? mt : m;
                    const float corr = mn == m ? 1.f : ex2(m - mn);
                    l *= corr;
#pragma unroll
                    for (int j = 0; j < C::NTD; ++j) {
                        o[j][0] *= corr; o[j][1] *= corr; o[j][2] *= corr; o[j][3] *= corr;
                    }
                    m = mn;
                }
                const float base = (m == -INFINITY ? 0.f : m) - PD_UP;
                float p[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) p[k] = ex2(sc[k] - base);
                l += (p[0] + p[1]) + (p[2] + p[3]);
                uint32_t pa[4];
                pd_split(p[0], p[1], pa[0], pa[1]);
                pd_split(p[2], p[3], pa[2], pa[3]);
                // ---- o += p v: word u of run q holds dims 64 q + 16 u + g and + 8 of the lane's four rows
#pragma unroll
                for (int q = 0; q < HD / 64; ++q) {
                    const uint4 x = lds128(sl + pg_off_v(HD) + q * 512 + lane * 16);
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int hb = 0; hb < 2; ++hb) {
                        const uint32_t d0 = vd[2 * q + hb][0], d1 = vd[2 * q + hb][1], z0 = h2_mul(d0, PD_M24),
                                       z1 = h2_mul(d1, PD_M24);
#pragma unroll
                        for (int u = 2 * hb; u < 2 * hb + 2; ++u) {
                            const int j = 8 * q + 2 * u;
                            mma_16816(o[j], pa, h2_fma(pd_code<0>(w[u]), d0, z0), h2_fma(pd_code<2>(w[u]), d1, z1), o[j]);
                            mma_16816(o[j + 1], pa, h2_fma(pd_code<1>(w[u]), d0, z0), h2_fma(pd_code<3>(w[u]), d1, z1),
                                      o[j + 1]);
                        }
                    }
                }
            }
            __syncwarp();  // every lane is done with the slot
            issue();
            if (++wslot == PD_SLOTS) {
                wslot = 0;
                wpar ^= 1u;
            }
        }
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (bad) break;
        const long long sbeg = max(u0, w0);
        if (sbeg == u0 && send == u1) {  // the whole unit
            if (real) {
                const float inv = l == 0.f ? 0.f : 1.f / l;
                T *out = (T *)a.out_dev + row * a.out_stride + (size_t)head * HD + 2 * t;
                const bool pair = ((uintptr_t)out & (2 * sizeof(T) - 1)) == 0;
#pragma unroll
                for (int j = 0; j < C::NTD; ++j) {
                    const float y0 = l == 0.f ? 0.f : (o[j][0] + o[j][2]) * inv, y1 = l == 0.f ? 0.f : (o[j][1] + o[j][3]) * inv;
                    __align__(8) T v[2] = {pg_cvt<T>(y0), pg_cvt<T>(y1)};
                    if (pair) {
                        if constexpr (sizeof(T) == 4) *reinterpret_cast<uint2 *>(out + 8 * j) = *reinterpret_cast<uint2 *>(v);
                        else *reinterpret_cast<uint32_t *>(out + 8 * j) = *reinterpret_cast<uint32_t *>(v);
                    } else {
                        out[8 * j] = v[0];
                        out[8 * j + 1] = v[1];
                    }
                }
                if (a.lse_dev && t == 0)
                    a.lse_dev[(size_t)row * a.n_heads + head] =
                        l == 0.f ? -INFINITY : (m - PD_UP + log2f(l)) * 0.6931471805599453f;
            }
        } else {
            // a state: the last segment's goes into the ring (nothing is on its way there any more)
            const int off = send == w1 ? warp * C::RING : C::OFF_FIRST + warp * C::STATE * 4;
            float *st = reinterpret_cast<float *>(smem + off);
#pragma unroll
            for (int j = 0; j < C::NTD; ++j)
                *reinterpret_cast<float2 *>(st + g * HD + 8 * j + 2 * t) = make_float2(o[j][0] + o[j][2], o[j][1] + o[j][3]);
            if (t == 0) {
                st[PD_ROWS * HD + g] = m;
                st[PD_ROWS * HD + 8 + g] = l;
            }
            if (lane == 0) ms.seg[2 * warp + (send == w1)] = {u0, u1, b, rg, h, off};
        }
    }
    if (bad) {
        if (lane == 0) atomicOr(P.p.flags, ER_FLAG_WAIT);
        ms.wait_bad = 1;
        // copies may still be landing: wait for them (each again with a limit)
        for (long long k = inext - PD_SLOTS > w0 ? inext - PD_SLOTS : w0; k < inext; ++k)
            mbar_wait(bars + (int)((k - w0) % PD_SLOTS), (uint32_t)(((k - w0) / PD_SLOTS) & 1));
    }
    __syncthreads();
    if (tid == 0) {  // runs of neighbouring states of one unit
        int n = 0, k = 0;
        for (int e = 0; e < 2 * PD_WARPS; ++e)
            if (ms.seg[e].off >= 0) {
                if (n == 0 || ms.seg[n - 1].u0 != ms.seg[e].u0) ms.run[k++] = n;
                ms.seg[n++] = ms.seg[e];
            }
        ms.run[k] = n;
        ms.n_runs = ms.wait_bad ? 0 : k;
    }
    __syncthreads();
    const int n_runs = ms.n_runs;
    constexpr int V = HD / 32;  // dims of a lane
    // a row of a unit, joined: o of dims V lane .. , the reference m and sum l
    auto write_row = [&](const PdSeg &sg, int r, const float (&y)[V], float mm, float ll) {
        const int q0 = a.q_start_dev[sg.b], qn = a.q_start_dev[sg.b + 1] - q0;
        int row, head, tok;
        pd_row(r, sg.rg, G, q0, sg.h, row, head, tok);
        if (tok >= qn) return;
        T *out = (T *)a.out_dev + row * a.out_stride + (size_t)head * HD + V * lane;
#pragma unroll
        for (int e = 0; e < V; ++e) out[e] = pg_cvt<T>(ll == 0.f ? 0.f : y[e] / ll);
        if (a.lse_dev && lane == 0)
            a.lse_dev[(size_t)row * a.n_heads + head] =
                ll == 0.f ? -INFINITY : (mm - PD_UP + log2f(ll)) * 0.6931471805599453f;
    };
    for (int it = warp; it < n_runs * PD_ROWS; it += PD_WARPS) {
        const int run = it / PD_ROWS, r = it % PD_ROWS;
        const int e0 = ms.run[run], e1 = ms.run[run + 1];
        const PdSeg &sg = ms.seg[e0];
        float M = -INFINITY;
        for (int e = e0; e < e1; ++e) M = fmaxf(M, reinterpret_cast<float *>(smem + ms.seg[e].off)[PD_ROWS * HD + r]);
        const float base = M == -INFINITY ? 0.f : M;
        float y[V], L = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) y[e] = 0.f;
        for (int e = e0; e < e1; ++e) {
            const float *st = reinterpret_cast<float *>(smem + ms.seg[e].off);
            const float f = ex2(st[PD_ROWS * HD + r] - base);
            L += f * st[PD_ROWS * HD + 8 + r];
#pragma unroll
            for (int k = 0; k < V; ++k) y[k] += f * st[r * HD + V * lane + k];
        }
        if (sg.u0 >= c0 && sg.u1 <= c1) {
            write_row(sg, r, y, M, L);
        } else {
            float *st = P.part + ((size_t)blockIdx.x * 2 + (sg.u0 < c0 ? 0 : 1)) * C::STATE;
#pragma unroll
            for (int k = 0; k < V; ++k) __stcg(st + r * HD + V * lane + k, y[k]);
            if (lane == 0) {
                __stcg(st + PD_ROWS * HD + r, M);
                __stcg(st + PD_ROWS * HD + 8 + r, L);
            }
        }
    }
    // ---- units of several CTAs: the last to arrive joins their states in CTA order
    __threadfence();
    __syncthreads();
    if (tid == 0) {
        ms.last[0] = ms.last[1] = -1;
        int k = 0;
        for (int run = 0; run < n_runs; ++run) {
            const PdSeg &sg = ms.seg[ms.run[run]];
            if (sg.u0 >= c0 && sg.u1 <= c1) continue;
            const int ca = (int)(((sg.u0 + 1) * C_ - 1) / N), cb = (int)((sg.u1 * C_ - 1) / N);
            if (atom_add_acq_rel_gpu(P.cnt + ca, 1) == cb - ca) {
                P.cnt[ca] = 0;
                ms.last[k++] = run;
            }
        }
    }
    __syncthreads();
    float *wts = reinterpret_cast<float *>(smem);                      // [8][CTAs] weights (the ring is free)
    float *acc = reinterpret_cast<float *>(smem) + PD_ROWS * 512;      // [warps][HD]
    for (int k = 0; k < 2; ++k) {
        if (ms.last[k] < 0) break;
        const PdSeg sg = ms.seg[ms.run[ms.last[k]]];
        __syncthreads();  // the states in the ring are read before the weights go there
        const int ca = (int)(((sg.u0 + 1) * C_ - 1) / N), cb = (int)((sg.u1 * C_ - 1) / N), nc = cb - ca + 1;
        auto state = [&](int c) { return P.part + ((size_t)c * 2 + (sg.u0 < c * N / C_ ? 0 : 1)) * C::STATE; };
        const int f0 = sg.rg * PD_ROWS, qn = a.q_start_dev[sg.b + 1] - a.q_start_dev[sg.b];
        const int rows = (int)min((long long)PD_ROWS, (long long)qn * G - f0);
        for (int r = warp; r < rows; r += PD_WARPS) {
            float M = -INFINITY;
            for (int c = lane; c < nc; c += 32) {
                const float x = __ldcg(state(ca + c) + PD_ROWS * HD + r);
                wts[r * 512 + c] = x;
                M = fmaxf(M, x);
            }
#pragma unroll
            for (int off = 16; off; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
            const float base = M == -INFINITY ? 0.f : M;
            for (int c = lane; c < nc; c += 32) wts[r * 512 + c] = ex2(wts[r * 512 + c] - base);
            if (lane == 0) acc[PD_WARPS * HD + r] = M;
        }
        __syncthreads();
        // warp (r, part): every row's CTAs in `parts` pieces
        const int parts = max(1, PD_WARPS / rows);
        float y[V], L = 0.f;
        const int r = warp / parts, part = warp % parts;
        const int ra = (int)((long long)part * nc / parts), rb = (int)((long long)(part + 1) * nc / parts);
        if (r < rows) {
#pragma unroll
            for (int e = 0; e < V; ++e) y[e] = 0.f;
#pragma unroll 8
            for (int c = ra; c < rb; ++c) {
                const float *st = state(ca + c);
                const float f = wts[r * 512 + c];
                L += f * __ldcg(st + PD_ROWS * HD + 8 + r);
                if constexpr (V == 4) {
                    const float4 x = __ldcg(reinterpret_cast<const float4 *>(st + r * HD) + lane);
                    y[0] += f * x.x; y[1] += f * x.y; y[2] += f * x.z; y[3] += f * x.w;
                } else {
                    const float2 x = __ldcg(reinterpret_cast<const float2 *>(st + r * HD) + lane);
                    y[0] += f * x.x; y[1] += f * x.y;
                }
            }
#pragma unroll
            for (int e = 0; e < V; ++e) acc[warp * HD + V * lane + e] = y[e];
            if (lane == 0) acc[PD_WARPS * HD + PD_ROWS + warp] = L;
        }
        __syncthreads();
        if (r < rows && part == 0) {
            float z[V], LL = 0.f;
#pragma unroll
            for (int e = 0; e < V; ++e) z[e] = 0.f;
            for (int x = 0; x < parts; ++x) {
                LL += acc[PD_WARPS * HD + PD_ROWS + warp + x];
#pragma unroll
                for (int e = 0; e < V; ++e) z[e] += acc[(warp + x) * HD + V * lane + e];
            }
            write_row(sg, r, z, acc[PD_WARPS * HD + r], LL);
        }
        __syncthreads();
    }
}

size_t pages_attn_part_floats(int num_sms) { return (size_t)num_sms * 2 * (PD_ROWS * 128 + 16); }

template <class T, int HD>
static cudaError_t decode_prepare() {
    return cudaFuncSetAttribute(pages_decode_kernel<T, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, PdCfg<HD>::SMEM);
}
cudaError_t pages_attn_prepare() {
    cudaError_t e[6] = {decode_prepare<float, 64>(), decode_prepare<float, 128>(), decode_prepare<__half, 64>(),
                        decode_prepare<__half, 128>(), decode_prepare<__nv_bfloat16, 64>(),
                        decode_prepare<__nv_bfloat16, 128>()};
    for (cudaError_t x : e)
        if (x != cudaSuccess) return x;
    return cudaSuccess;
}

template <class T>
static cudaError_t attn_t(const PdArgs &P, int num_sms, cudaStream_t st) {
    if (P.p.hd == 128) pages_decode_kernel<T, 128><<<num_sms, PD_THREADS, PdCfg<128>::SMEM, st>>>(P);
    else pages_decode_kernel<T, 64><<<num_sms, PD_THREADS, PdCfg<64>::SMEM, st>>>(P);
    return cudaGetLastError();
}

cudaError_t launch_pages_attention(const PagesView &p, const er_pages_attention_args &a, float *part, int *cnt,
                                   int num_sms, cudaStream_t st) {
    const PdArgs P = {p, a, part, cnt};
    return a.type == ER_F32   ? attn_t<float>(P, num_sms, st)
           : a.type == ER_F16 ? attn_t<__half>(P, num_sms, st)
                              : attn_t<__nv_bfloat16>(P, num_sms, st);
}

cudaError_t set_wait_limit_pages(unsigned long long ns) { return set_wait_limit_here(ns); }

}  // namespace er
