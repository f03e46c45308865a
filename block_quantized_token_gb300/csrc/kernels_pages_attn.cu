// Attention over the paged 4-bit K/V cache (pages.cuh) for few query rows a sequence: o = softmax(scale q k^T) v
// over the rows that a token attends, in one pass with a running reference m and sums
//   p_r = 2^(s_r - m + 7),  l = sum p_r,  o = sum p_r v_r   (s in log2 units),
// rescaled by 2^(m - m') when a score passes m by more than 8 (so p <= 2^15, an fp16 number, and most tiles skip the
// rescale).
//
// What bounds it: the cache's bytes (18 / 32 a value); next, instructions, two a value to turn codes into operands
// and feed the tensor cores, so a tile's codes are laid out as the operands take them.  Measured, 16 sequences of 8192 rows,
// 32 / 8 heads of 128: bf16 51 us (3.0 TB/s of cache, 0.45 of a copy's rate), fp32 62 us; about a quarter of that is the
// way to the first tile and the joining of states, the rest the loop at half the SM's issue rate (long chains of
// dependent products and exponentials in 2 or 3 warps a scheduler).
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
// Arithmetic (mma.sync m16n8k16, fp32 sums), the cached side as the A operand, the 8 query rows as B's columns:
//   S^T = K Q^T.  fp32 and fp16 queries: K's values as they are (fp16 numbers, pages.cuh), Q exact (fp16) or as hi + lo
//         halves (fp32: 2^-22 of the row's largest).  bf16 queries, exact too: K's codes c - 8 without their scale (9
//         instructions for 8 codes against 14), and the row's scale multiplies the block's sum.  (With the offsets of 1032 and
//         72 left in the codes and taken off the sums it is 5 instructions and the same time, but the error goes with sum
//         |q| d, however small the values beside a block's largest are.)
//   O^T += V^T P^T.  One code word is a lane's whole A operand, a mask and one FMA a pair, exact.  Probabilities go from
//         the scores' layout to B's by movmatrix, as hi + lo halves (2^-22).  hi alone (2^-11) is 47.4 us for 50.8 of bf16,
//         16 x 8192, and moves one bf16 output in twenty by its last bit.
// Masks.  Tiles that some row of the unit attends only in part go through a path that masks scores and zeroes the
// scales of rows nobody attends (they may hold anything).  There a NaN value is carried by the scores of the tokens that
// attend it, where the unit's tokens differ in that (all their dims become NaN).
#include <type_traits>

#include "pages.cuh"
#include "pages.h"

namespace er {

constexpr int PD_MAX_WARPS = 12;
constexpr int PD_STEP = 32;      // rows of a step: two tiles
constexpr int PD_ROWS = 8;       // query rows of a unit
constexpr int PD_SEQS = 512;     // sequences of a launch (more: several launches)
constexpr int PD_MIN_STEPS = 8;  // steps of a CTA at least (fewer only add states to join); of 12 warps 4 have none then
constexpr float PD_UP = 7.f;     // p = 2^(s - m + PD_UP)
constexpr float PD_SLACK = 8.f;  // scores may pass m by this much
constexpr float PD_NONE = -3e38f;  // m before any score

template <class T>
struct PdType;  // RAW: K enters as codes c - 8 (bf16); QLO: queries have a lo half
template <>
struct PdType<float> {
    static constexpr bool RAW = false, QLO = true;
};
template <>
struct PdType<__half> {
    static constexpr bool RAW = false, QLO = false;
};
template <>
struct PdType<__nv_bfloat16> {
    static constexpr bool RAW = true, QLO = false;
};

struct PdSeq {  // a sequence: its rows of q, its length, its steps (-1: rows with nothing to attend)
    int q0, qn, len, ns;
};
// 12 warps hide more latency than 8 where 168 registers a thread nearly hold a warp's state, which they do for HD = 64 (fp32
// stores 12 bytes) and for bf16 queries at 128 dims (32 bytes stored, 44 loaded): ragged 61 x 0..4001, bf16: 45 us against 51;
// 1 x 2048, 64 dims, fp32: 12.7 against 14.7.  fp32 and fp16 queries at 128 dims spill more (16 x 8192 fp32: 69 us against 62).
template <class T, int HD>
struct PdCfg {
    static constexpr int WARPS = HD == 64 || sizeof(T) == 2 && PdType<T>::RAW ? PD_MAX_WARPS : 8;
    static constexpr int THREADS = WARPS * 32;
    static constexpr int SLOTS = WARPS == 8 ? 4 : 3;  // steps in a warp's ring
    static constexpr int TILE = pg_tile_bytes(HD);
    static constexpr int NB = HD / 32;               // 32-dim blocks
    static constexpr int STATE = PD_ROWS * HD + 16;  // floats of a state: o [8][HD], m [8], l [8]
    static constexpr int RING = SLOTS * 2 * TILE; // a warp's; later its last segment's state
    static constexpr int OFF_FIRST = WARPS * RING;
    static constexpr int OFF_W = OFF_FIRST + WARPS * STATE * 4;
    static constexpr int OFF_SEQ = OFF_W + (PD_SEQS + 2) * 8;
    static constexpr int OFF_BARS = OFF_SEQ + PD_SEQS * (int)sizeof(PdSeq);
    static constexpr int OFF_MISC = OFF_BARS + WARPS * SLOTS * 8;
    static constexpr int SMEM = OFF_MISC + 2048;
    static_assert(RING >= STATE * 4 && OFF_W % 8 == 0 && OFF_BARS % 8 == 0 && SMEM <= 232448, "shared memory layout");
};

// a piece of a unit that some warp holds as a state
struct PdSeg {
    long long u0, u1;  // the unit's steps in the list
    int b, rg, h;
    int off;  // byte offset of the state in shared memory, -1: none
};
struct PdMisc {
    PdSeg seg[2 * PD_MAX_WARPS];
    long long wsum[PD_MAX_WARPS];
    int run[2 * PD_MAX_WARPS + 1];  // first of each run in ent
    short ent[2 * PD_MAX_WARPS];    // the states that there are, in list order
    int n_runs;
    int wait_bad;
    int last[2];
};

ER_DEV void pd_split(float a, float b, uint32_t &hi, uint32_t &lo) {
    hi = pg_pack(a, b);
    const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    lo = pg_pack(a - h.x, b - h.y);
}
ER_DEV uint32_t h2_add(uint32_t a, uint32_t b) {
    __half2 r = __hadd2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
    return *reinterpret_cast<uint32_t *>(&r);
}
// nibble 0 / 1 of each half of w as the fp16 pair c - 8: 1024 + c or 64 + c as a mask leaves it, less 1032 or 72
ER_DEV uint32_t pd_low(uint32_t w) { return h2_add(lop3_and_or(w, 0x000F000Fu, 0x64006400u), 0xE408E408u); }
ER_DEV uint32_t pd_high(uint32_t w) { return h2_add(lop3_and_or(w, 0x00F000F0u, 0x54005400u), 0xD480D480u); }
// d += A B without volatile: the compiler may move it between the loads and conversions of other tiles
ER_DEV void pd_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// d = A B + c
ER_DEV void pd_mma_c(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, const float (&c)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}
// the 8x8 transpose of a packed pair matrix
ER_DEV uint32_t pd_trans(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
struct PdArgs {
    PagesView p;
    er_pages_attention_args a;
    int max_rows;  // sequences with as many query rows a KV head, or more, are another kernel's
    float *part;  // [CTAs][2] states of units that several CTAs share
    int *cnt;     // [CTAs] arrivals, zero between launches
    int shortfall;  // tests of the give-up path: arrivals that CTA 0 waits for in vain
};

// the first row that any of a sequence's qn new tokens attends
ER_DEV int pd_row0(int len, int qn, int window) { return pg_first(len - qn, window); }
// x / d for x >= 0, mostly below 2^32
ER_DEV long long pd_div(long long x, int d) {
    return (x >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)d) : x / d;
}

// the CTA of list entry i: the c with c N / C <= i < (c + 1) N / C
ER_DEV int pd_cta(long long i, long long N, int C) { return (int)(((i + 1) * C - 1) / N); }

// query row r of group rg of sequence b, KV head h: its token's row in q / out and its head
ER_DEV void pd_row(int r, int rg, int G, int q0, int h, int &row, int &head, int &i) {
    const int f = rg * PD_ROWS + r;
    i = f / G;
    row = q0 + i;
    head = h * G + (f - i * G);
}

template <class T, int HD>
__global__ void __launch_bounds__((PdCfg<T, HD>::THREADS), 1) pages_decode_kernel(const PdArgs P) {
    using C = PdCfg<T, HD>;
    constexpr int PD_WARPS = C::WARPS, PD_THREADS = C::THREADS, PD_SLOTS = C::SLOTS;
    using Y = PdType<T>;
    extern __shared__ __align__(128) uint8_t smem[];
    long long *W = reinterpret_cast<long long *>(smem + C::OFF_W);
    PdSeq *SQ = reinterpret_cast<PdSeq *>(smem + C::OFF_SEQ);
    PdMisc &ms = *reinterpret_cast<PdMisc *>(smem + C::OFF_MISC);
    static_assert(sizeof(PdMisc) <= 2048, "misc");
    const er_pages_attention_args &a = P.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int KV = P.p.KV, G = a.n_heads / KV, R = P.p.page_rows;
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BARS) + warp * PD_SLOTS;
    uint8_t *ring = smem + warp * C::RING;
    if (lane < PD_SLOTS) mbar_init(bars + lane, 1 + (blockIdx.x == 0 ? P.shortfall : 0));
    if (tid == 0) ms.wait_bad = 0;
    if (lane < 2) ms.seg[2 * warp + lane].off = -1;
    fence_mbar_init();

    // ---- the list: tiles of every sequence, prefix sums in W
    {
        constexpr int PER = (PD_SEQS + PD_THREADS - 1) / PD_THREADS;
        const int per = (a.n_seqs + PD_THREADS - 1) / PD_THREADS;
        long long own[PER], sum = 0;
#pragma unroll
        for (int k = 0; k < PER; ++k) {
            own[k] = 0;
            const int b = tid * per + k;
            if (k < per && b < a.n_seqs) {
                const int q0 = a.q_start_dev[b], q1 = a.q_start_dev[b + 1], len = a.lens_dev[b];
                int ns = 0;
                const bool bad = q0 < 0 || q1 < q0 || q1 > a.n_tokens || len < 0 ||
                                 len > pg_max_len(a.table_stride, R);
                if (bad) {
                    if (blockIdx.x == 0) atomicOr(P.p.flags, ER_PAGES_FLAG_RANGE);
                } else if ((long long)(q1 - q0) * G >= P.max_rows) {
                    ns = 0;
                } else if (q1 > q0 && len > 0) {
                    ns = (len - 1) / PD_STEP - pd_row0(len, q1 - q0, a.window) / PD_STEP + 1;
                    own[k] = (long long)ns * ((((long long)(q1 - q0) * G + PD_ROWS - 1) / PD_ROWS) * KV);
                } else if (q1 > q0) {
                    ns = -1;
                }
                SQ[b] = {q0, q1 - q0, len, ns};
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
        if (SQ[b].ns != -1) continue;
        const int q0 = SQ[b].q0;
        const long long n = (long long)SQ[b].qn * a.n_heads;
        for (long long i = tid; i < n * HD; i += PD_THREADS) {
            const int row = q0 + (int)(i / HD / a.n_heads), head = (int)(i / HD % a.n_heads);
            ((T *)a.out_dev)[row * a.out_stride + (size_t)head * HD + i % HD] = pg_cvt<T>(0.f);
        }
        if (a.lse_dev)
            for (long long i = tid; i < n; i += PD_THREADS) a.lse_dev[(size_t)q0 * a.n_heads + i] = -INFINITY;
    }
    const long long N = W[a.n_seqs];
    if (N == 0) return;
    const int C_ = (int)min((long long)gridDim.x, (N + PD_MIN_STEPS - 1) / PD_MIN_STEPS);
    if ((int)blockIdx.x >= C_) return;
    const long long c0 = pd_div(blockIdx.x * N, C_), c1 = pd_div((blockIdx.x + 1) * N, C_);
    const long long w0 = c0 + pd_div(warp * (c1 - c0), PD_WARPS), w1 = c0 + pd_div((warp + 1) * (c1 - c0), PD_WARPS);

    auto seq_of = [&](long long i) {  // the sequence of list entry i: the last b with W[b] <= i (empty ones are skipped)
        int lo = 0, hi = a.n_seqs - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (W[mid] <= i) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    };
    const int cnt = (int)(w1 - w0);  // this warp's steps
    struct Unit {
        long long u0, u1;
        int q0, qn, len, rg, h, b;
    };
    auto unit_at = [&](int k) {
        Unit u;
        u.b = seq_of(w0 + k);
        const PdSeq q = SQ[u.b];
        const long long unit = pd_div(w0 + k - W[u.b], q.ns);
        u.q0 = q.q0; u.qn = q.qn; u.len = q.len;
        u.u0 = W[u.b] + unit * q.ns;
        u.u1 = u.u0 + q.ns;
        u.rg = (int)pd_div(unit, KV);
        u.h = (int)(unit - (long long)u.rg * KV);
        return u;
    };
    // the lane's part of a unit's queries: column g, dims 32 bb + 8 t .. + 7, as they are
    const bool vec = ((uintptr_t)a.q_dev & 15) == 0 && (a.q_stride * sizeof(T)) % 16 == 0;
    __align__(16) T raw[C::NB][8];
    auto load_q = [&](const Unit &u) {
        int row, head, tok;
        pd_row(g, u.rg, G, u.q0, u.h, row, head, tok);
        const T *src = (const T *)a.q_dev + row * a.q_stride + (size_t)head * HD + 8 * t;
#pragma unroll
        for (int bb = 0; bb < C::NB; ++bb) {
            if (tok >= u.qn) {
#pragma unroll
                for (int e = 0; e < 8; ++e) raw[bb][e] = pg_cvt<T>(0.f);
            } else if (vec) {
#pragma unroll
                for (int k = 0; k < (int)(8 * sizeof(T)) / 16; ++k)
                    reinterpret_cast<uint4 *>(raw[bb])[k] = reinterpret_cast<const uint4 *>(src + 32 * bb)[k];
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) raw[bb][e] = src[32 * bb + e];
            }
        }
    };
    Unit U;
    if (cnt > 0) {
        U = unit_at(0);
        load_q(U);
    }
    // where the two tiles of step k lie, as tile numbers of the pool (it holds fewer than 2^32); ABSENT: one that lies
    // outside the rows that the unit attends
    constexpr uint32_t ABSENT = 0xFFFFFFFFu;
    auto source = [&](int k, uint32_t &x0, uint32_t &x1) {
        x0 = x1 = ABSENT;
        if (k >= cnt) return;
        const int b = seq_of(w0 + k);
        const PdSeq q = SQ[b];
        const long long rem = w0 + k - W[b], unit = pd_div(rem, q.ns);
        const int lo = pd_row0(q.len, q.qn, a.window), h = (int)(unit - pd_div(unit, KV) * KV);
        const int row = (lo / PD_STEP + (int)(rem - unit * q.ns)) * PD_STEP;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int rn = row + 16 * n;
            if (rn >= q.len || rn + 15 < lo) continue;
            const int blk = (int)((uint32_t)rn / (uint32_t)R);
            int page = a.tables_dev[(size_t)b * a.table_stride + blk];
            if (page < 0 || page >= P.p.n_pages) {
                atomicOr(P.p.flags, ER_PAGES_FLAG_RANGE);
                page = 0;
            }
            (n ? x1 : x0) = ((uint32_t)page * KV + h) * (R >> 4) + ((rn - blk * R) >> 4);
        }
    };
    // the 32 steps among which the next one to request lies are in cur, a lane each, the 32 after them in nxt
    int inext = 0, islot = 0;
    uint32_t cur0, cur1, nxt0 = 0, nxt1 = 0;
    source(lane, cur0, cur1);
    auto issue = [&]() {  // requests the next step: the lane that knows where it lies
        if (inext >= cnt) return;
        if ((inext & 31) == 0) {
            if (inext) {
                cur0 = nxt0;
                cur1 = nxt1;
            }
            source((inext | 31) + 1 + lane, nxt0, nxt1);
        }
        if (lane == (inext & 31)) {
            uint8_t *dst = ring + islot * (2 * C::TILE);
            mbar_arrive_expect_tx(bars + islot, (cur0 != ABSENT ? C::TILE : 0) + (cur1 != ABSENT ? C::TILE : 0));
            if (cur0 != ABSENT) bulk_g2s(dst, P.p.pool + (size_t)cur0 * C::TILE, C::TILE, bars + islot);
            if (cur1 != ABSENT) bulk_g2s(dst + C::TILE, P.p.pool + (size_t)cur1 * C::TILE, C::TILE, bars + islot);
        }
        ++inext;
        if (++islot == PD_SLOTS) islot = 0;
    };
#pragma unroll 1
    for (int k = 0; k < PD_SLOTS; ++k) issue();

    const float qscale = (a.scale != 0.f ? a.scale : 1.f / sqrtf((float)HD)) * 1.4426950408889634f;
    int wslot = 0;     // ring slot and parity of the next step to consume
    uint32_t wpar = 0;
    bool bad = false;  // a wait gave up

    for (int k0 = 0; k0 < cnt;) {
        // rows that the lane's columns 2 t, 2 t + 1 attend, and the ranges that all and any of the unit's rows attend
        const int past = U.len - U.qn;
        const int tok0 = U.rg * PD_ROWS / G, tok1 = min((U.rg * PD_ROWS + PD_ROWS - 1) / G, U.qn - 1);
        int pos[2], first[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int tok = (U.rg * PD_ROWS + 2 * t + c) / G;
            pos[c] = tok < U.qn ? past + tok : -1;
            first[c] = pg_first(pos[c], a.window);
        }
        // Values that are NaN: a step that only some of the unit's rows attend carries them by its scores instead, and its values
        // with them are 0.  `carry`, `carried`: the largest magnitude of a scale that is left to the values, of the steps
        // whose scores are next and whose values are (infinity's, or NaN's where nothing is carried: one token, or scores that
        // were not masked).
        constexpr uint32_t NEVER = 0x7FFFu;
        const uint32_t carry = tok0 < tok1 ? 0x7C00u : NEVER;
        uint32_t carried = carry;
        const int any_lo = pg_first(past + tok0, a.window), any_hi = past + tok1;
        const int all_lo = pg_first(past + tok1, a.window), all_hi = past + tok0;

        // the queries as B: k16 steps 2 bb + i, the lane's dims 32 bb + 8 t + 4 i .. + 3 of column g
        uint32_t qh[2 * C::NB][2];
        [[maybe_unused]] uint32_t ql[2 * C::NB][2];
        float down[2];
        {
            float top = 0.f;
            bool odd = false;  // infinite and NaN queries: their scores are NaN through `down`
#pragma unroll
            for (int bb = 0; bb < C::NB; ++bb)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x = fabsf(pg_ld<T>(&raw[bb][e]));
                    top = fmaxf(top, x);
                    odd |= !(x <= 3.4028235e38f);
                }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            odd = __ballot_sync(0xffffffffu, odd) >> (lane & ~3) & 15;
            // a power of two, up, brings the row's largest to [2^14, 2^15): its lo halves are normal, and of a 16-bit row
            // the values down to 2^-31 of that are exact
            const int ex = min(max((int)(__float_as_uint(top) >> 23), 15), 253);
            const float up = odd ? 0.f : __uint_as_float((uint32_t)(268 - ex) << 23);
            const float dn = odd ? NAN : __uint_as_float((uint32_t)(ex - 14) << 23);
#pragma unroll
            for (int bb = 0; bb < C::NB; ++bb) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x0 = odd ? 0.f : pg_ld<T>(&raw[bb][2 * i]) * up, x1 = odd ? 0.f : pg_ld<T>(&raw[bb][2 * i + 1]) * up;
                    if constexpr (Y::QLO) {
                        pd_split(x0, x1, qh[2 * bb + (i >> 1)][i & 1], ql[2 * bb + (i >> 1)][i & 1]);
                    } else {
                        qh[2 * bb + (i >> 1)][i & 1] = pg_pack(x0, x1);
                    }
                }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) down[c] = __shfl_sync(0xffffffffu, dn, 4 * (2 * t + c)) * qscale;
        }
        float m[2] = {PD_NONE, PD_NONE}, l[2] = {0.f, 0.f};
        float o[HD / 16][4];  // dims 16 j + g (0, 1) and + 8 (2, 3) of columns 2 t, 2 t + 1
#pragma unroll
        for (int j = 0; j < HD / 16; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

        // A step (rows r0 .. r0 + 31, in the ring at sl) is three parts: its scores, its probabilities, its products with V.
        // EDGE: some row of the unit may not attend all of them.
        // Scores: rows r0 + 16 n + g (x[n][0], x[n][1]) and + 8 (x[n][2], x[n][3]) of columns 2 t, 2 t + 1.
        auto scores = [&](auto edge_tag, const uint8_t *sl, int r0, float (&x)[2][4]) {
            constexpr bool EDGE = decltype(edge_tag)::value;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const uint8_t *sn = sl + n * C::TILE;
                uint32_t kw[2][C::NB], ks[2][C::NB / 2];
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const int rr = 8 * v + g;
                    if constexpr (HD == 128) {
                        const uint4 y = *reinterpret_cast<const uint4 *>(sn + rr * 64 + t * 16);
                        kw[v][0] = y.x; kw[v][1] = y.y; kw[v][2] = y.z; kw[v][3] = y.w;
                        const uint2 z = *reinterpret_cast<const uint2 *>(sn + pg_off_ks(HD) + rr * 8);
                        ks[v][0] = z.x; ks[v][1] = z.y;
                    } else {
                        const uint2 y = *reinterpret_cast<const uint2 *>(sn + rr * 32 + t * 8);
                        kw[v][0] = y.x; kw[v][1] = y.y;
                        ks[v][0] = *reinterpret_cast<const uint32_t *>(sn + pg_off_ks(HD) + rr * 4);
                    }
                }
                float sc[4] = {0.f, 0.f, 0.f, 0.f};
                if constexpr (Y::RAW) {
#pragma unroll
                    for (int bb = 0; bb < C::NB; ++bb) {
                        const uint32_t w0 = kw[0][bb], w1 = kw[1][bb], u0 = w0 >> 8, u1 = w1 >> 8;
                        const uint32_t a0[4] = {pd_low(w0), pd_low(w1), pd_high(w0), pd_high(w1)};
                        const uint32_t a1[4] = {pd_low(u0), pd_low(u1), pd_high(u0), pd_high(u1)};
                        const float2 e0 = __half22float2(*reinterpret_cast<const __half2 *>(&ks[0][bb >> 1]));
                        const float2 e1 = __half22float2(*reinterpret_cast<const __half2 *>(&ks[1][bb >> 1]));
                        const float d0 = (bb & 1) ? e0.y : e0.x, d1 = (bb & 1) ? e1.y : e1.x;
                        float acc[4];
                        const float none[4] = {0.f, 0.f, 0.f, 0.f};
                        pd_mma_c(acc, a0, qh[2 * bb][0], qh[2 * bb][1], none);
                        pd_mma(acc, a1, qh[2 * bb + 1][0], qh[2 * bb + 1][1]);
                        sc[0] = fmaf(d0, acc[0], sc[0]); sc[1] = fmaf(d0, acc[1], sc[1]);
                        sc[2] = fmaf(d1, acc[2], sc[2]); sc[3] = fmaf(d1, acc[3], sc[3]);
                    }
                } else {
                    float part[4] = {0.f, 0.f, 0.f, 0.f};  // a second chain of products
#pragma unroll
                    for (int bb = 0; bb < C::NB; ++bb) {
                        const uint32_t w0 = kw[0][bb], w1 = kw[1][bb];
                        const uint32_t d0 = prmt(ks[0][bb >> 1], 0u, (bb & 1) ? 0x3232u : 0x1010u), z0 = pg_m24(d0);
                        const uint32_t d1 = prmt(ks[1][bb >> 1], 0u, (bb & 1) ? 0x3232u : 0x1010u), z1 = pg_m24(d1);
                        const uint32_t a0[4] = {h2_fma(pg_code<0>(w0), d0, z0), h2_fma(pg_code<0>(w1), d1, z1),
                                                h2_fma(pg_code<1>(w0), d0, z0), h2_fma(pg_code<1>(w1), d1, z1)};
                        const uint32_t a1[4] = {h2_fma(pg_code<2>(w0), d0, z0), h2_fma(pg_code<2>(w1), d1, z1),
                                                h2_fma(pg_code<3>(w0), d0, z0), h2_fma(pg_code<3>(w1), d1, z1)};
                        pd_mma(sc, a0, qh[2 * bb][0], qh[2 * bb][1]);
                        pd_mma(part, a1, qh[2 * bb + 1][0], qh[2 * bb + 1][1]);
                        if constexpr (Y::QLO) {
                            pd_mma(sc, a0, ql[2 * bb][0], ql[2 * bb][1]);
                            pd_mma(part, a1, ql[2 * bb + 1][0], ql[2 * bb + 1][1]);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) sc[k] += part[k];
                }
                if constexpr (EDGE) {
                    bool vnan[2] = {false, false};  // rows g, g + 8 hold a NaN value: their scores carry it
                    const unsigned short *vs = reinterpret_cast<const unsigned short *>(sn + pg_off_vs(HD));
#pragma unroll
                    for (int bb = 0; bb < C::NB; ++bb)
#pragma unroll
                        for (int v = 0; v < 2; ++v)
                            vnan[v] |= (vs[(((g >> 1) * C::NB + bb) * 2 + v) * 2 + (g & 1)] & 0x7FFF) > carry;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int r = r0 + 16 * n + g + 8 * (k >> 1);
                        if (vnan[k >> 1]) sc[k] = NAN;
                        x[n][k] = r < first[k & 1] || r > pos[k & 1] ? -INFINITY : sc[k] * down[k & 1];
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[n][k] = sc[k] * down[k & 1];
                }
            }
        };
        uint32_t ph[2][2];  // B of P: rows 16 n + 8 v .. + 7
        uint32_t pl[2][2];
        auto reference = [&](const float (&x)[2][4]) {
            // a score far above the reference: a new one for the column, and the sums follow
            const float t0 = fmaxf(fmaxf(x[0][0], x[0][2]), fmaxf(x[1][0], x[1][2]));
            const float t1 = fmaxf(fmaxf(x[0][1], x[0][3]), fmaxf(x[1][1], x[1][3]));
            if (__any_sync(0xffffffffu, t0 > m[0] + PD_SLACK || t1 > m[1] + PD_SLACK)) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float mt = c ? t1 : t0;
#pragma unroll
                    for (int off = 4; off < 32; off <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, off));
                    const float mn = mt > m[c] + PD_SLACK ? mt : m[c];
                    const float corr = mn == m[c] ? 1.f : pg_ex2(m[c] - mn);
                    l[c] *= corr;
#pragma unroll
                    for (int j = 0; j < HD / 16; ++j) {
                        o[j][c] *= corr;
                        o[j][2 + c] *= corr;
                    }
                    m[c] = mn;
                }
            }
        };
        auto probabilities = [&](const float (&x)[2][4]) {
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                float p[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) p[k] = pg_ex2(x[n][k] - (m[k & 1] - PD_UP));
                l[0] += p[0] + p[2];
                l[1] += p[1] + p[3];
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    pd_split(p[2 * v], p[2 * v + 1], ph[n][v], pl[n][v]);
                    ph[n][v] = pd_trans(ph[n][v]);
                    pl[n][v] = pd_trans(pl[n][v]);
                }
            }
        };
        // o += p v.  fp32: a tile's products are summed from 0 and added to o rounded to nearest: the tensor cores' sums
        // truncate, and over thousands of rows that shows.
        auto values = [&](auto edge_tag, const uint8_t *sl, int r0) {
            constexpr bool EDGE = decltype(edge_tag)::value;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const uint8_t *sn = sl + n * C::TILE;
                // V scales of rows 2t, 2t + 1 (vd[.][0]) and 2t + 8, 2t + 9 (vd[.][1]), a pair a word
                uint32_t vw[HD / 64][4], vd[C::NB][2];
#pragma unroll
                for (int k = 0; k < C::NB / 2; ++k) {
                    const uint4 y = *reinterpret_cast<const uint4 *>(sn + pg_off_vs(HD) + t * (C::NB * 8) + 16 * k);
                    vd[2 * k][0] = y.x; vd[2 * k][1] = y.y; vd[2 * k + 1][0] = y.z; vd[2 * k + 1][1] = y.w;
                }
#pragma unroll
                for (int q = 0; q < HD / 64; ++q) {
                    const uint4 y = *reinterpret_cast<const uint4 *>(sn + pg_off_v(HD) + q * 512 + lane * 16);
                    vw[q][0] = y.x; vw[q][1] = y.y; vw[q][2] = y.z; vw[q][3] = y.w;
                }
                if constexpr (EDGE) {  // scales of rows that nobody attends, or that are NaN and carried by the scores: 0
#pragma unroll
                    for (int bb = 0; bb < C::NB; ++bb)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int r = r0 + 16 * n + 2 * t + (k & 1) + 8 * (k >> 1);
                            const uint32_t half = (k & 1) ? 0xFFFF0000u : 0x0000FFFFu;
                            const uint32_t above = (k & 1) ? carried << 16 | 0xFFFFu : carried;
                            if ((vd[bb][k >> 1] & half & 0x7FFF7FFFu) > above || r < any_lo || r > any_hi)
                                vd[bb][k >> 1] &= ~half;
                        }
                }
#pragma unroll
                for (int bb = 0; bb < C::NB; ++bb) {
                    const uint32_t d0 = vd[bb][0], d1 = vd[bb][1], z0 = pg_m24(d0), z1 = pg_m24(d1);
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const uint32_t w = vw[bb >> 1][2 * (bb & 1) + u];
                        const uint32_t va[4] = {h2_fma(pg_code<0>(w), d0, z0), h2_fma(pg_code<1>(w), d0, z0),
                                                h2_fma(pg_code<2>(w), d1, z1), h2_fma(pg_code<3>(w), d1, z1)};
                        if constexpr (Y::QLO) {
                            float sum[4] = {0.f, 0.f, 0.f, 0.f};
                            pd_mma(sum, va, ph[n][0], ph[n][1]);
                            pd_mma(sum, va, pl[n][0], pl[n][1]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) o[2 * bb + u][e] += sum[e];
                        } else {
                            pd_mma(o[2 * bb + u], va, ph[n][0], ph[n][1]);
                            pd_mma(o[2 * bb + u], va, pl[n][0], pl[n][1]);
                        }
                    }
                }
            }
        };

        const int kend = (int)(min(U.u1, w1) - w0);  // the segment: steps k0 .. kend - 1
        int r0 = (pd_row0(U.len, U.qn, a.window) / PD_STEP + (int)(w0 + k0 - U.u0)) * PD_STEP;
        // Software pipeline: a step's products with V and the next one's scores stand in one piece of code, so that two
        // chains of conversions and products are in flight in a warp (there are only two warps a scheduler).
        auto arrived = [&]() {  // the step at wslot, wpar
            if (__all_sync(0xffffffffu, mbar_wait(bars + wslot, wpar))) return true;
            bad = true;
            return false;
        };
        auto plain = [&](int r) { return r >= all_lo && r + PD_STEP - 1 <= all_hi; };
        float x[2][4];
        const uint8_t *sl = ring + wslot * (2 * C::TILE);
        if (arrived()) {
            scores(std::true_type{}, sl, r0, x);
            for (int k = k0;; ++k) {
                const bool more = k + 1 < kend;
                const uint8_t *here = sl;
                if (++wslot == PD_SLOTS) {
                    wslot = 0;
                    wpar ^= 1u;
                }
                if (more) {
                    sl = ring + wslot * (2 * C::TILE);
                    if (!arrived()) break;
                }
                reference(x);
                probabilities(x);
                if (more && plain(r0) && plain(r0 + PD_STEP)) {
                    values(std::false_type{}, here, r0);
                    scores(std::false_type{}, sl, r0 + PD_STEP, x);
                    carried = NEVER;
                } else {
                    values(std::true_type{}, here, r0);
                    if (more) scores(std::true_type{}, sl, r0 + PD_STEP, x);
                    carried = carry;
                }
                __syncwarp();  // every lane has read the slot
                issue();
                r0 += PD_STEP;
                if (!more) break;
            }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], off);
        if (bad) break;
        const bool whole = U.u0 >= w0 + k0 && U.u1 <= w1;
        const Unit D = U;  // done
        if (kend < cnt) {  // the next unit's queries, while this one's results are written
            U = unit_at(kend);
            load_q(U);
        }
        k0 = kend;
        if (whole) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                int row, head, tok;
                pd_row(2 * t + c, D.rg, G, D.q0, D.h, row, head, tok);
                if (tok >= D.qn) continue;
                const float inv = 1.f / l[c];
                T *out = (T *)a.out_dev + row * a.out_stride + (size_t)head * HD + g;
#pragma unroll
                for (int j = 0; j < HD / 16; ++j) {
                    out[16 * j] = pg_cvt<T>(l[c] == 0.f ? 0.f : o[j][c] * inv);
                    out[16 * j + 8] = pg_cvt<T>(l[c] == 0.f ? 0.f : o[j][2 + c] * inv);
                }
                if (a.lse_dev && g == 0)
                    a.lse_dev[(size_t)row * a.n_heads + head] =
                        l[c] == 0.f ? -INFINITY : (m[c] - PD_UP + log2f(l[c])) * 0.6931471805599453f;
            }
        } else {
            // a state: the last segment's goes into the ring (nothing is on its way there any more)
            const int off = kend == cnt ? warp * C::RING : C::OFF_FIRST + warp * C::STATE * 4;
            float *st = reinterpret_cast<float *>(smem + off);
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int j = 0; j < HD / 16; ++j) {
                    st[(2 * t + c) * HD + 16 * j + g] = o[j][c];
                    st[(2 * t + c) * HD + 16 * j + g + 8] = o[j][2 + c];
                }
                if (g == 0) {
                    st[PD_ROWS * HD + 2 * t + c] = m[c];
                    st[PD_ROWS * HD + 8 + 2 * t + c] = l[c];
                }
            }
            if (lane == 0) ms.seg[2 * warp + (kend == cnt)] = {D.u0, D.u1, D.b, D.rg, D.h, off};
        }
    }
    if (bad) {
        if (lane == 0) atomicOr(P.p.flags, ER_FLAG_WAIT);
        ms.wait_bad = 1;
        // copies may still be landing; an injected shortfall's arrivals are made up for, so that the barriers tell
        if (blockIdx.x == 0 && lane < PD_SLOTS)
            for (int k = 0; k < P.shortfall; ++k) mbar_arrive(bars + lane);
        __syncwarp();
        for (int k = max(0, inext - PD_SLOTS); k < inext; ++k) pg_drain(bars + k % PD_SLOTS, (k / PD_SLOTS) & 1);
    }
    __syncthreads();
    if (warp == 0) {  // runs of neighbouring states of one unit; lane e looks at the e-th place for one
        static_assert(2 * PD_WARPS <= 32, "a lane for each state");
        const bool there = lane < 2 * PD_WARPS && ms.seg[lane].off >= 0;
        const unsigned all = __ballot_sync(0xffffffffu, there);
        const int before = 31 - __clz((int)(all & ((1u << lane) - 1u)));  // the state before this one, or -1
        const bool starts = there && (before < 0 || ms.seg[before].u0 != ms.seg[lane].u0);
        const unsigned runs = __ballot_sync(0xffffffffu, starts);
        if (there) ms.ent[__popc(all & ((1u << lane) - 1u))] = (short)lane;
        if (starts) ms.run[__popc(runs & ((1u << lane) - 1u))] = __popc(all & ((1u << lane) - 1u));
        if (lane == 0) {
            ms.run[__popc(runs)] = __popc(all);
            ms.n_runs = ms.wait_bad ? 0 : __popc(runs);
        }
    }
    __syncthreads();
    const int n_runs = ms.n_runs;
    constexpr int V = HD / 32;  // dims of a lane
    // a row of a unit, joined: o of dims V lane .. , the reference m and sum l
    auto write_row = [&](const PdSeg &sg, int r, const float (&y)[V], float mm, float ll) {
        int row, head, tok;
        pd_row(r, sg.rg, G, SQ[sg.b].q0, sg.h, row, head, tok);
        if (tok >= SQ[sg.b].qn) return;
        T *out = (T *)a.out_dev + row * a.out_stride + (size_t)head * HD + V * lane;
#pragma unroll
        for (int e = 0; e < V; ++e) out[e] = pg_cvt<T>(ll == 0.f ? 0.f : y[e] / ll);
        if (a.lse_dev && lane == 0)
            a.lse_dev[(size_t)row * a.n_heads + head] =
                ll == 0.f ? -INFINITY : (mm - PD_UP + log2f(ll)) * 0.6931471805599453f;
    };
    // real rows of a unit
    auto rows_of = [&](const PdSeg &sg) {
        return (int)min((long long)PD_ROWS, (long long)SQ[sg.b].qn * G - (long long)sg.rg * PD_ROWS);
    };
    for (int it = warp; it < n_runs * PD_ROWS; it += PD_WARPS) {
        const int run = it / PD_ROWS, r = it % PD_ROWS;
        const int e0 = ms.run[run], ne = ms.run[run + 1] - e0;
        const PdSeg &sg = ms.seg[ms.ent[e0]];
        if (r >= rows_of(sg)) continue;
        // lane e: the weight of the run's e-th state
        const int off = lane < ne ? ms.seg[ms.ent[e0 + lane]].off : 0;
        const float *mine = reinterpret_cast<const float *>(smem + off);
        float M = lane < ne ? mine[PD_ROWS * HD + r] : PD_NONE;
        const float own = M;
#pragma unroll
        for (int x = 16; x; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
        const float f = lane < ne ? pg_ex2(own - M) : 0.f;
        float L = lane < ne ? f * mine[PD_ROWS * HD + 8 + r] : 0.f;
#pragma unroll
        for (int x = 16; x; x >>= 1) L += __shfl_xor_sync(0xffffffffu, L, x);
        float y[V];
#pragma unroll
        for (int e = 0; e < V; ++e) y[e] = 0.f;
#pragma unroll 4
        for (int e = 0; e < ne; ++e) {
            const float fe = __shfl_sync(0xffffffffu, f, e);
            const float *st = reinterpret_cast<const float *>(smem + __shfl_sync(0xffffffffu, off, e));
#pragma unroll
            for (int k = 0; k < V; ++k) y[k] += fe * st[r * HD + V * lane + k];
        }
        if (sg.u0 >= c0 && sg.u1 <= c1) {
            write_row(sg, r, y, M, L);
        } else {
            float *st = P.part + ((size_t)blockIdx.x * 2 + (sg.u0 < c0 ? 0 : 1)) * C::STATE;
            if constexpr (V == 4) __stcg(reinterpret_cast<float4 *>(st + r * HD) + lane, make_float4(y[0], y[1], y[2], y[V - 1]));
            else __stcg(reinterpret_cast<float2 *>(st + r * HD) + lane, make_float2(y[0], y[1]));
            if (lane == 0) {
                __stcg(st + PD_ROWS * HD + r, M);
                __stcg(st + PD_ROWS * HD + 8 + r, L);
            }
        }
    }
    // ---- units of several CTAs: the last to arrive joins their states in CTA order
    __threadfence();
    __syncthreads();
    if (tid < 2) ms.last[tid] = -1;
    __syncwarp();
    if (tid < n_runs) {  // at most 2 * PD_WARPS runs; two of them reach into other CTAs
        const PdSeg &sg = ms.seg[ms.ent[ms.run[tid]]];
        if (sg.u0 < c0 || sg.u1 > c1) {
            const int ca = pd_cta(sg.u0, N, C_), cb = pd_cta(sg.u1 - 1, N, C_);
            if (atom_add_acq_rel_gpu(P.cnt + ca, 1) == cb - ca) {
                P.cnt[ca] = 0;
                ms.last[sg.u0 < c0 ? 0 : 1] = tid;
            }
        }
    }
    __syncthreads();
    float *acc = reinterpret_cast<float *>(smem + C::OFF_FIRST);  // [warps][HD + 4], where the first states were
    for (int k = 0; k < 2; ++k) {
        if (ms.last[k] < 0) continue;
        const PdSeg sg = ms.seg[ms.ent[ms.run[ms.last[k]]]];
        const int ca = pd_cta(sg.u0, N, C_), nc = pd_cta(sg.u1 - 1, N, C_) - ca + 1, rows = rows_of(sg);
        // the unit's state of its c-th CTA: the first one's second place (the unit starts there), the others' first
        auto state = [&](int c) { return P.part + (size_t)((ca + c) * 2 + (c == 0)) * C::STATE; };
        // warp (r, part): row r, the CTAs part, part + parts, ...
        const int parts = max(1, PD_WARPS / rows), r = warp / parts, part = warp - r * parts;
        float M = PD_NONE, L = 0.f, y[V];
#pragma unroll
        for (int e = 0; e < V; ++e) y[e] = 0.f;
        if (r < rows) {
            for (int c = lane; c < nc; c += 32) M = fmaxf(M, __ldcg(state(c) + PD_ROWS * HD + r));
#pragma unroll
            for (int x = 16; x; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
            // 4 states' loads at a time (8 are more code, read from memory by every launch: 0.3 us more)
            for (int c0_ = part; c0_ < nc; c0_ += 4 * parts) {
                float f[4], ll[4], z[4][V];
#pragma unroll
                for (int k2 = 0; k2 < 4; ++k2) {
                    const int c = min(c0_ + k2 * parts, nc - 1);
                    const float *st = state(c);
                    f[k2] = __ldcg(st + PD_ROWS * HD + r);
                    ll[k2] = __ldcg(st + PD_ROWS * HD + 8 + r);
                    if constexpr (V == 4) {
                        const float4 q = __ldcg(reinterpret_cast<const float4 *>(st + r * HD) + lane);
                        z[k2][0] = q.x; z[k2][1] = q.y; z[k2][2] = q.z; z[k2][V - 1] = q.w;
                    } else {
                        const float2 q = __ldcg(reinterpret_cast<const float2 *>(st + r * HD) + lane);
                        z[k2][0] = q.x; z[k2][1] = q.y;
                    }
                }
#pragma unroll
                for (int k2 = 0; k2 < 4; ++k2) {
                    const float w = c0_ + k2 * parts < nc ? pg_ex2(f[k2] - M) : 0.f;
                    if (c0_ + k2 * parts < nc) {
                        L += w * ll[k2];
#pragma unroll
                        for (int e = 0; e < V; ++e) y[e] += w * z[k2][e];
                    }
                }
            }
        }
        if (parts > 1) {
            __syncthreads();  // the place is free: the states in it, or the other unit's sums, are read
#pragma unroll
            for (int e = 0; e < V; ++e) acc[warp * (HD + 4) + V * lane + e] = y[e];
            if (lane == 0) acc[warp * (HD + 4) + HD] = L;
            __syncthreads();
            if (part == 0 && r < rows)
                for (int x = 1; x < parts; ++x) {
                    L += acc[(warp + x) * (HD + 4) + HD];
#pragma unroll
                    for (int e = 0; e < V; ++e) y[e] += acc[(warp + x) * (HD + 4) + V * lane + e];
                }
        }
        if (part == 0 && r < rows) write_row(sg, r, y, M, L);
    }
}

size_t pages_attn_part_floats(int num_sms) { return (size_t)num_sms * 2 * (PD_ROWS * 128 + 16); }

template <class T, int HD>
static cudaError_t decode_prepare() {
    return cudaFuncSetAttribute(pages_decode_kernel<T, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, PdCfg<T, HD>::SMEM);
}
cudaError_t pages_attn_prepare() {
    if (cudaError_t e = pages_prompt_prepare(); e != cudaSuccess) return e;
    cudaError_t e[6] = {decode_prepare<float, 64>(), decode_prepare<float, 128>(), decode_prepare<__half, 64>(),
                        decode_prepare<__half, 128>(), decode_prepare<__nv_bfloat16, 64>(),
                        decode_prepare<__nv_bfloat16, 128>()};
    for (cudaError_t x : e)
        if (x != cudaSuccess) return x;
    return cudaSuccess;
}

template <class T>
static cudaError_t decode_t(const PdArgs &P, int num_sms, cudaStream_t st) {
    if (P.p.hd == 128) pages_decode_kernel<T, 128><<<num_sms, PdCfg<T, 128>::THREADS, PdCfg<T, 128>::SMEM, st>>>(P);
    else pages_decode_kernel<T, 64><<<num_sms, PdCfg<T, 64>::THREADS, PdCfg<T, 64>::SMEM, st>>>(P);
    return cudaGetLastError();
}

// From this many query rows of a KV head on, several tokens of a sequence go to the prompt kernel.  Its CTA takes as long for 16
// rows as for 128 and walks all of a sequence's rows by itself; this file's kernel takes rows in eights and spreads them over
// the SMs.  us, bf16, 32 / 8 heads of 128, 16 / 32 / 64 / 128 / 256 query rows of each of 8 sequences over 4096 rows: here
// 33 / 49 / 82 / 147 / 277, there 81 / 82 / 82 / 83 / 87; fp32 38 / 61 / 108 / 201 / 381 and 70 / 70 / 71 / 71 / 71; bf16
// heads of 64: 25 / 35 / 58 / 101 / 187 and 63 / 64 / 64 / 66 / 75.  So 64 is the crossing where prompts fill the SMs.
// One sequence alone crosses later, near 512 rows (bf16, 4096 rows: 19 / 23 / 26 / 33 / 49, at 512 82, against 79 to 83; fp32 21
// / 23 / 27 / 38 / 61, at 512 108, against 70): which kernel is the faster there depends on the whole call, which no rule here
// looks at.  A single token with all heads on one K/V head is 64 rows and always this kernel's: 64 / 1 heads of 128, bf16,
// 512 / 4096 / 32768 rows, 13 / 15 / 23 us here, 21 / 80 / 555 there.
constexpr int PD_PROMPT_ROWS = 64;

cudaError_t launch_pages_attention(const PagesView &p, const er_pages_attention_args &a, float *part, int *cnt,
                                   int shortfall, int num_sms, cudaStream_t st) {
    // The lengths are on the device, so the split is made there, sequence by sequence.  Here: too few rows for any prompt, or a
    // step of at most as many tokens as sequences, taken for a decode step, which stays one launch.  (A prompt among that
    // many idle sequences is worked by the kernel of few rows too: right, but slower the longer it is.)
    const int G = a.n_heads / p.KV, from = PD_PROMPT_ROWS > G ? PD_PROMPT_ROWS : G + 1;  // (G rows are a single token)
    const bool prompts = (long long)a.n_tokens * G >= from && a.n_tokens > a.n_seqs;
    if (prompts)
        if (cudaError_t e = launch_pages_prompt(p, a, from, shortfall, st); e != cudaSuccess) return e;
    for (int b = 0; b < a.n_seqs; b += PD_SEQS) {
        PdArgs P = {p, a, prompts ? from : 2147483647, part, cnt, shortfall};
        P.a.n_seqs = a.n_seqs - b < PD_SEQS ? a.n_seqs - b : PD_SEQS;
        P.a.q_start_dev += b;
        P.a.lens_dev += b;
        P.a.tables_dev += (size_t)b * a.table_stride;
        const cudaError_t e = a.type == ER_F32   ? decode_t<float>(P, num_sms, st)
                              : a.type == ER_F16 ? decode_t<__half>(P, num_sms, st)
                                                 : decode_t<__nv_bfloat16>(P, num_sms, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

cudaError_t set_wait_limit_pages(unsigned long long ns) { return set_wait_limit_here(ns); }

}  // namespace er
