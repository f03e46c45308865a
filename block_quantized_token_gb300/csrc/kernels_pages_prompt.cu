// Attention over the paged 4-bit K/V cache (pages.cuh) for prompts: many query rows a sequence, on the tcgen05
// tensor cores.  o = softmax(scale q k^T) v with a running reference m and sums, as in kernels_pages_attn.cu:
//   p_r = 2^(s_r - m + 7),  l = sum p_r,  o = sum p_r v_r   (s in log2 units; rescaled when a score passes m by 8).
//
// Work.  A CTA takes one (sequence, KV head) and some query rows (a row is a (token, head of the KV head's group), so
// a group's heads share the cached rows), and walks the cached rows in blocks of 128.
//   16-bit rows (pages_prompt_kernel): two tiles of 128 query rows.
//     warps 0-3, 4-7  a tile's softmax: thread = row = TMEM lane.  Reads S, writes P over it (hi and lo fp16 halves, 2^-22:
//                     A operands of the second product), keeps m and l, rescales O when it has to, writes the output.
//     warp 12         one thread issues the products: S = Q K^T (M = 128, N = 128), O += P V (N = HD, hi and lo of P), the
//                     two tiles in turn, so the tensor cores work on one tile while the other's softmax runs.
//     TMEM: S/P of both tiles (2 x 128 columns), O of both (2 x HD).
//   P as one half (2^-11) would be 434 us for 8192 bf16 tokens against 557, but then a bf16 output in twenty differs by its
//   last bit from what exact probabilities give, and an fp16 output is off by as much again as its own rounding.
//   fp32 rows (pages_prompt32_kernel): one tile; queries enter as hi + lo halves too, two products each.  The tensor cores'
//   sums truncate (over thousands of rows 2^-18 of the output and growing), so a block's O starts from 0 and is added to
//   sums in registers, rounded to nearest.
//     warps 0-3, 4-7  two threads a row, one for either half of the columns of S and of O: softmax, as above, with the
//                     row's largest score exchanged through shared memory; then o = o * factor + the last block's O.
//                     (One thread a row is bound by its own latency: 212 us against 167 for 4 x 500 tokens.  For 16-bit
//                     rows, where two tiles take turns, two threads a row cost more than they gave: 546 us against 492
//                     for 8192 tokens.)
//     warp 12         S of the block after next goes to the buffer whose P is used up, so the softmax never waits for it
//     TMEM: two buffers of S/P, two of a block's O.
//   Both: warps 8-11 turn codes into fp16 operands in shared memory, exactly (pages.cuh), K and V K-major with the
//   128-byte swizzle, two stages each; warp 13 requests the cached tiles: bulk copies into a ring of three half blocks, each
//   used by two operand warps (ring.h).
//
// Registers (the launch's 128 a thread, shared out anew: 2 softmax + operands + rest = 512).  A spill in any role delays the
// others.  16 bits: 208, 48, 48 (8 bytes spilled at HD = 128; 8192 bf16 tokens: 552 us in the build that had these figures; 200, 56, 56: 585; 200, 64, 48: 588).
// fp32: 200, 64, 48 (8 bytes; 4 x 500 tokens: 135 us; 200, 80, 32: 138).
//
// The block's rows are put in the order k' = 32 a + 8 t + 4 b + 2 i + e for row 32 a + 16 b + 8 i + 2 t + e, in K's rows,
// hence S's and P's columns, and in V's K dimension: so a thread that holds a code word of V of two 16-row tiles
// holds 16 bytes of the operand.
//
// What bounds it: at HD = 128 a block and two tiles take the tensor cores six products of 512 cycles (one tile of fp32
// four), shared memory 2560 (the products' reads, the operands' writes), and about 4000 in all with the softmax and
// its hand-overs (4770 of the whole launch's, the ways in and out and the last, uneven CTAs among them).
// Measured: 8192 bf16 tokens, 32 / 8 heads of 128: 557 us = 0.99 PFLOP/s, 0.52 of the library's matrix product (with the lo
// halves' product counted 0.77); 4 x 300..500 fp32 tokens over 900..4100 rows: 135 us.
//
// Masks.  Blocks that some row attends only in part mask S; there, rows of V that no row of the CTA attends are
// zeroed (they may hold anything), and a NaN value of V is carried by K instead, so only rows that attend it see it.
#include <type_traits>

#include "pages.cuh"
#include "pages.h"
#include "ring.h"

namespace er {

constexpr int PP_WARPS = 16;  // 0-3, 4-7 softmax, 8-11 operands, 12 products, 13 copies (14, 15 only give registers)
constexpr int PP_THREADS = PP_WARPS * 32;
constexpr int PP_BLOCK = 128;  // cached rows of a block
constexpr int PP_RAW = 3;      // half blocks (four 16-row tiles) in the ring
constexpr float PP_UP = 7.f, PP_SLACK = 8.f, PP_NONE = -3e38f;

// 128-row operands in shared memory: Q of two tiles (fp32: hi and lo of one), two stages of K and of V; the ring
template <int HD>
struct PpCfg {
    static constexpr int TILE = pg_tile_bytes(HD);
    static constexpr int NB = HD / 32;
    static constexpr int OP = 128 * HD * 2;  // bytes of an operand
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_K = OFF_Q + 2 * OP;
    static constexpr int OFF_V = OFF_K + 2 * OP;
    static constexpr int OFF_RAW = OFF_V + 2 * OP;
    static constexpr int OFF_BARS = OFF_RAW + PP_RAW * 4 * TILE;
    static constexpr int OFF_ROWS = OFF_BARS + 512;      // fp32: [2 blocks][2 halves][128] values of the rows
    static constexpr int SMEM = OFF_ROWS + 2048 + 1024;  // + alignment of the base
    static_assert(SMEM <= 232448, "shared memory");
};

struct PpArgs {
    PagesView p;
    er_pages_attention_args a;
    int min_rows;  // sequences with fewer query rows a KV head are another kernel's
    int shortfall;  // tests of the give-up path: arrivals that CTA 0 waits for in vain
};

struct PpBars {
    uint64_t raw[PP_RAW], rawfree[PP_RAW], kfull[2], kempty[2], vfull[2], vempty[2], s[2], p[2], o[2], oempty[2], x[2], q, end;
    uint32_t tmem;
    int item[6];  // sequence, first query row, KV head, found, first row of q, query rows
};
static_assert(sizeof(PpBars) <= 512, "barriers");

// ---------------------------------------------------------------------------
// tcgen05 wrappers
// ---------------------------------------------------------------------------
// kind::f16: fp16 A and B (both K-major), fp32 D, M = 128
constexpr uint32_t pp_idesc(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24); }
// The products are issued by code that the whole warp runs with equal operands (so they can sit in uniform
// registers); only the lane with `one` set issues.  D (+)= A B^T, A in shared memory / in TMEM.
ER_DEV void pp_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
        "r"(accumulate), "r"(one)
        : "memory");
}
ER_DEV void pp_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
        "r"(accumulate), "r"(one)
        : "memory");
}
// the mbarrier arrives once every product that this thread issued before has completed
ER_DEV void pp_commit(uint64_t *bar, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(one)
        : "memory");
}
ER_DEV uint32_t pp_elect() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one;
}
// 32 consecutive 32-bit columns of this thread's lane
ER_DEV void pp_st32(uint32_t taddr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
ER_DEV void pp_st16(uint32_t taddr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
ER_DEV void pp_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// the loaded registers are valid after pp_wait_ld, which takes them through so that no use moves ahead of it
ER_DEV void pp_ld32(uint32_t taddr, float *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
          "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
          "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr));
}
ER_DEV void pp_wait_ld(float *v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                   "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                   "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
                 :
                 : "memory");
}
// two fp32 operations an instruction
ER_DEV float2 pp_fma2(float2 a, float2 b, float2 c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)), "l"(*reinterpret_cast<uint64_t *>(&c)));
    return *reinterpret_cast<float2 *>(&d);
}
ER_DEV float2 pp_add2(float2 a, float2 b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(*reinterpret_cast<uint64_t *>(&a)), "l"(*reinterpret_cast<uint64_t *>(&b)));
    return *reinterpret_cast<float2 *>(&d);
}
ER_DEV float pp_max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
// values of nibble N of each half of w with scale pair d, z = -24 d
template <int N>
ER_DEV uint32_t pp_val(uint32_t w, uint32_t d, uint32_t z) {
    return h2_fma(pg_code<N>(w), d, z);
}
// row of a block at place k' (see the header)
__host__ __device__ constexpr int pp_row(int k) {
    return (k & ~31) + ((k >> 2) & 1) * 16 + ((k >> 1) & 1) * 8 + ((k >> 3) & 3) * 2 + (k & 1);
}

// What a CTA works on: query rows f0 .. f0 + nf - 1 of sequence b, KV head h, against rows any_lo .. any_hi (those that
// any of them attends) in nblk blocks from row base on; all of them attend rows all_lo .. all_hi.
struct PpItem {
    int b, h, f0, nf, q0, past, any_lo, any_hi, all_lo, all_hi, base, nblk;
};
// The item of this CTA: (sequence, ROWS query rows, KV head), heads fastest, long sequences first and a sequence's
// last rows first.  False: none.
template <int ROWS>
ER_DEV bool pp_find(const PpArgs &P, PpBars &B, int warp, int lane, PpItem &I) {
    const er_pages_attention_args &a = P.a;
    const int KV = P.p.KV, G = a.n_heads / KV, R = P.p.page_rows;
    if (warp == 0) {
        const int x = blockIdx.x / KV;
        int found = 0, base = 0;
        for (int b0 = 0; b0 < a.n_seqs && !found; b0 += 32) {
            const int b = b0 + lane;
            int n = 0, len = -1;
            if (b < a.n_seqs) {
                const int q0 = a.q_start_dev[b], q1 = a.q_start_dev[b + 1];
                len = a.lens_dev[b];
                if (q0 < 0 || q1 < q0 || q1 > a.n_tokens || len < 0 || len > pg_max_len(a.table_stride, R)) {
                    if (blockIdx.x == 0) atomicOr(P.p.flags, ER_PAGES_FLAG_RANGE);
                } else if ((long long)(q1 - q0) * G >= P.min_rows) {
                    n = (int)(((long long)(q1 - q0) * G + ROWS - 1) / ROWS);
                }
            }
            // the items before this sequence's: of 32 sequences the longest come first, so that the last items are short
            int first = base, all = 0;
            for (int o = 0; o < 32; ++o) {
                const int len_o = __shfl_sync(0xffffffffu, len, o), n_o = __shfl_sync(0xffffffffu, n, o);
                if (len_o > len || (len_o == len && o < lane)) first += n_o;
                all += n_o;
            }
            const bool mine = x >= first && x < first + n;
            if (mine) {
                B.item[0] = b;
                B.item[1] = (n - 1 - (x - first)) * ROWS;
                B.item[2] = blockIdx.x % KV;
            }
            found = __any_sync(0xffffffffu, mine);
            base += all;
        }
        if (lane == 0) B.item[3] = found;
    }
    __syncthreads();
    if (!B.item[3]) return false;
    I.b = B.item[0];
    I.f0 = B.item[1];
    I.h = B.item[2];
    I.q0 = a.q_start_dev[I.b];
    const int qn = a.q_start_dev[I.b + 1] - I.q0;
    I.past = a.lens_dev[I.b] - qn;
    I.nf = (int)min((long long)qn * G - I.f0, (long long)ROWS);
    if (threadIdx.x == 0) {
        B.item[4] = I.q0;
        B.item[5] = I.nf;
    }
    I.any_hi = I.past + (I.f0 + I.nf - 1) / G;
    I.any_lo = pg_first(I.past + I.f0 / G, a.window);
    I.base = I.any_lo & ~15;
    I.nblk = I.any_hi < 0 ? 0 : (I.any_hi - I.base) / PP_BLOCK + 1;
    I.all_hi = I.past + I.f0 / G;
    I.all_lo = pg_first(I.any_hi, a.window);
    return true;
}

// Whole warp: false once a wait gave up.  What depends on a warp that gave up waits in vain and gives up too, so every
// wait ends.
ER_DEV bool pp_wait(const PpArgs &P, uint64_t *bar, uint32_t par, int lane) {
    const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, par));
    if (!ok && lane == 0) atomicOr(P.p.flags, ER_FLAG_WAIT);
    return ok;
}

ER_DEV const uint8_t *pp_shfl(const uint8_t *p, int lane) {
    return reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, (unsigned long long)p, lane));
}

// NR query rows as rows row0 .. of the K-major operand at dst: lane i < NR knows row row0 + i's address, or NULL (zeros).
// A row is times a power of two that brings its largest value to [2^14, 2^15) (and the scale's sign); LO: the lo halves go
// to dst + OP.  down[row]: the factor that takes its scores to log2 units.
// Neighbouring lanes take 16 bytes each of a row, first as they are to places of its operand (every row on its way at
// once, in no registers), then from there, row by row, into the operand.  A thread a row and four loads at a time took
// 20,000 cycles of a CTA.
template <class T, int HD, bool LO, int NR>
ER_DEV void pp_queries(const er_pages_attention_args &a, uint8_t *dst, float *down, const T *mine, int row0, int lane) {
    using C = PpCfg<HD>;
    constexpr int LPR = HD * (int)sizeof(T) / 16, RPP = 32 / LPR, V = 16 / (int)sizeof(T);
    constexpr int HALF = HD / 8;  // 16-byte places of a row of one operand
    const bool vec = ((uintptr_t)a.q_dev & 15) == 0 && (a.q_stride * sizeof(T)) % 16 == 0;
    const int c = lane % LPR;  // values V c .. of the row
    auto place = [&](int r, int ch) { return dst + r * 128 + (ch >> 3) * 16384 + (((ch & 7) ^ (r & 7)) << 4); };
    auto raw_at = [&](int r) { return place(r, c & (HALF - 1)) + (c / HALF) * C::OP; };
#pragma unroll 1
    for (int p = 0; p < NR; p += RPP) {
        const int i = p + lane / LPR;
        const uint8_t *src = pp_shfl(reinterpret_cast<const uint8_t *>(mine), i);
        uint8_t *to = raw_at(row0 + i);
        if (vec) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)),
                         "l"(src ? src + 16 * c : (const uint8_t *)a.q_dev), "r"(src ? 16 : 0)
                         : "memory");
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e)
                reinterpret_cast<T *>(to)[e] = src ? reinterpret_cast<const T *>(src)[V * c + e] : pg_cvt<T>(0.f);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    const float scale = a.scale != 0.f ? a.scale : 1.f / sqrtf((float)HD);
#pragma unroll 2
    for (int p = 0; p < NR; p += RPP) {
        const int r = row0 + p + lane / LPR;
        __align__(16) T v[V];
        *reinterpret_cast<uint4 *>(v) = *reinterpret_cast<const uint4 *>(raw_at(r));
        float x[V];
        uint32_t top = 0;  // the largest magnitude's bits; an infinity's or a NaN's are above every number's
#pragma unroll
        for (int e = 0; e < V; ++e) {
            x[e] = pg_ld<T>(v + e);
            top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
        }
#pragma unroll
        for (int o = 1; o < LPR; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        __syncwarp();  // the row is read: its places may be written
        // an infinite or NaN query: the row is NaN, and so are its scores
        const int ex = min(max((int)(top >> 23), 15), 253);
        const float up = top >= 0x7F800000u ? NAN : copysignf(__uint_as_float((uint32_t)(268 - ex) << 23), scale);
        uint32_t hi[V / 2];
        [[maybe_unused]] uint32_t lo[V / 2];
#pragma unroll
        for (int k = 0; k < V / 2; ++k) {
            const float y0 = x[2 * k] * up, y1 = x[2 * k + 1] * up;
            hi[k] = pg_pack(y0, y1);
            if constexpr (LO) {
                const float2 z = __half22float2(*reinterpret_cast<const __half2 *>(&hi[k]));
                lo[k] = pg_pack(y0 - z.x, y1 - z.y);
            }
        }
        uint8_t *d = place(r, V * c / 8);
        if constexpr (V == 8) {
            *reinterpret_cast<uint4 *>(d) = make_uint4(hi[0], hi[1], hi[V / 2 - 2], hi[V / 2 - 1]);
        } else {
            *reinterpret_cast<uint2 *>(d + 8 * (c & 1)) = make_uint2(hi[0], hi[1]);
            if constexpr (LO) *reinterpret_cast<uint2 *>(d + C::OP + 8 * (c & 1)) = make_uint2(lo[0], lo[1]);
        }
        // (a factor too small for fp32 still has to leave -infinity as it is)
        if (c == 0)
            down[r] = fmaxf(__uint_as_float((uint32_t)(ex - 14) << 23) * (fabsf(scale) * 1.4426950408889634f), 1.2e-38f);
    }
    static_assert(LO == (V == 4), "fp32 rows have lo halves");
}

// ---- operands (warps 8-11).  Half block i of the walk (block i / 2) lies in ring slot i % PP_RAW; warps 8, 9 use the first
// halves, 10 and 11 the second
template <int HD>
ER_DEV void pp_operands(const PpArgs &P, PpBars &B, uint8_t *smem, const PpItem &I, int warp, int lane) {
    using C = PpCfg<HD>;
    const int any_lo = I.any_lo, any_hi = I.any_hi, all_lo = I.all_lo, all_hi = I.all_hi, base = I.base, nblk = I.nblk;
    auto wait = [&](uint64_t *bar, uint32_t par) { return pp_wait(P, bar, par, lane); };
    const int pw = warp - 8, g = lane >> 2, t = lane & 3, half = pw >> 1;
    const uint8_t *ring = smem + C::OFF_RAW;
    // K: a job is 8 rows, a lane one row's words of quad lane t.  An odd row writes its blocks in the other order: 8 lanes
    // then cover all the bank groups.  Row 32 pw + 8 job + g goes to place 32 pw + 8 (g / 2) + 4 (job / 2) + 2 (job % 2) + g % 2.
    const int odd = g & 1;
    const uint32_t kat = (uint32_t)((32 * pw + 8 * (g >> 1) + odd) * 128), kch = (uint32_t)(((4 * odd + t) ^ odd) << 4);
    const uint32_t sel0 = odd ? 0x3232u : 0x1010u, sel1 = odd ? 0x1010u : 0x3232u;
    auto keys = [&](auto edge_tag, const uint8_t *raw, uint8_t *kd) {
        constexpr bool EDGE = decltype(edge_tag)::value;
#pragma unroll 1
        for (int job = 0; job < 4; ++job) {
            const int in = 8 * (job & 1) + g;
            const uint8_t *src = raw + (2 * pw + (job >> 1) & 3) * C::TILE;
            uint32_t w[C::NB], ds[C::NB / 2];
            if constexpr (HD == 128) {
                const uint4 x = *reinterpret_cast<const uint4 *>(src + in * 64 + t * 16);
                w[0] = odd ? x.y : x.x; w[1] = odd ? x.x : x.y; w[2] = odd ? x.w : x.z; w[C::NB - 1] = odd ? x.z : x.w;
                const uint2 y = *reinterpret_cast<const uint2 *>(src + pg_off_ks(HD) + in * 8);
                ds[0] = y.x; ds[C::NB / 2 - 1] = y.y;
            } else {
                const uint2 x = *reinterpret_cast<const uint2 *>(src + in * 32 + t * 8);
                w[0] = odd ? x.y : x.x; w[1] = odd ? x.x : x.y;
                ds[0] = *reinterpret_cast<const uint32_t *>(src + pg_off_ks(HD) + in * 4);
            }
            if constexpr (EDGE) {  // a row with a NaN value: its K carries it
                const unsigned short *vs = reinterpret_cast<const unsigned short *>(src + pg_off_vs(HD));
                bool nan = false;
#pragma unroll
                for (int bb = 0; bb < C::NB; ++bb) nan |= (vs[pg_vs_half(in, bb, HD)] & 0x7FFF) > 0x7C00;
                if (nan)
#pragma unroll
                    for (int k = 0; k < C::NB / 2; ++k) ds[k] = 0x7FFF7FFFu;
            }
            const int at = 2 * (job & 1) + 4 * (job >> 1);
            uint8_t *dst = kd + kat + at * 128;
            const uint32_t ch = kch ^ (uint32_t)(at << 4);
#pragma unroll
            for (int k = 0; k < C::NB; ++k) {
                const uint32_t d = prmt(ds[k >> 1], 0u, (k & 1) ? sel1 : sel0), z = pg_m24(d);
                *reinterpret_cast<uint4 *>(dst + (k >> 1) * 16384 + (ch ^ ((k & 1) * 64u))) =
                    make_uint4(pp_val<0>(w[k], d, z), pp_val<1>(w[k], d, z), pp_val<2>(w[k], d, z), pp_val<3>(w[k], d, z));
            }
        }
    };
    // V: a lane holds 4 rows of one dim of two tiles: 16 bytes of the operand.  Odd g takes the half block's two pairs of
    // tiles in the other order (bank groups again).  HD = 64: a warp takes half the words of a lane.
    constexpr int NU = HD == 128 ? 4 : 2;
    const int q = HD == 128 ? pw & 1 : 0, u0 = HD == 128 ? 0 : 2 * (pw & 1);
    auto vals = [&](auto edge_tag, const uint8_t *raw, uint8_t *vd, int r0) {
        constexpr bool EDGE = decltype(edge_tag)::value;
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
            const int pair = k ^ odd;  // of the half block
            const uint8_t *sa = raw + 2 * pair * C::TILE, *sb = sa + C::TILE;
            uint32_t wa[NU], wb[NU], da[NU / 2][2], db[NU / 2][2];
            if constexpr (HD == 128) {
                const uint4 x = *reinterpret_cast<const uint4 *>(sa + pg_off_v(HD) + q * 512 + lane * 16);
                const uint4 y = *reinterpret_cast<const uint4 *>(sb + pg_off_v(HD) + q * 512 + lane * 16);
                wa[0] = x.x; wa[1] = x.y; wa[2] = x.z; wa[NU - 1] = x.w;
                wb[0] = y.x; wb[1] = y.y; wb[2] = y.z; wb[NU - 1] = y.w;
                const uint4 v = *reinterpret_cast<const uint4 *>(sa + pg_off_vs(HD) + t * 32 + 16 * q);
                const uint4 z = *reinterpret_cast<const uint4 *>(sb + pg_off_vs(HD) + t * 32 + 16 * q);
                da[0][0] = v.x; da[0][1] = v.y; da[NU / 2 - 1][0] = v.z; da[NU / 2 - 1][1] = v.w;
                db[0][0] = z.x; db[0][1] = z.y; db[NU / 2 - 1][0] = z.z; db[NU / 2 - 1][1] = z.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2 *>(sa + pg_off_v(HD) + lane * 16 + 4 * u0);
                const uint2 y = *reinterpret_cast<const uint2 *>(sb + pg_off_v(HD) + lane * 16 + 4 * u0);
                wa[0] = x.x; wa[1] = x.y;
                wb[0] = y.x; wb[1] = y.y;
                const uint2 v = *reinterpret_cast<const uint2 *>(sa + pg_off_vs(HD) + t * 16 + 4 * u0);
                const uint2 z = *reinterpret_cast<const uint2 *>(sb + pg_off_vs(HD) + t * 16 + 4 * u0);
                da[0][0] = v.x; da[0][1] = v.y;
                db[0][0] = z.x; db[0][1] = z.y;
            }
            if constexpr (EDGE) {  // scales of rows that nobody attends, or that are NaN: 0
#pragma unroll
                for (int x = 0; x < NU / 2; ++x)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t part = e ? 0xFFFF0000u : 0x0000FFFFu, inf = 0x7C007C00u & part;
                            const int ra = r0 + 64 * half + 32 * pair + 2 * t + e + 8 * i, rb = ra + 16;
                            if ((da[x][i] & 0x7FFF7FFFu & part) > inf || ra < any_lo || ra > any_hi) da[x][i] &= ~part;
                            if ((db[x][i] & 0x7FFF7FFFu & part) > inf || rb < any_lo || rb > any_hi) db[x][i] &= ~part;
                        }
            }
            uint8_t *dst = vd + half * (HD * 128) + (((pair * 4 + t) ^ g) << 4);
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                const uint32_t a0 = da[u >> 1][0], a1 = da[u >> 1][1], b0 = db[u >> 1][0], b1 = db[u >> 1][1];
                const uint32_t za0 = pg_m24(a0), za1 = pg_m24(a1), zb0 = pg_m24(b0), zb1 = pg_m24(b1);
                const int d = 64 * q + 16 * (u0 + u) + g;
                *reinterpret_cast<uint4 *>(dst + d * 128) =
                    make_uint4(pp_val<0>(wa[u], a0, za0), pp_val<2>(wa[u], a1, za1), pp_val<0>(wb[u], b0, zb0),
                               pp_val<2>(wb[u], b1, zb1));
                *reinterpret_cast<uint4 *>(dst + (d + 8) * 128) =
                    make_uint4(pp_val<1>(wa[u], a0, za0), pp_val<3>(wa[u], a1, za1), pp_val<1>(wb[u], b0, zb0),
                               pp_val<3>(wb[u], b1, zb1));
            }
        }
    };
    bool ok = true;
    RingWalk<PP_RAW> at(half);  // of half block 2 j + half
    for (int j = 0; j < nblk; ++j, at.step()) {
        const int st = j & 1, ph = (j >> 1) & 1;
        ok = at.ready([&](int slot, int par) { return wait(B.rawfree + slot, par); },
                      [&](int slot, int par) { return wait(B.raw + slot, par); });
        if (!ok) break;
        const uint8_t *raw = ring + at.slot * (4 * C::TILE);
        const int r0 = base + PP_BLOCK * j;
        const bool edge = r0 < all_lo || r0 + PP_BLOCK - 1 > all_hi;
        if (j >= 2) ok = wait(B.kempty + st, ph ^ 1);
        if (!ok) break;
        uint8_t *kd = smem + C::OFF_K + st * C::OP, *vd = smem + C::OFF_V + st * C::OP;
        if (edge) keys(std::true_type{}, raw, kd);
        else keys(std::false_type{}, raw, kd);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(B.kfull + st);
        if (j >= 2) ok = wait(B.vempty + st, ph ^ 1);
        if (!ok) break;
        if (edge) vals(std::true_type{}, raw, vd, r0);
        else vals(std::false_type{}, raw, vd, r0);
        fence_proxy_async_smem();
        __syncwarp();
        // in this order: no warp gets three blocks ahead of one that has not given its slot back (RingWalk)
        if (lane == 0) mbar_arrive(B.rawfree + at.slot);
        if (lane == 0) mbar_arrive(B.vfull + st);
    }
}

// ---- copies (warp 13): lane i < 4 requests tile i of each half block; the pages are looked up one half block ahead
template <int HD>
ER_DEV void pp_copies(const PpArgs &P, PpBars &B, uint8_t *smem, const PpItem &I, int lane) {
    using C = PpCfg<HD>;
    const er_pages_attention_args &a = P.a;
    const int KV = P.p.KV, R = P.p.page_rows, b = I.b, h = I.h, base = I.base, any_hi = I.any_hi;
    auto wait = [&](uint64_t *bar, uint32_t par) { return pp_wait(P, bar, par, lane); };
    const int nhalf = 2 * I.nblk;
    auto page_of = [&](int i) {  // the table's entry for tile `lane` of half block i; -1: nothing to read there
        const int row = base + 64 * i + 16 * lane;
        return lane < 4 && i < nhalf && row <= any_hi ? a.tables_dev[(size_t)b * a.table_stride + row / R] : -1;
    };
    int page = page_of(0), slot = 0, par = 1;
    bool ok = true;
    int i = 0;
    for (; i < nhalf; ++i) {
        if (i >= PP_RAW) ok = wait(B.rawfree + slot, par);
        if (!ok) break;
        const int row = base + 64 * i + 16 * lane;
        const bool there = lane < 4 && row <= any_hi;
        if (there && (page < 0 || page >= P.p.n_pages)) {
            atomicOr(P.p.flags, ER_PAGES_FLAG_RANGE);
            page = 0;
        }
        const int n = __popc(__ballot_sync(0xffffffffu, there));
        if (lane == 0) mbar_arrive_expect_tx(B.raw + slot, n * C::TILE);
        __syncwarp();
        if (there)
            bulk_g2s(smem + C::OFF_RAW + (slot * 4 + lane) * C::TILE,
                     P.p.pool + (((size_t)page * KV + h) * (R >> 4) + ((row % R) >> 4)) * C::TILE, C::TILE,
                     B.raw + slot);
        page = page_of(i + 1);
        if (++slot == PP_RAW) {
            slot = 0;
            par ^= 1;
        }
    }
    // copies may still be landing where this warp or one that uses them gave up
    for (int k = max(0, i - PP_RAW); k < i; ++k) pg_drain(B.raw + k % PP_RAW, (k / PP_RAW) & 1);
}

// barriers (thread 0) and the whole of TMEM (warp 12)
// query_warps, softmax_warps: warps that make the queries' operands, and that share a tile's P
ER_DEV void pp_setup(PpBars &B, int tid, int warp, int query_warps, int softmax_warps, int shortfall) {
    if (tid == 0) {
        for (int i = 0; i < PP_RAW; ++i) {
            mbar_init(B.raw + i, 1);
            mbar_init(B.rawfree + i, 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(B.kfull + i, 4 + (blockIdx.x == 0 ? shortfall : 0));
            mbar_init(B.kempty + i, 1);
            mbar_init(B.vfull + i, 4);
            mbar_init(B.vempty + i, 1);
            mbar_init(B.s + i, 1);
            mbar_init(B.p + i, softmax_warps);
            mbar_init(B.o + i, 1);
            mbar_init(B.oempty + i, 8);
            mbar_init(B.x + i, 8);
        }
        mbar_init(&B.q, query_warps);
        mbar_init(&B.end, 1);
        fence_mbar_init();
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&B.tmem)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
}
ER_DEV void pp_close(PpBars &B, int warp) {
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(B.tmem), "r"(512) : "memory");
    }
}
// the whole of TMEM is allocated: it starts at 0, which keeps its addresses constants
constexpr uint32_t PP_TMEM = 0;

// S = Q K^T, D (+)= P V, issued by the lane with `one` set
template <int HD>
ER_DEV void pp_score(uint32_t d, uint32_t q, uint32_t k, bool more, uint32_t one) {
#pragma unroll
    for (int i = 0; i < HD / 16; ++i) {
        const uint32_t at = (uint32_t)((i >> 2) * 16384 + (i & 3) * 32);
        pp_mma_ss(d, tc_desc_sw128(q) + (at >> 4), tc_desc_sw128(k) + (at >> 4), pp_idesc(128), more || i > 0, one);
    }
}
// P's lo halves lie 64 columns after the hi ones
template <int HD>
ER_DEV void pp_value(uint32_t d, uint32_t p, uint32_t v, bool more, uint32_t one) {
#pragma unroll
    for (int i = 0; i < PP_BLOCK / 16; ++i) {
        const uint64_t b = tc_desc_sw128(v) + (((i >> 2) * (HD * 128) + (i & 3) * 32) >> 4);
        pp_mma_ts(d, p + i * 8, b, pp_idesc(HD), more || i > 0, one);
        pp_mma_ts(d, p + 64 + i * 8, b, pp_idesc(HD), 1, one);
    }
}

// One block's scores of a row in registers: masked, their largest, and the probabilities written over them.
template <int N>
ER_DEV void pp_mask(float (&s)[N], int lo, int hi) {  // (places 64 on are 64 rows on: pp_row)
#pragma unroll
    for (int k = 0; k < N; ++k)
        if (pp_row(k) < lo || pp_row(k) > hi) s[k] = -INFINITY;
}
template <int N>
ER_DEV float pp_largest(const float (&s)[N]) {
    float mx[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
    for (int k = 4; k < N - 4; k += 8)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = pp_max3(mx[e], s[k + 2 * e], s[k + 2 * e + 1]);
    return pp_max3(pp_max3(mx[0], mx[1], fmaxf(s[N - 4], s[N - 3])), pp_max3(mx[2], mx[3], s[N - 2]), s[N - 1]);
}
// p = 2^(s down - m + PP_UP) as hi and lo halves to N / 2 columns at tP and 64 columns on; returns their sum
template <int N>
ER_DEV float pp_probabilities(const float (&s)[N], uint32_t tP, float down, float m) {
    const float2 nb = make_float2(PP_UP - m, PP_UP - m), dn = make_float2(down, down);
    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int q = 0; q < N / 32; ++q) {  // 32 columns of S become 16 of P: few registers beside S itself
        uint32_t ph[16];
        uint32_t pl[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            float2 x = pp_fma2(make_float2(s[32 * q + 2 * k], s[32 * q + 2 * k + 1]), dn, nb);
            x.x = pg_ex2(x.x);
            x.y = pg_ex2(x.y);
            sum[k & 1] = pp_add2(sum[k & 1], x);
            ph[k] = pg_pack(x.x, x.y);
            const float2 z = pp_fma2(__half22float2(*reinterpret_cast<const __half2 *>(&ph[k])), make_float2(-1.f, -1.f), x);
            pl[k] = pg_pack(z.x, z.y);
        }
        pp_st16(tP + 16 * q, ph);
        pp_st16(tP + 64 + 16 * q, pl);
    }
    return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}
// N = 2 HD / sizeof(T) values of an output row a thread, 32 at a time from `load`, to `mine` (NULL: not a real row).  Through shared memory (`stage`: 2 HD bytes a row, the warp's own place in the queries, which nothing reads any
// more), so that neighbouring lanes write a row: a thread a row takes a cycle a 16-byte piece.
template <class T, int HD, class Load>
ER_DEV void pp_store(const er_pages_attention_args &a, uint8_t *stage, T *mine, int lane, Load load) {
    constexpr int N = 2 * HD / (int)sizeof(T), ROW = 2 * HD, LPR = ROW / 16, V = 16 / (int)sizeof(T);
    const bool vec = ((uintptr_t)a.out_dev & 15) == 0 && (a.out_stride * sizeof(T)) % 16 == 0;
#pragma unroll
    for (int k = 0; k < N / 32; ++k) {
        float o[32];
        load(k, o);
        __align__(16) T v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = pg_cvt<T>(o[e]);
        if (vec) {
#pragma unroll
            for (int e = 0; e < 32 / V; ++e)
                *reinterpret_cast<uint4 *>(stage + lane * ROW + (((32 / V * k + e) ^ (lane & 7)) << 4)) = reinterpret_cast<uint4 *>(v)[e];
        } else if (mine) {
#pragma unroll
            for (int e = 0; e < 32; ++e) mine[32 * k + e] = v[e];
        }
    }
    if (!vec) return;
    __syncwarp();
    const int c = lane % LPR;
#pragma unroll 4
    for (int p = 0; p < 32; p += 32 / LPR) {
        const int i = p + lane / LPR;
        const uint8_t *dst = pp_shfl(reinterpret_cast<const uint8_t *>(mine), i);
        if (dst) const_cast<uint4 *>(reinterpret_cast<const uint4 *>(dst))[c] = *reinterpret_cast<const uint4 *>(stage + i * ROW + ((c ^ (i & 7)) << 4));
    }
}
ER_DEV float pp_lse(float m, float l) { return l == 0.f ? -INFINITY : (m - PP_UP + log2f(l)) * 0.6931471805599453f; }

// ---------------------------------------------------------------------------
template <class T, int HD>
__global__ void __launch_bounds__(PP_THREADS, 1) pages_prompt_kernel(const PpArgs P) {
    using C = PpCfg<HD>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);  // swizzle atoms: 1024-aligned
    PpBars &B = *reinterpret_cast<PpBars *>(smem + C::OFF_BARS);
    const er_pages_attention_args &a = P.a;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // so that the compiler knows it is the same in the whole warp
    const int G = a.n_heads / P.p.KV;
    PpItem I;
    if (!pp_find<256>(P, B, warp, lane, I)) return;
    const int nx = I.nf > 128 ? 2 : 1;  // tiles
    pp_setup(B, tid, warp, 4 * nx, 4, P.shortfall);
    // a softmax thread's tile and row
    const int X = warp >> 2, r = tid & 127, f = I.f0 + X * 128 + r, tok = f / G;
    const int row = I.q0 + tok, head = I.h * G + (f - tok * G);
    const bool soft = warp < 8 && X < nx, real = X * 128 + r < I.nf;
    auto wait = [&](uint64_t *bar, uint32_t par) { return pp_wait(P, bar, par, lane); };

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
        if (soft) {
            const uint32_t tl = PP_TMEM + ((uint32_t)(32 * (warp & 3)) << 16);  // this warp's lanes
            const uint32_t tS = tl + X * 128, tO = tl + 256 + X * HD;
            const int pos = real ? max(I.past + tok, -1) : 2147483647;  // rows past the last are computed (from zeros) and dropped
            const int first = a.window && real ? max(0, pos - a.window + 1) : 0;
            float m = PP_NONE, l = 0.f;
            float *rows = reinterpret_cast<float *>(smem + C::OFF_ROWS) + X * 128;
            pp_queries<T, HD, false, 32>(a, smem + C::OFF_Q + X * C::OP, rows,
                                         real ? (const T *)a.q_dev + row * a.q_stride + (size_t)head * HD : nullptr,
                                         32 * (warp & 3), lane);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.q);
            const float down = rows[r];
            bool ok = true;
            for (int j = 0; j < I.nblk; ++j) {
                ok = wait(B.s + X, j & 1);
                if (!ok) break;
                tc_fence_after();
                float s[128];
#pragma unroll
                for (int k = 0; k < 4; ++k) pp_ld32(tS + 32 * k, s + 32 * k);
#pragma unroll
                for (int k = 0; k < 4; ++k) pp_wait_ld(s + 32 * k);
                const int r0 = I.base + PP_BLOCK * j;
                if (__any_sync(0xffffffffu, r0 < first || r0 + PP_BLOCK - 1 > pos)) pp_mask(s, first - r0, min(pos, r0 + PP_BLOCK) - r0);
                const float mt = pp_largest(s) * down;
                if (__any_sync(0xffffffffu, mt > m + PP_SLACK)) {
                    const float mn = mt > m + PP_SLACK ? mt : m;
                    const float corr = mn == m ? 1.f : pg_ex2(m - mn);
                    l *= corr;
                    m = mn;
                    if (j > 0) {
#pragma unroll
                        for (int k = 0; k < HD / 32; ++k) {
                            float o[32];
                            pp_ld32(tO + 32 * k, o);
                            pp_wait_ld(o);
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= corr;
                            pp_st32(tO + 32 * k, reinterpret_cast<uint32_t *>(o));
                        }
                    }
                }
                l += pp_probabilities(s, tS, down, m);
                pp_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(B.p + X);
            }
            if (ok) ok = I.nblk > 0 ? wait(B.o + X, 0) : wait(&B.q, 0);  // the queries' place is free
            if (ok) {
                tc_fence_after();
                const float inv = 1.f / l;
                // the row once more, from shared memory: it would cost registers in the loop
                const volatile int *item = B.item;
                const int f = item[1] + X * 128 + r, tok = f / G, row = item[4] + tok, head = item[2] * G + (f - tok * G);
                const bool real = X * 128 + r < item[5];
                pp_store<T, HD>(a, smem + C::OFF_Q + warp * (64 * HD), real ? (T *)a.out_dev + row * a.out_stride + (size_t)head * HD : nullptr,
                                lane, [&](int k, float (&o)[32]) {
                                    if (I.nblk > 0) {
                                        pp_ld32(tO + 32 * k, o);
                                        pp_wait_ld(o);
                                    }
#pragma unroll
                                    for (int e = 0; e < 32; ++e) o[e] = l == 0.f ? 0.f : o[e] * inv;
                                });
                if (real && a.lse_dev) a.lse_dev[(size_t)row * a.n_heads + head] = pp_lse(m, l);
            }
        }
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        pp_operands<HD>(P, B, smem, I, warp, lane);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        if (warp == 12 && I.nblk > 0) {
            const uint32_t qb = smem_u32(smem + C::OFF_Q), kb = smem_u32(smem + C::OFF_K), vb = smem_u32(smem + C::OFF_V);
            const uint32_t one = pp_elect();
            bool ok = wait(&B.q, 0) && wait(B.kfull + 0, 0);
            if (ok) {
                tc_fence_after();
                for (int x = 0; x < nx; ++x) {
                    pp_score<HD>(PP_TMEM + x * 128, qb + x * C::OP, kb, false, one);
                    pp_commit(B.s + x, one);
                }
                pp_commit(B.kempty + 0, one);
            }
            for (int j = 0; ok && j < I.nblk; ++j) {
                const int st = j & 1, j1 = j + 1, st1 = j1 & 1;
                ok = wait(B.vfull + st, (j >> 1) & 1);
                for (int x = 0; ok && x < nx; ++x) {
                    ok = wait(B.p + x, j & 1);
                    if (!ok) break;
                    tc_fence_after();
                    pp_value<HD>(PP_TMEM + 256 + x * HD, PP_TMEM + x * 128, vb + st * C::OP, j > 0, one);
                    if (x == nx - 1) pp_commit(B.vempty + st, one);
                    if (j1 == I.nblk) {
                        pp_commit(B.o + x, one);
                    } else {
                        if (x == 0) ok = wait(B.kfull + st1, (j1 >> 1) & 1);
                        if (!ok) break;
                        tc_fence_after();
                        pp_score<HD>(PP_TMEM + x * 128, qb + x * C::OP, kb + st1 * C::OP, false, one);
                        pp_commit(B.s + x, one);
                        if (x == nx - 1) pp_commit(B.kempty + st1, one);
                    }
                }
            }
            if (!ok) {  // given up: products in flight read shared memory and TMEM until they end
                pp_commit(&B.end, one);
                pg_drain(&B.end, 0);
            }
        } else if (warp == 13) {
            pp_copies<HD>(P, B, smem, I, lane);
        }
    }
    pp_close(B, warp);
}

// ---------------------------------------------------------------------------
template <int HD>
__global__ void __launch_bounds__(PP_THREADS, 1) pages_prompt32_kernel(const PpArgs P) {
    using C = PpCfg<HD>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);  // swizzle atoms: 1024-aligned
    PpBars &B = *reinterpret_cast<PpBars *>(smem + C::OFF_BARS);
    const er_pages_attention_args &a = P.a;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // so that the compiler knows it is the same in the whole warp
    const int G = a.n_heads / P.p.KV;
    PpItem I;
    if (!pp_find<128>(P, B, warp, lane, I)) return;
    pp_setup(B, tid, warp, 8, 8, P.shortfall);
    // warps 0-3 and 4-7: thread = query row, W = which half of its columns
    const int r = tid & 127, W = warp >> 2, f = I.f0 + r, tok = f / G;
    const int row = I.q0 + tok, head = I.h * G + (f - tok * G);
    const bool real = r < I.nf;
    float *xch = reinterpret_cast<float *>(smem + C::OFF_ROWS);  // [2 blocks][2 halves][128]
    auto wait = [&](uint64_t *bar, uint32_t par) { return pp_wait(P, bar, par, lane); };
    const uint32_t tl = PP_TMEM + ((uint32_t)(32 * (warp & 3)) << 16);  // this warp's lanes

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
        constexpr int HO = HD / 2;  // columns of O of a thread
        const int pos = real ? max(I.past + tok, -1) : 2147483647;  // rows past the last are computed (from zeros) and dropped
        const int first = a.window && real ? max(0, pos - a.window + 1) : 0;
        float m = PP_NONE, l = 0.f, last = 1.f;  // last: the factor of the block whose O is still to come
        float o[HO];
#pragma unroll
        for (int e = 0; e < HO; ++e) o[e] = 0.f;
        // the queries, 16 rows a warp; the factors lie where block 1's exchange will be (nobody gets there before both of a
        // row's threads have read them)
        const int row0 = 32 * (warp & 3) + 16 * W, fq = I.f0 + row0 + (lane & 15), tq = fq / G;
        pp_queries<float, HD, true, 16>(a, smem + C::OFF_Q, xch + 256,
                                        row0 + (lane & 15) < I.nf ? (const float *)a.q_dev + (I.q0 + tq) * a.q_stride +
                                                                        (size_t)(I.h * G + (fq - tq * G)) * HD : nullptr,
                                        row0, lane);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.q);
        bool ok = wait(&B.q, 0);
        const float down = xch[256 + r];
        auto gather = [&](int j) {  // o = o * factor + O of block j
            const int buf = j & 1;
            if (!wait(B.o + buf, (j >> 1) & 1)) return false;
            tc_fence_after();
            float d[HO];
#pragma unroll
            for (int k = 0; k < HO / 32; ++k) pp_ld32(tl + 256 + buf * HD + W * HO + 32 * k, d + 32 * k);
#pragma unroll
            for (int k = 0; k < HO / 32; ++k) pp_wait_ld(d + 32 * k);
            const float2 c = make_float2(last, last);
#pragma unroll
            for (int e = 0; e < HO; e += 2) {
                const float2 y = pp_fma2(make_float2(o[e], o[e + 1]), c, make_float2(d[e], d[e + 1]));
                o[e] = y.x;
                o[e + 1] = y.y;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(B.oempty + buf);
            return true;
        };
        for (int j = 0; ok && j < I.nblk; ++j) {
            const int buf = j & 1, ph = (j >> 1) & 1;
            ok = wait(B.s + buf, ph);
            if (!ok) break;
            tc_fence_after();
            const uint32_t tS = tl + buf * 128;
            float s[64];
            pp_ld32(tS + 64 * W, s);
            pp_ld32(tS + 64 * W + 32, s + 32);
            pp_wait_ld(s);
            pp_wait_ld(s + 32);
            const int r0 = I.base + PP_BLOCK * j + 64 * W;
            if (__any_sync(0xffffffffu, r0 < first || r0 + 63 > pos)) pp_mask(s, first - r0, min(pos, r0 + PP_BLOCK) - r0);
            const float mine = pp_largest(s) * down;
            // the other half's largest; past this wait both halves of S are in registers, and P may go over them
            xch[buf * 256 + W * 128 + r] = mine;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(B.x + buf);
            ok = wait(B.x + buf, ph);
            if (!ok) break;
            tc_fence_after();
            const float mt = fmaxf(mine, xch[buf * 256 + (W ^ 1) * 128 + r]);
            const float mn = mt > m + PP_SLACK ? mt : m;
            const float corr = mn == m ? 1.f : pg_ex2(m - mn);
            l *= corr;
            m = mn;
            l += pp_probabilities(s, tS + 32 * W, down, m);
            pp_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(B.p + buf);
            if (j > 0) {
                ok = gather(j - 1);
                if (!ok) break;
            }
            last = corr;
        }
        if (ok && I.nblk > 0) ok = gather(I.nblk - 1);
        if (ok) {  // the two halves' sums, exchanged as one more block's largest would be
            const int buf = I.nblk & 1;
            xch[buf * 256 + W * 128 + r] = l;
            __syncwarp();
            if (lane == 0) mbar_arrive(B.x + buf);
            ok = wait(B.x + buf, (I.nblk >> 1) & 1);
        }
        if (ok) {
            l += xch[(I.nblk & 1) * 256 + (W ^ 1) * 128 + r];
            const float inv = 1.f / l;
            pp_store<float, HD>(a, smem + C::OFF_Q + warp * (64 * HD),
                                real ? (float *)a.out_dev + row * a.out_stride + (size_t)head * HD + W * HO : nullptr, lane,
                                [&](int k, float (&y)[32]) {
#pragma unroll
                                    for (int e = 0; e < 32; ++e) y[e] = l == 0.f ? 0.f : o[32 * k + e] * inv;
                                });
            if (a.lse_dev && W == 0 && real) a.lse_dev[(size_t)row * a.n_heads + head] = pp_lse(m, l);
        }
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
        pp_operands<HD>(P, B, smem, I, warp, lane);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 48;");
        if (warp == 12 && I.nblk > 0) {
            const uint32_t qb = smem_u32(smem + C::OFF_Q), kb = smem_u32(smem + C::OFF_K), vb = smem_u32(smem + C::OFF_V);
            const uint32_t one = pp_elect();
            auto score = [&](int j) {  // S of block j, hi then lo halves of the queries
                const int st = j & 1;
                pp_score<HD>(PP_TMEM + st * 128, qb, kb + st * C::OP, false, one);
                pp_score<HD>(PP_TMEM + st * 128, qb + C::OP, kb + st * C::OP, true, one);
                pp_commit(B.s + st, one);
                pp_commit(B.kempty + st, one);
            };
            bool ok = wait(&B.q, 0);
            for (int j = 0; ok && j < min(2, I.nblk); ++j) {
                ok = wait(B.kfull + j, 0);
                if (!ok) break;
                tc_fence_after();
                score(j);
            }
            for (int j = 0; ok && j < I.nblk; ++j) {
                const int st = j & 1, ph = (j >> 1) & 1;
                ok = wait(B.vfull + st, ph);
                if (ok && j >= 2) ok = wait(B.oempty + st, ph ^ 1);
                if (ok) ok = wait(B.p + st, ph);
                if (!ok) break;
                tc_fence_after();
                pp_value<HD>(PP_TMEM + 256 + st * HD, PP_TMEM + st * 128, vb + st * C::OP, false, one);
                pp_commit(B.o + st, one);
                pp_commit(B.vempty + st, one);
                if (j + 2 < I.nblk) {
                    ok = wait(B.kfull + st, ph ^ 1);
                    if (!ok) break;
                    tc_fence_after();
                    score(j + 2);
                }
            }
            if (!ok) {  // given up: products in flight read shared memory and TMEM until they end
                pp_commit(&B.end, one);
                pg_drain(&B.end, 0);
            }
        } else if (warp == 13) {
            pp_copies<HD>(P, B, smem, I, lane);
        }
    }
    pp_close(B, warp);
}

template <class T, int HD>
static auto prompt_kernel() {
    if constexpr (sizeof(T) == 4) return pages_prompt32_kernel<HD>;
    else return pages_prompt_kernel<T, HD>;
}
template <class T, int HD>
static cudaError_t prompt_prepare() {
    return cudaFuncSetAttribute(prompt_kernel<T, HD>(), cudaFuncAttributeMaxDynamicSharedMemorySize, PpCfg<HD>::SMEM);
}
cudaError_t pages_prompt_prepare() {
    cudaError_t e[6] = {prompt_prepare<float, 64>(), prompt_prepare<float, 128>(), prompt_prepare<__half, 64>(),
                        prompt_prepare<__half, 128>(), prompt_prepare<__nv_bfloat16, 64>(),
                        prompt_prepare<__nv_bfloat16, 128>()};
    for (cudaError_t x : e)
        if (x != cudaSuccess) return x;
    return cudaSuccess;
}

template <class T>
static cudaError_t prompt_t(const PpArgs &P, unsigned grid, cudaStream_t st) {
    if (P.p.hd == 128) prompt_kernel<T, 128>()<<<grid, PP_THREADS, PpCfg<128>::SMEM, st>>>(P);
    else prompt_kernel<T, 64>()<<<grid, PP_THREADS, PpCfg<64>::SMEM, st>>>(P);
    return cudaGetLastError();
}

cudaError_t launch_pages_prompt(const PagesView &p, const er_pages_attention_args &a, int min_rows, int shortfall,
                                cudaStream_t st) {
    const PpArgs P = {p, a, min_rows, shortfall};
    const long long G = a.n_heads / p.KV, rows = a.type == ER_F32 ? 128 : 256;  // query rows of a CTA
    const long long items = ((long long)a.n_tokens * G + rows - 1) / rows + (a.n_seqs < a.n_tokens ? a.n_seqs : a.n_tokens);
    if (items * p.KV > 2147483647ll) return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)(items * p.KV);
    return a.type == ER_F32   ? prompt_t<float>(P, grid, st)
           : a.type == ER_F16 ? prompt_t<__half>(P, grid, st)
                              : prompt_t<__nv_bfloat16>(P, grid, st);
}

cudaError_t set_wait_limit_prompt(unsigned long long ns) { return set_wait_limit_here(ns); }

}  // namespace er
