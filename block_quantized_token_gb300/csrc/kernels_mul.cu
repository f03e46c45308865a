// Products of a block-quantized matrix with any number of tokens, and the adapters of requests beside them:
//   y[t] = W x[t] + scale_a B_a (A_a x[t]),  a = ids[t]
// in up to four kernels on one stream, each started while the one before it ends (what a kernel does before it waits for those
// touches nothing but W):
//   mul_prep    a token's row x[t] times a power of two that brings its largest value to [2^14, 2^15), as fp16 (fp32 rows: as a
//               hi and a lo half, 2^-22), K-major with the 128-byte swizzle, as tiles [64 columns][8 tokens]: any run of
//               tokens of one 64-column step is then one bulk copy.  16-bit rows stay exact (see er_requests.h).
//   with adapters, up to 64 tokens:
//   mul_front   in its place: the same, v[t] = scale_a A_a x[t] and the adapters' steps (below)
//   with adapters, more tokens, behind mul_prep:
//   mul_shrink  v[t] (mma.sync, fp32 sums)
//   mul_expand  the adapters' steps
//   mul_main    the product on the tcgen05 tensor cores, weights dequantised on the way, adapters as further steps of it
// Up to MU_FEW_TOKENS tokens the product is mul_few's (kernels_mul_few.cu), which reads nothing of W twice and needs no tensor
// memory: 32000 x 4096 Q8_0 with 16 bf16 tokens takes 32 us there and 51 us here, 4096 x 4096 7 and 15 us, 128256 x 4096 with 16
// fp32 tokens 172 and 191 us.  Here 64 tokens cost what 16 do (55 us), there twice as much for every 8 more.
//
// Weights.  A value d q has up to 19 bits.  Times a power of two of its row (the largest |d| times the largest code to
// [2^14, 2^15)) it enters as two fp16 numbers: hi = fp16(d q), lo = d q - hi, exactly.  (A scale below some 2^-21 of a row's largest
// is then a subnormal fp16 number; it loses bits, 2^-25 of 2^7 (Q4_0: 2^11) at most, where the largest is 256 (4096) and more, as
// d has none below 2^-24.)
//
// Work.  A tile is 128 rows of W times NT tokens.  Every CTA takes whole tiles first (tile w * grid + cta, so that CTAs that run
// at the same time share tiles of x and W in L2).  Of the tiles left over each is one CTA's, or S CTAs', or all of them are cut
// evenly, whichever mu_share counts as least; sums of a tile that several CTAs share are added in the order of the CTAs by the
// one that comes last.
//
// A CTA's warps, for each step of 64 columns (a unit):
//   warps 0, 3  bulk copies of W, two units of 8 row groups at a time by turns, into a ring
//   warp 1      bulk copies of x's tiles into a ring
//   warp 2      one thread issues the products: D += lo x + hi x (fp32 rows: lo x_hi + hi x_lo + hi x_hi)
//   warps 4 ..  two groups (tiles of up to 64 tokens: four) of four warps that take steps by turns: thread = row = TMEM lane;
//               codes to fp16 hi and lo, to TMEM (A operands)
//   the last 4  D to y: factors taken back, rows brought together through shared memory.  Tiles of up to 128 tokens take D into
//               registers every MU_CHUNK steps (fp32 rows: the tensor cores cut sums off, so they add up two steps alone;
//               four steps take 9 % less time at three times the error), wider ones keep D in TMEM: all columns' products are added
//               there, and 14336 columns' sums are off by some 2e-5 of their size in norm (fp16 results by 2.089e-4 in place of the
//               rounding's 2.078e-4, bf16 results by no more than the rounding).
//
// What bounds it.  Many tokens: the tensor cores.  8192 bf16 tokens x 4096 x 14336 take 1050 us, the hi and lo products alone,
// 1.92 PFLOP, at 1.83 PFLOP/s, 0.95 of what a bf16 library product reaches (tensor pipe active 85 %); call after call, where the
// power limit lowers the clock, 1130 us, 0.99 of the library's sustained rate.  With adapters of five requests 1150 and 1185 us.
// fp32 rows: three products, and a chunk's way through registers (500 x 4096 x 4096 50 us; with adapters 80 us: shrinking
// and expanding are 12 us each under a profiler, the product then has nine steps more).
// Few tokens: each tcgen05.mma with A from TMEM costs some 80 clocks whatever its width, 8 (fp32: 12) of them a step: 0.41 us a
// step of 64 x 128 weights on every SM, 61 fp16 tokens x 32000 x 4096 55 us (2.5 TB/s of W).  An adapters' step costs a tile 1 us, as
// rows of B come straight from global memory (61 fp16 tokens x 11008 x 4096 Q4_0 27 us, with 2 such steps 34 us, with 14 46 us).
#include <cuda_bf16.h>

#include "gemv_core.cuh"
#include "pages.cuh"
#include "requests.h"
#include "tcgen05.cuh"
#include "unit_rows.cuh"

namespace er {

constexpr int MU_SMALL_TOKENS = 64;  // tiles up to this have four groups of warps for the weights, larger ones two
constexpr int MU_REG_TOKENS = 128;  // tiles up to this keep their sums in registers
constexpr int MU_MAX_TOKENS = 256;  // (fp32 rows: MU_REG_TOKENS)
constexpr int MU_EXTRA = 16;        // steps of 64 that adapters may add to a tile
// what sharing a tile costs, in steps: joining it, a CTA that takes part, and tiles cut anywhere (CTAs with pieces of two)
constexpr double MU_JOIN = 6, MU_JOIN_EACH = 1, MU_SPREAD = 18;
constexpr int MU_FEW_TOKENS = 16;   // calls up to this are mul_few's (kernels_mul_few.cu)
constexpr int MU_NA = 4;            // TMEM buffers of A (64 columns each: hi, lo)
constexpr int MU_CHUNK32 = 2;       // steps that the tensor cores add up before registers do, fp32 rows
constexpr int MU_CHUNK16 = 16;      // the same, 16-bit rows in small tiles
constexpr int MU_STAGE = 32 * 132;  // floats: 32 tokens' 128 rows on their way out
constexpr int MU_MAX_RING = 10;
constexpr int MU_SMEM = 231424;

constexpr int MU_SU = 2;            // units of a bulk copy
constexpr int MU_PRODUCERS = 2;     // warps that copy W

// bytes of a row group in a slot: rounded up to 128 and then 16 more, so that 8 row groups start in 8 bank groups
template <int QT>
constexpr int mu_rgs() { return (MU_SU * QTraits<QT>::unit_bytes + 127) / 128 * 128 + 16; }

struct MulArgs {
    const uint8_t *W;
    const float *row_up;
    int R, UPR, rows, n;
    int NT, ntl, MT, waves, rem, grid, grem;  // grem: CTAs that share the left-over tiles
    int rs;                                   // slots of W's ring
    const uint8_t *x;
    size_t plane;  // bytes of a plane of x
    int natoms;
    const float *tok_up, *tok_down;
    AdaptersView ad;
    const int32_t *ids;  // NULL: no adapters
    const float *v;      // [n][r16]
    void *y;
    long long y_stride;
    int type;
    // adapters' steps of the tiles of tokens: operand behind x's, entries of 16 columns, their number
    const int2 *ksteps;
    const int *nksteps;  // NULL: none
    float *part;
    int *cnt;
    int *flags;
    int shortfall;  // tests of the give-up path: arrivals that CTA 0 waits for in vain
};

// ---------------------------------------------------------------------------------------------------
// factors of W's rows, at create time
// ---------------------------------------------------------------------------------------------------
__global__ void mul_row_up_kernel(const uint8_t *W, int qt, int UPR, int R, float *up) {
    const int row = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32, lane = threadIdx.x & 31;
    if (row >= 16 * R) return;
    float m = 0.f;
    for (int b = lane; b < 2 * UPR; b += 32) {
        const uint8_t *u = W + ((size_t)(row >> 4) * UPR + (b >> 1)) * unit_bytes_of(qt);
        const float d = fabsf(__half2float(*reinterpret_cast<const __half *>(u + scale_offset(qt, row & 15, b & 1))));
        if (isfinite(d)) m = fmaxf(m, d);
    }
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (lane == 0) {
        // codes reach 128 (Q8_0) or 8: m * that is at most 2^15
        int e = 0;
        if (m > 0.f) {
            frexpf(m, &e);
            e = (qt == Q8_0 ? 8 : 12) - e;
        }
        up[row] = ldexpf(1.f, e);
    }
}

cudaError_t launch_matrix_row_up(const Mat &m, float *up, cudaStream_t st) {
    mul_row_up_kernel<<<(16 * m.R + 7) / 8, 256, 0, st>>>(m.d, m.qt, m.UPR, m.R, up);
    return cudaGetLastError();
}

// ---------------------------------------------------------------------------------------------------
// adapters into their slots
// ---------------------------------------------------------------------------------------------------
// the power of two that brings a largest magnitude to [2^14, 2^15), within +-2^126
ER_DEV int mu_exponent(float top) {
    int e = 0;
    if (top > 0.f) {
        frexpf(top, &e);
        e = min(max(15 - e, -126), 126);
    }
    return e;
}
ER_DEV float mu_pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

template <class T>
__global__ void adapters_a_kernel(AdaptersView v, int slot, int rank, int cols, float scale, const T *a) {
    __shared__ float tops[8];
    const int j = blockIdx.x, tid = threadIdx.x;
    __half *out = reinterpret_cast<__half *>(const_cast<uint8_t *>(v.a)) + ((size_t)slot * v.r16 + j) * v.Kp;
    float top = 0.f;
    if (j < rank)
        for (int k = tid; k < cols; k += 256) {
            const float x = fabsf(pg_ld<T>(a + (size_t)j * cols + k));
            if (isfinite(x)) top = fmaxf(top, x);
        }
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((tid & 31) == 0) tops[tid >> 5] = top;
    __syncthreads();
    for (int i = 0; i < 8; ++i) top = fmaxf(top, tops[i]);
    const int e = mu_exponent(top);
    const float up = mu_pow2(e);
    for (int k = tid; k < v.Kp; k += 256)
        out[k] = __float2half_rn(j < rank && k < cols ? pg_ld<T>(a + (size_t)j * cols + k) * up : 0.f);
    if (tid == 0) {
        const_cast<float *>(v.down)[(size_t)slot * v.r16 + j] = mu_pow2(-e) * scale;
        if (j == 0) {
            const_cast<int *>(v.rank)[slot] = (rank + 15) & ~15;
            const_cast<int *>(v.wild)[slot] = 0;
        }
    }
}

// Behind adapters_a_kernel, which empties the slot's `wild`.  B's rows are operands that all tokens of a tile meet (with zeros where
// a token has another adapter): a value that is infinite or NaN there, as it is or times the factor of W's row (2^35 at most), would be
// NaN for all of them.  Tiles with such an adapter add it by mu_adapters.
constexpr float MU_WILD = 0x1p92f;
__global__ void adapters_b_kernel(AdaptersView v, int slot, int rank, const uint16_t *b) {
    uint16_t *out = reinterpret_cast<uint16_t *>(const_cast<uint8_t *>(v.b)) + (size_t)slot * v.rows * v.r16;
    const size_t n = (size_t)v.rows * v.r16;
    for (size_t i = blockIdx.x * (size_t)blockDim.x + threadIdx.x; i < n; i += (size_t)gridDim.x * blockDim.x) {
        const int row = (int)(i / v.r16), j = (int)(i - (size_t)row * v.r16);
        const uint16_t w = j < rank ? b[(size_t)row * rank + j] : (uint16_t)0;
        const float f = v.bf16 ? __uint_as_float((uint32_t)w << 16) : __half2float(__ushort_as_half(w));
        if (!(fabsf(f) < MU_WILD)) atomicOr(const_cast<int *>(v.wild) + slot, 1);
        out[i] = w;
    }
}

__global__ void adapters_clear_kernel(AdaptersView v, int slot) { const_cast<int *>(v.rank)[slot] = 0; }

cudaError_t launch_adapters_set(const AdaptersView &v, int slot, int rank, int cols, float scale, const void *a, const void *b,
                                cudaStream_t st) {
    if (v.bf16)
        adapters_a_kernel<<<v.r16, 256, 0, st>>>(v, slot, rank, cols, scale, reinterpret_cast<const __nv_bfloat16 *>(a));
    else
        adapters_a_kernel<<<v.r16, 256, 0, st>>>(v, slot, rank, cols, scale, reinterpret_cast<const __half *>(a));
    adapters_b_kernel<<<(unsigned)min((size_t)1024, ((size_t)v.rows * v.r16 + 255) / 256), 256, 0, st>>>(
        v, slot, rank, reinterpret_cast<const uint16_t *>(b));
    return cudaGetLastError();
}

cudaError_t launch_adapters_clear(const AdaptersView &v, int slot, cudaStream_t st) {
    adapters_clear_kernel<<<1, 1, 0, st>>>(v, slot);
    return cudaGetLastError();
}

// two 16-bit values as fp32
template <bool BF16>
ER_DEV float2 mu_pair(uint32_t w) {
    if (BF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// ---------------------------------------------------------------------------------------------------
// a token's row into the operand
// ---------------------------------------------------------------------------------------------------
// 8 values from p
template <class T>
ER_DEV void mu_load8(const T *p, bool vec, float (&v)[8]) {
    __align__(16) T r[8];
    if (vec) {
        constexpr int N = sizeof(T) / 2;
#pragma unroll
        for (int i = 0; i < N; ++i) reinterpret_cast<uint4 *>(r)[i] = reinterpret_cast<const uint4 *>(p)[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = p[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = pg_ld<T>(r + i);
}

// The CTA's largest magnitude (as bits; above every number's for an infinity or a NaN) to the row's exponent, or MU_BAD.
constexpr int MU_BAD = 1 << 20;
ER_DEV int mu_top_exponent(uint32_t top, uint32_t *tops) {
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, tops[i]);
    return top >= 0x7F800000u ? MU_BAD : mu_exponent(__uint_as_float(top));
}
// A row's factor alone (NaN: the row holds an infinity or a NaN); the CTA may use `tops` again when it returns.
template <class T>
ER_DEV float mu_row_factor(const T *row, int K, uint32_t *tops) {
    const bool vec = ((uintptr_t)row & 15) == 0;
    uint32_t top = 0;
    float v[8];
    for (int ch = threadIdx.x; ch < K / 8; ch += 256) {
        mu_load8(row + 8 * ch, vec, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    }
    const int e = mu_top_exponent(top, tops);
    __syncthreads();
    return e == MU_BAD ? NAN : mu_pow2(e);
}
// Row t by a CTA of 256 threads: its factors and its place in the operand.  A row with an infinity
// or a NaN becomes NaN by its factors, its operand zeros.
template <class T>
ER_DEV void mu_prep_row(const T *row, int t, int K, int UPR, uint8_t *out, size_t plane, int natoms, float *tok_up, float *tok_down,
                        uint32_t *tops) {
    constexpr bool LO = sizeof(T) == 4;
    const int tid = threadIdx.x;
    const bool vec = ((uintptr_t)row & 15) == 0;
    uint32_t top = 0;
    float v[8], first[2][8];  // (the first two of a thread are kept, the others read again)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) first[c][i] = 0.f;
        if (tid + 256 * c < K / 8) mu_load8(row + 8 * (tid + 256 * c), vec, first[c]);
    }
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(first[c][i]) & 0x7FFFFFFFu);
#pragma unroll 2
    for (int ch = tid + 512; ch < K / 8; ch += 256) {
        mu_load8(row + 8 * ch, vec, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
    }
    const int e = mu_top_exponent(top, tops);
    const bool bad = e == MU_BAD;
    const float up = mu_pow2(bad ? 0 : e);
    if (tid == 0) {
        tok_up[t] = bad ? NAN : up;
        tok_down[t] = bad ? NAN : mu_pow2(-e);
    }
    uint8_t *base = out + (size_t)(t >> 3) * 1024 + (t & 7) * 128;
    auto put = [&](int ch, bool there, const float (&v)[8]) {
        uint32_t hi[4];
        [[maybe_unused]] uint32_t lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float y0 = there ? v[2 * i] * up : 0.f, y1 = there ? v[2 * i + 1] * up : 0.f;
            hi[i] = pg_pack(y0, y1);
            if constexpr (LO) {
                const float2 z = __half22float2(*reinterpret_cast<const __half2 *>(&hi[i]));
                lo[i] = pg_pack(y0 - z.x, y1 - z.y);
            }
        }
        uint8_t *d = base + (size_t)(ch >> 3) * natoms * 1024 + (((ch & 7) ^ (t & 7)) << 4);
        *reinterpret_cast<uint4 *>(d) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        if constexpr (LO) *reinterpret_cast<uint4 *>(d + plane) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    };
#pragma unroll
    for (int c = 0; c < 2; ++c)
        if (tid + 256 * c < 8 * UPR) put(tid + 256 * c, !bad, first[c]);
    for (int ch = tid + 512; ch < 8 * UPR; ch += 256) {
        const bool there = ch < K / 8 && !bad;
        if (there) mu_load8(row + 8 * ch, vec, v);
        put(ch, there, v);
    }
}

template <class T>
__global__ void __launch_bounds__(256) mul_prep_kernel(const T *x, long long stride, int K, int UPR, uint8_t *out, size_t plane,
                                                       int natoms, float *tok_up, float *tok_down, int *cnt, int ncnt) {
    __shared__ uint32_t tops[8];
    const int t = blockIdx.x;
    pdl_launch_dependents();
    pdl_wait();
    mu_prep_row(x + (size_t)t * stride, t, K, UPR, out, plane, natoms, tok_up, tok_down, tops);
    for (long long i = t * 256ll + threadIdx.x; i < ncnt; i += gridDim.x * 256ll) cnt[i] = 0;  // (256 times 2^23 tokens pass 31 bits)
}

// Adapters as steps of the product: for every kind of adapter among a tile's tokens, every 16 of its rank and every pair of
// pieces, 16 columns in A (rows of B_a, bf16) and in the operand (v of the tokens that have it, else 0).  v enters as bf16 pieces,
// two (2^-17 of the adapter's share of a 16-bit result) or for fp32 three; B_a in fp16 as two pieces, exactly.  The last pieces
// do not meet.  Four such entries are a step of 64 columns.  A tile with more kinds than MU_EXTRA steps hold, or with one whose B holds
// what is no number (AdaptersView::wild), has none (nksteps -1), and its adapters are added row by row (mu_adapters): 15 steps take
// 61 fp16 tokens x 11008 x 4096 46 us, row by row 59; 36 entries 500 fp32 tokens x 4096 x 4096 80 us and 169 (more than fit: 176
// to 187).  With room for 32 steps 24 of them would take the first 53 us where 16 adapters of rank 32 now take 60, and calls of few
// kinds 4 us more (512 bf16 tokens with five of rank 16: 60 to 64 us).
struct MuKinds {
    int kind[256], start[256], total;  // of a tile's tokens: adapter, the first entry of the kind where this token is its first
    int entry_kind[4 * MU_EXTRA], entry_pair[4 * MU_EXTRA], entry_col[4 * MU_EXTRA];
};
__host__ __device__ constexpr int mu_pairs(bool bf16, int planes) { return bf16 ? planes + 1 : 2 * planes + 1; }
// pair h: pieces of v and of B_a
ER_DEV int mu_pair_v(int h, int planes) { return h <= planes ? h : h - planes - 1; }
ER_DEV int mu_pair_b(int h, int planes) { return h <= planes ? 0 : 1; }
// By the CTA's threads: K for tokens tok0 .. tok0 + nt - 1 (at most 256) of n.
ER_DEV void mu_kinds(MuKinds &K, const int32_t *ids, const AdaptersView &ad, int tok0, int nt, int n, int planes, int *flags) {
    const int t = threadIdx.x, per = mu_pairs(ad.bf16, planes);
    int id = t < nt && tok0 + t < n ? ids[tok0 + t] : -1;
    if (id >= ad.slots) {
        atomicOr(flags, ER_MUL_FLAG_RANGE);
        id = -1;
    }
    const int r = id >= 0 ? ad.rank[id] : 0;
    if (!r) id = -1;
    K.kind[t] = id;
    for (int i = t; i < 4 * MU_EXTRA; i += 256) K.entry_kind[i] = -1, K.entry_pair[i] = K.entry_col[i] = 0;
    const int wild = __syncthreads_or(id >= 0 && ad.wild[id]);
    bool first = id >= 0;
    for (int i = 0; i < t && first; ++i) first = K.kind[i] != id;
    const int mine = first ? r / 16 * per : 0;
    K.start[t] = mine;
    __syncthreads();
    if (t < 32) {  // sums before: eight tokens a lane
        int s = 0, v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = s, s += K.start[8 * t + i];
        int incl = s;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, incl, o);
            if (t >= o) incl += u;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) K.start[8 * t + i] = v[i] + incl - s;
        if (t == 31) K.total = wild || incl > 4 * MU_EXTRA ? -1 : incl;
    }
    __syncthreads();
    if (first && K.total >= 0)
        for (int i = 0; i < mine; ++i) {
            const int e = K.start[t] + i;
            K.entry_kind[e] = id;
            K.entry_pair[e] = i % per;
            K.entry_col[e] = i / per * 16;
        }
    __syncthreads();
}
// entry e for the product's warps: adapter and piece of B_a, or -1; first column
ER_DEV int2 mu_kstep(const MuKinds &K, int e, int planes) {
    return make_int2(K.entry_kind[e] < 0 ? -1 : K.entry_kind[e] << 1 | mu_pair_b(K.entry_pair[e], planes), K.entry_col[e]);
}
// piece k of two values, bf16
ER_DEV uint32_t mu_piece(float x, float y, int k) {
    __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    for (; k; --k) {
        x -= __low2float(h);
        y -= __high2float(h);
        h = __floats2bfloat162_rn(x, y);
    }
    return *reinterpret_cast<const uint32_t *>(&h);
}

// The same and v[t] = scale A x of the token's adapter, 8 of the rank a CTA (token, part of the rank): for few tokens, where a
// kernel less counts and adapters are hardly shared.  A CTA's threads take 8 columns each of the row as it is in memory.  With
// nksteps it also writes the token's places of the adapters' steps.
constexpr int MU_FRONT_TOKENS = 64;
template <class T>
__global__ void __launch_bounds__(256) mul_front_kernel(const T *x, long long stride, int K, int UPR, uint8_t *out, size_t plane,
                                                        int natoms, float *tok_up, float *tok_down, int *cnt, int ncnt,
                                                        const int32_t *ids, AdaptersView ad, float *v, int2 *ksteps, int *nksteps, int *flags) {
    constexpr int PLANES = sizeof(T) == 4 ? 2 : 1;
    __shared__ uint32_t tops[8];
    __shared__ float sums[8][8], vs[8];
    __shared__ MuKinds kinds;
    const int t = blockIdx.x, j0 = blockIdx.y * 8, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_launch_dependents();
    pdl_wait();
    const T *row = x + (size_t)t * stride;
    const int id = ids[t];
    const bool any = id >= 0 && id < ad.slots && ad.rank[id] > j0;
    const bool write = blockIdx.y == 0;
    if (any) {
        const bool vec = ((uintptr_t)row & 15) == 0;
        const uint4 *a = reinterpret_cast<const uint4 *>(ad.a + (((size_t)id * ad.r16 + j0) * ad.Kp) * 2);
        // where a sum overflows (A's rows reach 2^15, x may be next to float32's largest), x enters times 2^-60
        for (float down = 1.f;; down = 0x1p-60f) {
            float s[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] = 0.f;
            for (int ch = tid; ch < K / 8; ch += 256) {
                uint4 w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = __ldg(a + (size_t)j * (ad.Kp / 8) + ch);
                float f[8];
                mu_load8(row + 8 * ch, vec, f);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] *= down;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 a0 = mu_pair<false>(w[j].x), a1 = mu_pair<false>(w[j].y), a2 = mu_pair<false>(w[j].z),
                                 a3 = mu_pair<false>(w[j].w);
                    float p = a0.x * f[0], q = a2.x * f[4];
                    p = fmaf(a0.y, f[1], p);
                    q = fmaf(a2.y, f[5], q);
                    p = fmaf(a1.x, f[2], p);
                    q = fmaf(a3.x, f[6], q);
                    p = fmaf(a1.y, f[3], p);
                    q = fmaf(a3.y, f[7], q);
                    s[j] += p + q;
                }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
#pragma unroll
                for (int o = 16; o; o >>= 1) s[j] += __shfl_xor_sync(0xffffffffu, s[j], o);
                if (lane == 0) sums[warp][j] = s[j];
            }
            __syncthreads();
            float r = 0.f;
            if (tid < 8)
                for (int w = 0; w < 8; ++w) r += sums[w][tid];
            if (tid < 8) vs[tid] = v[(size_t)t * ad.r16 + j0 + tid] = r * (ad.down[(size_t)id * ad.r16 + j0 + tid] / down);
            if (!__syncthreads_or(!isfinite(r)) || down < 1.f) break;
        }
    }
    if (nksteps) {
        if (!write && !any) return;
        mu_kinds(kinds, ids, ad, 0, gridDim.x, gridDim.x, PLANES, flags);
        const float up = mu_row_factor(row, K, tops);
        const int total = kinds.total;
        if (t == 0 && write) {
            if (tid == 0) *nksteps = total;
            if (tid < 4 * MU_EXTRA) ksteps[tid] = mu_kstep(kinds, tid, PLANES);
        }
        // 8 columns a thread: of its own kind those of this CTA's part of the rank, of the others zeros
        for (int i = tid; i < (total + 3) / 4 * 8; i += 256) {
            const int e = i >> 1;
            const bool own = id >= 0 && kinds.entry_kind[e] == id && any;
            if (own ? kinds.entry_col[e] + 8 * (i & 1) != j0 : !write) continue;
            uint32_t w[4] = {0, 0, 0, 0};
            if (own && !isnan(up)) {
                const int piece = mu_pair_v(kinds.entry_pair[e], PLANES);
#pragma unroll
                for (int j = 0; j < 4; ++j) w[j] = mu_piece(vs[2 * j] * up, vs[2 * j + 1] * up, piece);
            }
            *reinterpret_cast<uint4 *>(out + ((size_t)(UPR + (e >> 2)) * natoms + (t >> 3)) * 1024 + (t & 7) * 128 +
                                       (((i & 7) ^ (t & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    if (write) mu_prep_row(row, t, K, UPR, out, plane, natoms, tok_up, tok_down, tops);
    if (write)
        for (int i = t * 256 + tid; i < ncnt; i += gridDim.x * 256) cnt[i] = 0;
}

// ---------------------------------------------------------------------------------------------------
// v = scale A x: CTA (8 tokens, 16 of the rank, the z-th adapter among the tokens), warps share K
// ---------------------------------------------------------------------------------------------------
template <bool LO>
__global__ void __launch_bounds__(256) mul_shrink_kernel(const uint8_t *x, size_t plane, int natoms, int UPR, int n,
                                                         const float *tok_down, const int32_t *ids, AdaptersView ad, float *v) {
    __shared__ float sums[8][16][8];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int atom = blockIdx.x, j0 = blockIdx.y * 16;
    pdl_launch_dependents();
    pdl_wait();  // (also for a CTA that does nothing: this kernel's end stands for the one before it)
    // the z-th distinct adapter of the group
    const int tok = 8 * atom + (lane & 7);
    int id = tok < n ? ids[tok] : -1;
    if (id >= ad.slots) id = -1;
    const int rank = id >= 0 ? ad.rank[id] : 0;
    if (rank <= j0) id = -1;
    const unsigned same = __match_any_sync(0xffffffffu, id);
    const bool leader = lane < 8 && id >= 0 && (__ffs(same) - 1) == lane;
    unsigned leaders = __ballot_sync(0xffffffffu, leader);
    for (int z = 0; z < (int)blockIdx.z; ++z) leaders &= leaders - 1;
    if (!leaders) return;
    const int pick = __ffs(leaders) - 1;
    const unsigned mine = __shfl_sync(0xffffffffu, same, pick) & 0xFFu;
    id = __shfl_sync(0xffffffffu, id, pick);
    const uint8_t *a0 = ad.a + (((size_t)id * ad.r16 + j0 + g) * ad.Kp + 8 * t) * 2;
    const uint8_t *a1 = a0 + (size_t)8 * ad.Kp * 2;
    const uint8_t *xr = x + (size_t)atom * 1024 + g * 128;
    float d0[4] = {0.f, 0.f, 0.f, 0.f}, d1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
    for (int u = warp; u < UPR; u += 8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // 32 columns: lane t holds 8 of them
            const uint8_t *xp = xr + (size_t)u * natoms * 1024 + (((4 * h + t) ^ g) << 4);
            const uint4 b = __ldcg(reinterpret_cast<const uint4 *>(xp));
            const uint4 p = __ldg(reinterpret_cast<const uint4 *>(a0 + u * 128 + h * 64));
            const uint4 q = __ldg(reinterpret_cast<const uint4 *>(a1 + u * 128 + h * 64));
            const uint32_t A0[4] = {p.x, q.x, p.y, q.y}, A1[4] = {p.z, q.z, p.w, q.w};
            mma_16816(d0, A0, b.x, b.y, d0);
            mma_16816(d1, A1, b.z, b.w, d1);
            if (LO) {
                const uint4 l = __ldcg(reinterpret_cast<const uint4 *>(xp + plane));
                mma_16816(d0, A0, l.x, l.y, d0);
                mma_16816(d1, A1, l.z, l.w, d1);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) sums[warp][g + 8 * (i >> 1)][2 * t + (i & 1)] = d0[i] + d1[i];
    __syncthreads();
    if (threadIdx.x < 128) {
        const int j = threadIdx.x & 15, c = threadIdx.x >> 4, to = 8 * atom + c;
        if ((mine >> c) & 1) {
            float s = 0.f;
            for (int w = 0; w < 8; ++w) s += sums[w][j][c];
            v[(size_t)to * ad.r16 + j0 + j] = s * ad.down[(size_t)id * ad.r16 + j0 + j] * tok_down[to];
        }
    }
}

// ---------------------------------------------------------------------------------------------------
// the adapters' steps of many tokens: CTA (tile of tokens, step), thread = token
// ---------------------------------------------------------------------------------------------------
__global__ void __launch_bounds__(256) mul_expand_kernel(uint8_t *x, int natoms, int UPR, int n, int NT, int planes, const float *tok_up,
                                                         const int32_t *ids, AdaptersView ad, const float *v, int2 *ksteps,
                                                         int *nksteps, int *flags) {
    __shared__ MuKinds kinds;
    const int tn = blockIdx.x, e = blockIdx.y, t = threadIdx.x, tok = tn * NT + t;
    pdl_launch_dependents();
    pdl_wait();  // (also for a CTA that does nothing: this kernel's end stands for the ones before it)
    mu_kinds(kinds, ids, ad, tn * NT, NT, n, planes, flags);
    if (e == 0 && t == 0) nksteps[tn] = kinds.total;
    if (kinds.total <= 4 * e) return;
    if (t < 4) ksteps[((size_t)tn * MU_EXTRA + e) * 4 + t] = mu_kstep(kinds, 4 * e + t, planes);
    if (t >= NT) return;
    const int id = kinds.kind[t];
    uint8_t *base = x + ((size_t)(UPR + e) * natoms + (tn * NT + t) / 8) * 1024 + (t & 7) * 128;
    const float up = id >= 0 ? tok_up[tok] : 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = 0;
        if (id >= 0 && kinds.entry_kind[4 * e + k] == id && !isnan(up)) {
            const float4 *p = reinterpret_cast<const float4 *>(v + (size_t)tok * ad.r16 + kinds.entry_col[4 * e + k]);
            const int piece = mu_pair_v(kinds.entry_pair[4 * e + k], planes);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 f = __ldcg(p + i);
                w[2 * i] = mu_piece(f.x * up, f.y * up, piece);
                w[2 * i + 1] = mu_piece(f.z * up, f.w * up, piece);
            }
        }
        *reinterpret_cast<uint4 *>(base + (((2 * k) ^ (t & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        *reinterpret_cast<uint4 *>(base + (((2 * k + 1) ^ (t & 7)) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// ---------------------------------------------------------------------------------------------------
// the product
// ---------------------------------------------------------------------------------------------------
struct MuBars {
    uint64_t wfull[MU_MAX_RING], wempty[MU_MAX_RING];
    // a step's operands, A in TMEM and x's tile, share their barriers: one wait and one commit a step for the products
    uint64_t full[MU_NA], empty[MU_NA], dfull[4], dempty[4], end, meet;
    uint32_t tmem;
    int stop, last;
};

// The items of a CTA in their order: a tile and its steps u0 .. u1 - 1.
struct MuWalk {
    int w, tile, u0, u1;
    long long cur, end;
    ER_DEV explicit MuWalk(const MulArgs &a) : w(0), tile(0), u0(0), u1(0), cur(0), end(0) {
        const long long units = (long long)a.rem * a.UPR;
        if ((int)blockIdx.x < a.grem) {
            cur = blockIdx.x * units / a.grem;
            end = (blockIdx.x + 1) * units / a.grem;
        }
    }
    ER_DEV bool next(const MulArgs &a) {
        if (w < a.waves) {
            tile = w++ * a.grid + blockIdx.x;
            u0 = 0;
            u1 = a.UPR;
            return true;
        }
        if (cur >= end) return false;
        const int t = (int)(cur / a.UPR);
        tile = a.waves * a.grid + t;
        u0 = (int)(cur - (long long)t * a.UPR);
        u1 = (int)min((long long)a.UPR, u0 + end - cur);
        cur += u1 - u0;
        return true;
    }
};
// CTAs first .. first + n - 1 share a left-over tile (number t among them); where CTA j's sums of it lie
struct MuShare {
    int t, first, n;
    long long units;
    ER_DEV MuShare(const MulArgs &a, int tile) : t(tile - a.waves * a.grid), first(0), n(1), units((long long)a.rem * a.UPR) {
        if (t < 0) return;
        const long long u = (long long)t * a.UPR;
        first = (int)(((u + 1) * a.grem - 1) / units);
        n = (int)(((u + a.UPR) * a.grem - 1) / units) - first + 1;
    }
    ER_DEV size_t slot(const MulArgs &a, int j) const {
        return 2 * (size_t)j + (j * units / a.grem <= (long long)t * a.UPR ? 1 : 0);
    }
};

// a walk over a ring's slots
struct MuRing {
    int size, slot;
    uint32_t par;  // parity of this use of the slot
    unsigned n;    // uses so far
    bool again;    // the slot has been used before
    ER_DEV explicit MuRing(int size) : size(size), slot(0), par(0), n(0), again(false) {}
    ER_DEV void step() {
        ++n;
        if (++slot == size) {
            slot = 0;
            par ^= 1;
            again = true;
        }
    }
};

ER_DEV int mu_pos(int row) { return row + (row >> 5); }  // (32 lanes' rows, 16 apart, then lie in 32 banks)

// block b of a row's unit as 16 fp16 pairs (tw_unit_cols, one block)
template <int QT>
ER_DEV void mu_block_cols(uint32_t base, int b, uint32_t sel, uint32_t sh, uint32_t (&col)[16]) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        if (QT == Q8_0) {
            const uint4 c = lds128(base + 512 * b + 16 * t);
            col[t] = h2_sub(prmt(c.x, 0x64646464u, sel), 0x64806480u);
            col[4 + t] = h2_sub(prmt(c.y, 0x64646464u, sel), 0x64806480u);
            col[8 + t] = h2_sub(prmt(c.z, 0x64646464u, sel), 0x64806480u);
            col[12 + t] = h2_sub(prmt(c.w, 0x64646464u, sel), 0x64806480u);
        } else {
            const uint2 c = lds64(base + 16 * t + 8 * b);
            const uint32_t x = c.x >> sh, y = c.y >> sh;
            col[t] = tw_q4_pair(x);
            col[4 + t] = tw_q4_pair(x >> 8);
            col[8 + t] = tw_q4_pair(y);
            col[12 + t] = tw_q4_pair(y >> 8);
        }
    }
}

// Adapters' share of 32 tokens from `tok`, for this thread's row, times the factors of its sums, into its places of `stage`.
// Only tokens of `lo` .. `hi` - 1 of the tile's (those of a CTA that shares the tile).  False: none has any (nothing is written).
// Four tokens at a time: their loads (a row of B, the token's v, which all rows share) are on their way together.
template <bool BF16>
ER_DEV bool mu_adapters(const MulArgs &a, float *stage, int tok, int ntok, int row, int pos, float up, int lo, int hi, int lane) {
    int id = -1, rank = 0;
    if (lane < ntok) {
        id = a.ids[tok + lane];
        if (id >= a.ad.slots) {
            atomicOr(a.flags, ER_MUL_FLAG_RANGE);
            id = -1;
        }
        if (id >= 0) rank = a.ad.rank[id];
        if (tok + lane < lo || tok + lane >= hi) rank = 0;
    }
    const unsigned any = __ballot_sync(0xffffffffu, rank > 0);
    if (!any) return false;
    const int r = min(row, a.rows - 1);
    for (int c = 0; c < 32; c += 4) {
        float s[4] = {0.f, 0.f, 0.f, 0.f};
        const unsigned four = (any >> c) & 15u;
        if (four) {
            const int some = c + __ffs(four) - 1;  // one with an adapter: what those without it load, and drop
            int rk[4], most = 0;
            const uint4 *bp[4];
            const float4 *vp[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                rk[i] = __shfl_sync(0xffffffffu, rank, c + i);
                const int from = rk[i] ? c + i : some, slot = __shfl_sync(0xffffffffu, id, from);
                bp[i] = reinterpret_cast<const uint4 *>(a.ad.b + (((size_t)slot * a.ad.rows + r) * a.ad.r16) * 2);
                vp[i] = reinterpret_cast<const float4 *>(a.v + (size_t)(tok + from) * a.ad.r16);
                most = max(most, rk[i]);
            }
            for (int j = 0; j < most; j += 16) {
                uint4 b[4][2];
                float4 v[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    b[i][0] = __ldg(bp[i] + j / 8);
                    b[i][1] = __ldg(bp[i] + j / 8 + 1);
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[i][k] = __ldcg(vp[i] + j / 4 + k);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float t = 0.f, w = 0.f;
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float2 b0 = mu_pair<BF16>(b[i][k].x), b1 = mu_pair<BF16>(b[i][k].y), b2 = mu_pair<BF16>(b[i][k].z),
                                     b3 = mu_pair<BF16>(b[i][k].w);
                        t = fmaf(b0.x, v[i][2 * k].x, t);
                        w = fmaf(b2.x, v[i][2 * k + 1].x, w);
                        t = fmaf(b0.y, v[i][2 * k].y, t);
                        w = fmaf(b2.y, v[i][2 * k + 1].y, w);
                        t = fmaf(b1.x, v[i][2 * k].z, t);
                        w = fmaf(b3.x, v[i][2 * k + 1].z, w);
                        t = fmaf(b1.y, v[i][2 * k].w, t);
                        w = fmaf(b3.y, v[i][2 * k + 1].w, w);
                    }
                    if (j < rk[i]) s[i] += t + w;
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i] = rk[i] ? s[i] * a.tok_up[tok + c + i] * up : 0.f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) stage[(c + i) * 132 + pos] = s[i];
    }
    return true;
}

// a pair of an adapter's values times `up`, as bf16 (fp16 values: its hi half, or what that leaves)
ER_DEV uint32_t mu_b_bf16(uint32_t w, int bf16, int lo, float up) {
    float2 f = bf16 ? mu_pair<true>(w) : mu_pair<false>(w);
    f.x *= up;
    f.y *= up;
    __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
    if (lo) h = __floats2bfloat162_rn(f.x - __low2float(h), f.y - __high2float(h));
    return *reinterpret_cast<const uint32_t *>(&h);
}

// `ntok` tokens' 128 rows from `stage` to y, warp q every fourth token: a lane two neighbouring rows of each half, as one store
// where y's rows allow it
template <class T>
ER_DEV void mu_rows_out(const MulArgs &a, T *y, const float *stage, int tok, int ntok, int row0, float td, int q, int lane) {
    const bool pairs = ((uintptr_t)y | (size_t)a.y_stride * sizeof(T) | (size_t)row0 * sizeof(T)) % (2 * sizeof(T)) == 0;
    const int row = 2 * lane, left = a.rows - row0;
    const float *from = stage + row + (row >> 5);
    y += (long long)tok * a.y_stride + row0 + row;
    for (int c = q; c < ntok; c += 4) {
        const float f = __shfl_sync(0xffffffffu, td, c);
        T *to = y + (long long)c * a.y_stride;
#pragma unroll
        for (int k = 0; k < 2; ++k) {  // rows 64 k + row, + 1: places 66 k on
            __align__(8) T v[2] = {pg_cvt<T>(from[c * 132 + 66 * k] * f), pg_cvt<T>(from[c * 132 + 66 * k + 1] * f)};
            if (pairs && row + 64 * k + 1 < left) {
                if constexpr (sizeof(T) == 4) *reinterpret_cast<uint2 *>(to + 64 * k) = *reinterpret_cast<const uint2 *>(v);
                else *reinterpret_cast<uint32_t *>(to + 64 * k) = *reinterpret_cast<const uint32_t *>(v);
            } else {
                if (row + 64 * k < left) to[64 * k] = v[0];
                if (row + 64 * k + 1 < left) to[64 * k + 1] = v[1];
            }
        }
    }
}

// TOK: tokens whose sums the registers hold (0: tiles of more than MU_REG_TOKENS, whose sums stay in TMEM)
template <int TOK>
constexpr int mu_groups() { return TOK == MU_SMALL_TOKENS ? 4 : 2; }
template <int TOK>
constexpr int mu_threads() { return (8 + 4 * mu_groups<TOK>()) * 32; }

template <int QT, bool F32, int TOK>
__global__ void __launch_bounds__(mu_threads<TOK>(), 1) mul_main_kernel(const __grid_constant__ MulArgs a) {
    constexpr int UB = QTraits<QT>::unit_bytes, QB = QTraits<QT>::quant_bytes, RGS = mu_rgs<QT>(), SLOT = 8 * RGS;
    constexpr bool REG = TOK > 0;
    constexpr int GROUPS = mu_groups<TOK>(), OUT = 4 + 4 * GROUPS;  // OUT: the first of the sums' warps
    constexpr int CHUNK = F32 ? MU_CHUNK32 : MU_CHUNK16;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    const int bsz = a.NT * 128 * (F32 ? 2 : 1);
    uint8_t *ring_b = smem, *ring_w = smem + MU_NA * bsz;
    float *stage = reinterpret_cast<float *>(ring_w + a.rs * SLOT);
    MuBars &B = *reinterpret_cast<MuBars *>(stage + MU_STAGE);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    // D's buffers: columns 256 .. 511
    constexpr int dw = REG ? TOK : 256, nd = 256 / dw;

    if (warp == 0) {
        if (lane < MU_MAX_RING) {
            mbar_init(B.wfull + lane, 1);
            mbar_init(B.wempty + lane, 4 * MU_SU);  // four warps a unit
        }
        if (lane < MU_NA) {
            mbar_init(B.full + lane, 5 + (blockIdx.x == 0 ? a.shortfall : 0));  // four warps, x's copy
            mbar_init(B.empty + lane, 1);                                      // a commit
        }
        if (lane < 4) {
            mbar_init(B.dfull + lane, 1);
            mbar_init(B.dempty + lane, 4);
        }
        if (lane == 0) {
            mbar_init(&B.end, 1);
            mbar_init(&B.meet, 4);
            B.stop = 0;
        }
        fence_mbar_init();
    }
    __syncthreads();
    // the warps that use TMEM wait for it by themselves: copies start before
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&B.tmem)), "r"(512)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_fence_before();
    }
    if (warp == 2 || warp >= 4) {
        asm volatile("bar.sync 1, %0;" ::"n"(mu_threads<TOK>() - 96) : "memory");
        tc_fence_after();
    }
    const uint32_t tmem = B.tmem;  // (the copying warps do not use it)
    volatile int *stop = &B.stop;
    // whole warp, which goes on together: false once a wait gave up, this one or another's
    auto wait = [&](uint64_t *bar, uint32_t par) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, par))) return true;
        const uint64_t t0 = globaltimer_ns();
        do {
            if (__any_sync(0xffffffffu, *stop || globaltimer_ns() - t0 > wait_limit_ns())) {
                if (lane == 0) {
                    atomicOr(a.flags, ER_FLAG_WAIT);
                    *stop = 1;
                }
                __syncwarp();
                return false;
            }
        } while (!__all_sync(0xffffffffu, mbar_try_wait(bar, par)));
        return true;
    };

    // registers of the sums' warps: from the others.  The shares of the launch's warps by fours are 56 + 2 * 120 + 216 of 4 * 128,
    // and 40 + 4 * 72 + 152 of 6 * 80.
#define MU_REGISTERS(how, n2, n4)                                                                          \
    if constexpr (REG) {                                                                                   \
        if constexpr (GROUPS == 2) asm volatile("setmaxnreg." how ".sync.aligned.u32 " #n2 ";");           \
        else asm volatile("setmaxnreg." how ".sync.aligned.u32 " #n4 ";");                                 \
    }
    // adapters' steps behind a tile's last one
    auto extra = [&](const MuWalk &w) { return a.nksteps && w.u1 == a.UPR ? max(0, __ldcg(a.nksteps + w.tile / a.MT) + 3) / 4 : 0; };

    MuWalk it(a);
    if (warp < 4) {
        MU_REGISTERS("dec", 56, 40)
        if (warp == 0 || warp == 3) {
            // ---- W's units (constant: no wait for the kernels before this one), the two warps by turns
            const unsigned me = warp == 3;
            MuRing w(a.rs);
            bool ok = true;
            while (ok && it.next(a)) {
                const int rg = (it.tile % a.MT) * 8, nv = min(8, a.R - rg);
                const uint8_t *src = a.W + ((size_t)(rg + lane) * a.UPR + it.u0) * UB;
                for (int u = it.u0; u < it.u1; u += MU_SU, w.step(), src += MU_SU * UB) {
                    if (w.n % MU_PRODUCERS != me) continue;
                    const uint32_t bytes = (uint32_t)(min(MU_SU, it.u1 - u) * UB);
                    if (w.again && !(ok = wait(B.wempty + w.slot, w.par ^ 1))) break;
                    if (lane == 0) mbar_arrive_expect_tx(B.wfull + w.slot, nv * bytes);
                    __syncwarp();
                    if (lane < nv) bulk_g2s(ring_w + w.slot * SLOT + lane * RGS, src, bytes, B.wfull + w.slot);
                }
            }
            // no copy may still be landing when the CTA ends
            for (int i = 0; i < a.rs; ++i, w.step())
                if (w.n >= (unsigned)a.rs && (w.n - a.rs) % MU_PRODUCERS == me) pg_drain(B.wfull + w.slot, w.par ^ 1);
        } else if (warp == 1) {
            // ---- x's tiles
            pdl_wait();
            asm volatile("fence.proxy.async.global;" ::: "memory");
            MuRing x(MU_NA);
            bool ok = true;
            while (ok && it.next(a)) {
                const size_t step = (size_t)a.natoms * 1024;
                const uint8_t *src = a.x + (size_t)(it.tile / a.MT) * a.NT * 128 + it.u0 * step;
                const int end = it.u1 + extra(it);
                for (int u = it.u0; u < end; ++u, x.step(), src += step) {
                    if (x.again && !(ok = wait(B.empty + x.slot, x.par ^ 1))) break;
                    if (lane == 0) {
                        const bool two = F32 && u < it.u1;  // (an adapters' step has one plane)
                        mbar_arrive_expect_tx(B.full + x.slot, (uint32_t)(two ? bsz : a.NT * 128));
                        bulk_g2s(ring_b + x.slot * bsz, src, a.NT * 128, B.full + x.slot);
                        if (two) bulk_g2s(ring_b + x.slot * bsz + a.NT * 128, src + a.plane, a.NT * 128, B.full + x.slot);
                    }
                    __syncwarp();
                }
            }
            // no copy may still be landing when the CTA ends.  (After a wait that gave up a step's other arrivals may never come:
            // then 50 ms pass, far more than a copy takes.)
            const uint64_t t0 = globaltimer_ns();
            for (int i = 0; i < MU_NA; ++i, x.step())
                while (x.n >= (unsigned)MU_NA && !mbar_try_wait(B.full + x.slot, x.par ^ 1) && globaltimer_ns() - t0 < ER_WAIT_NS / 20) {
                }
        } else {
            // ---- products
            // the warp walks together, one thread issues (its operands uniform: two predicates an instruction less)
            const uint32_t mine = pp_elect(), one = 1, idesc = pp_idesc(a.NT);
            const uint64_t d0 = tc_desc_sw128(smem_u32(ring_b));
            MuRing w(MU_NA), sums(nd);
            bool ok = true;
            if (a.nksteps) pdl_wait();
            while (ok && it.next(a)) {
                const int end = it.u1 + extra(it);
                for (int u = it.u0; ok && u < end; sums.step()) {
                    if (sums.again && !(ok = wait(B.dempty + sums.slot, sums.par ^ 1))) break;
                    tc_fence_after();
                    const uint32_t D = tmem + 256 + sums.slot * dw;
                    const int ue = REG ? min(end, u + CHUNK) : end;
                    uint32_t acc = 0;
                    for (; u < ue; ++u, w.step()) {
                        if (!(ok = wait(B.full + w.slot, w.par))) break;
                        tc_fence_after();
                        const uint32_t A = tmem + w.slot * 64;
                        const uint64_t b = d0 + (uint64_t)((w.slot * bsz) >> 4), bl = b + (uint64_t)((a.NT * 128) >> 4);
                        if (mine) {
                            if (u >= it.u1) {  // adapters: bf16 operands
#pragma unroll
                                for (int k = 0; k < 4; ++k) pp_mma_ts(D, A + 8 * k, b + 2 * k, idesc | (1u << 7) | (1u << 10), k ? 1 : acc, one);
                            } else {
                                // the small products first: the sum that they are cut off against is then small too
#pragma unroll
                                for (int k = 0; k < 4; ++k) pp_mma_ts(D, A + 32 + 8 * k, b + 2 * k, idesc, k ? 1 : acc, one);
                                if (F32) {
#pragma unroll
                                    for (int k = 0; k < 4; ++k) pp_mma_ts(D, A + 8 * k, bl + 2 * k, idesc, 1, one);
                                }
#pragma unroll
                                for (int k = 0; k < 4; ++k) pp_mma_ts(D, A + 8 * k, b + 2 * k, idesc, 1, one);
                            }
                            pp_commit(B.empty + w.slot, one);
                        }
                        __syncwarp();
                        acc = 1;
                    }
                    if (ok && mine) pp_commit(B.dfull + sums.slot, one);
                    __syncwarp();
                }
            }
            if (mine) pp_commit(&B.end, one);
            __syncwarp();
            pg_drain(&B.end, 0);  // no product may still be reading when the CTA ends
        }
    } else if (warp < OUT) {
        MU_REGISTERS("dec", 120, 72)
        // ---- weights: lane l of warp q takes row q + 4 (l / 8) of row group l % 8: its 16-byte reads then hit 8 bank groups
        const int q = warp & 3, grp = (warp - 4) >> 2;
        const int rgi = lane & 7, r = q + 4 * (lane >> 3), g = r & 7, upper = r >> 3;
        const uint32_t tA = tmem + ((uint32_t)(32 * q) << 16);
        const uint32_t qoff = (uint32_t)(rgi * RGS + 64 * g), soff = (uint32_t)(rgi * RGS + QB + 8 * g + 2 * upper);
        const uint32_t sel = upper ? 0x4342u : 0x4140u, sh = upper ? 4u : 0u;
        const uint32_t rbase = smem_u32(ring_w);
        MuRing w(a.rs), A(MU_NA);
        bool ok = true;
        while (ok && it.next(a)) {
            const int row = 16 * ((it.tile % a.MT) * 8 + rgi) + r;
            const float up = a.row_up[min(row, 16 * a.R - 1)];
            for (int u = it.u0; ok && u < it.u1; u += MU_SU, w.step()) {
                const int cnt = min(MU_SU, it.u1 - u);
                for (int j = 0; j < cnt; ++j, A.step()) {
                    if ((int)(A.n % GROUPS) != grp) continue;  // a group takes every GROUPS-th step
                    // A's place first: then the products have taken all steps up to four before this one, and the use of W's slot
                    // before this one has long been over (no wait can pass for a phase two before its own)
                    if (A.again && !(ok = wait(B.empty + A.slot, A.par ^ 1))) break;
                    if (!(ok = wait(B.wfull + w.slot, w.par))) break;
                    tc_fence_after();
                    const uint32_t sb = rbase + w.slot * SLOT + j * UB;
#pragma unroll
                    for (int b = 0; b < 2; ++b) {  // a block at a time: fewer registers
                        uint32_t hi[16], lo[16];
                        mu_block_cols<QT>(sb + qoff, b, sel, sh, hi);
                        const float f = __half2float(__ushort_as_half((unsigned short)lds16(sb + soff + 4 * b))) * up;
                        const uint32_t d = pg_pack(f, f);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const uint32_t c = hi[i];
                            hi[i] = h2_fma(c, d, 0x80008000u);
                            lo[i] = h2_fma(c, d, hi[i] ^ 0x80008000u);
                        }
                        pp_st16(tA + A.slot * 64 + 16 * b, hi);
                        pp_st16(tA + A.slot * 64 + 32 + 16 * b, lo);
                    }
                    // the slot is read (a slot with one unit: its second four arrivals too)
                    __syncwarp();
                    if (lane == 0)
                        for (int i = cnt; i <= MU_SU; ++i) mbar_arrive(B.wempty + w.slot);
                    pp_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(B.full + A.slot);
                }
            }
            if (ok && a.nksteps) {  // adapters: rows of B, 16 columns an entry
                pdl_wait();
                const int tn = it.tile / a.MT, end = extra(it);
                const int2 *ks = a.ksteps + (size_t)tn * MU_EXTRA * 4;
                for (int e = 0; e < end; ++e, A.step()) {
                    if ((int)(A.n % GROUPS) != grp) continue;
                    uint32_t v[32];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int2 en = __ldcg(ks + 4 * e + k);  // slot (-1: none) and half, first column
                        uint4 p = make_uint4(0, 0, 0, 0), q = p;
                        if (en.x >= 0 && row < a.rows) {
                            const uint4 *src = reinterpret_cast<const uint4 *>(
                                a.ad.b + ((((size_t)(en.x >> 1) * a.ad.rows + row) * a.ad.r16) + en.y) * 2);
                            p = __ldg(src);
                            q = __ldg(src + 1);
                        }
                        const uint32_t c[8] = {p.x, p.y, p.z, p.w, q.x, q.y, q.z, q.w};
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[8 * k + i] = mu_b_bf16(c[i], a.ad.bf16, en.x & 1, up);
                    }
                    if (A.again && !(ok = wait(B.empty + A.slot, A.par ^ 1))) break;
                    tc_fence_after();
                    pp_st32(tA + A.slot * 64, v);
                    pp_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(B.full + A.slot);
                }
            }
        }
    } else {
        MU_REGISTERS("inc", 216, 152)
        // ---- sums to y
        const int q = warp & 3, thr = tid - 32 * OUT;
        const int rgi = lane & 7, r = q + 4 * (lane >> 3);
        const uint32_t tD = tmem + 256 + ((uint32_t)(32 * q) << 16);
        const int pos = mu_pos(16 * rgi + r);
        pdl_wait();
        MuRing sums(nd);
        bool ok = true;
        // The four warps meet; a limit on this wait too: when one of them gave up, the others must not wait for it for ever.
        uint32_t met = 0;
        auto meet = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.meet);
            const bool all = wait(&B.meet, met);
            met ^= 1;
            return all;
        };
        // one group's 32 tokens out: v in this thread's row, td the factor of token `lane`
        auto out = [&](int tok, int ntok, int row0, float up, float td, const float *v) {
            const float down = 1.f / up;
#pragma unroll
            for (int c = 0; c < 32; ++c) stage[c * 132 + pos] = v[c] * down;
            if (!meet()) return false;
            if (a.type == ER_F32) mu_rows_out(a, reinterpret_cast<float *>(a.y), stage, tok, ntok, row0, td, q, lane);
            else if (a.type == ER_BF16) mu_rows_out(a, reinterpret_cast<__nv_bfloat16 *>(a.y), stage, tok, ntok, row0, td, q, lane);
            else mu_rows_out(a, reinterpret_cast<__half *>(a.y), stage, tok, ntok, row0, td, q, lane);
            return meet();
        };
        auto factor = [&](int tok, int ntok) { return lane < ntok ? a.tok_down[tok + lane] : 0.f; };
        auto adapters = [&](int tok, int ntok, int row, float up, int lo, int hi) {
            return a.ad.bf16 ? mu_adapters<true>(a, stage, tok, ntok, row, pos, up, lo, hi, lane)
                             : mu_adapters<false>(a, stage, tok, ntok, row, pos, up, lo, hi, lane);
        };
        // the last of a shared tile's CTAs (sums of the others visible to all 128 threads); ok: the warps met
        auto last = [&](const MuShare &sh) {
            if (!(ok = meet())) return false;
            if (thr == 0) B.last = atom_add_acq_rel_gpu(a.cnt + sh.t, 1) == sh.n - 1;
            if (!(ok = meet())) return false;
            return B.last != 0;
        };
        while (ok && it.next(a)) {
            const int row0 = (it.tile % a.MT) * 128, tok0 = (it.tile / a.MT) * a.NT, ntok = min(a.NT, a.n - tok0);
            const int row = row0 + 16 * rgi + r;
            const float up = a.row_up[min(row, 16 * a.R - 1)];
            const MuShare sh(a, it.tile);
            // the tokens whose adapters this CTA adds
            const int ci = sh.n > 1 ? (int)blockIdx.x - sh.first : 0, lo = tok0 + ci * ntok / sh.n, hi = tok0 + (ci + 1) * ntok / sh.n;
            float4 *mine = reinterpret_cast<float4 *>(a.part) + (sh.n > 1 ? sh.slot(a, blockIdx.x) * a.NT * 32 : 0) + thr;
            if constexpr (REG) {
                const bool many = a.nksteps && __ldcg(a.nksteps + it.tile / a.MT) < 0;  // (no steps of their own)
                float acc[TOK], td[TOK / 32];
#pragma unroll
                for (int h = 0; h < TOK / 32; ++h) td[h] = factor(tok0 + 32 * h, ntok - 32 * h);
#pragma unroll
                for (int c = 0; c < TOK; ++c) acc[c] = 0.f;
#pragma unroll
                for (int h = 0; h < TOK / 32; ++h)
                    if (32 * h < ntok && many && adapters(tok0 + 32 * h, ntok - 32 * h, row, up, lo, hi)) {
#pragma unroll
                        for (int c = 0; c < 32; ++c) acc[32 * h + c] = stage[c * 132 + pos];
                    }
                const int end = it.u1 + extra(it);
                for (int u = it.u0; u < end; u += CHUNK, sums.step()) {
                    if (!(ok = wait(B.dfull + sums.slot, sums.par))) break;
                    tc_fence_after();
#pragma unroll
                    for (int h = 0; h < TOK / 32; ++h)
                        if (32 * h < a.NT) {
                            float d[32];
                            pp_ld32(tD + sums.slot * dw + 32 * h, d);
                            pp_wait_ld(d);
#pragma unroll
                            for (int c = 0; c < 32; ++c) acc[32 * h + c] += d[c];
                        }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(B.dempty + sums.slot);
                }
                if (!ok) break;
                if (sh.n > 1) {
#pragma unroll
                    for (int h = 0; h < TOK / 16; ++h)
                        if (16 * h < a.NT) {
#pragma unroll
                            for (int c = 16 * h; c < 16 * h + 16; c += 4)
                                __stcg(mine + c * 32, make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]));
                        }
                    if (!last(sh)) continue;
#pragma unroll
                    for (int c = 0; c < TOK; ++c) acc[c] = 0.f;
                    for (int j = 0; j < sh.n; j += 2) {  // two CTAs' on their way together
                        const float4 *p = reinterpret_cast<const float4 *>(a.part) + sh.slot(a, sh.first + j) * a.NT * 32 + thr;
                        const bool two = j + 1 < sh.n;
                        const float4 *p2 = two ? reinterpret_cast<const float4 *>(a.part) + sh.slot(a, sh.first + j + 1) * a.NT * 32 + thr : p;
#pragma unroll
                        for (int h = 0; h < TOK / 32; ++h)
                            if (32 * h < a.NT) {  // (a last half group that the tile does not have is read from the next slot)
                                float4 d[8], e[8];
#pragma unroll
                                for (int c = 0; c < 8; ++c) d[c] = __ldcg(p + (8 * h + c) * 128), e[c] = __ldcg(p2 + (8 * h + c) * 128);
#pragma unroll
                                for (int c = 0; c < 8; ++c) {
                                    float *t = acc + 32 * h + 4 * c;
                                    t[0] += d[c].x, t[1] += d[c].y, t[2] += d[c].z, t[3] += d[c].w;
                                    if (two) t[0] += e[c].x, t[1] += e[c].y, t[2] += e[c].z, t[3] += e[c].w;
                                }
                            }
                    }
                }
#pragma unroll
                for (int h = 0; h < TOK / 32; ++h)
                    if (ok && 32 * h < ntok) ok = out(tok0 + 32 * h, min(32, ntok - 32 * h), row0, up, td[h], acc + 32 * h);
            } else {
                if (!(ok = wait(B.dfull + sums.slot, sums.par))) break;
                tc_fence_after();
                const bool many = a.nksteps && __ldcg(a.nksteps + it.tile / a.MT) < 0;  // (no steps of their own)
                for (int h = 0; ok && 32 * h < a.NT; ++h) {
                    const int left = ntok - 32 * h;
                    const bool with = left > 0 && many && adapters(tok0 + 32 * h, left, row, up, lo, hi);
                    float d[32];
                    pp_ld32(tD + sums.slot * dw + 32 * h, d);
                    pp_wait_ld(d);
                    if (with) {
#pragma unroll
                        for (int c = 0; c < 32; ++c) d[c] += stage[c * 132 + pos];
                    }
                    if (sh.n > 1) {
#pragma unroll
                        for (int g = 0; g < 32; g += 16)
                            if (32 * h + g < a.NT) {
#pragma unroll
                                for (int c = g; c < g + 16; c += 4)
                                    __stcg(mine + (32 * h + c) * 32, make_float4(d[c], d[c + 1], d[c + 2], d[c + 3]));
                            }
                    } else if (left > 0) {
                        ok = out(tok0 + 32 * h, min(32, left), row0, up, factor(tok0 + 32 * h, left), d);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(B.dempty + sums.slot);
                sums.step();
                if (ok && sh.n > 1 && last(sh))
                    for (int h = 0; ok && 32 * h < ntok; ++h) {
                        float d[32];
#pragma unroll
                        for (int c = 0; c < 32; ++c) d[c] = 0.f;
                        for (int j = 0; j < sh.n; ++j) {
                            const float4 *p = reinterpret_cast<const float4 *>(a.part) + (sh.slot(a, sh.first + j) * a.NT + 32 * h) * 32 + thr;
                            float4 e[8];
#pragma unroll
                            for (int c = 0; c < 8; ++c) e[c] = __ldcg(p + c * 128);
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                d[4 * c] += e[c].x;
                                d[4 * c + 1] += e[c].y;
                                d[4 * c + 2] += e[c].z;
                                d[4 * c + 3] += e[c].w;
                            }
                        }
                        ok = out(tok0 + 32 * h, min(32, ntok - 32 * h), row0, up, factor(tok0 + 32 * h, ntok - 32 * h), d);
                    }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

// ---------------------------------------------------------------------------------------------------
// CTAs that share `rem` tiles of UPR steps each (fewer tiles than SMs), by what the last of them needs, in steps: a whole tile; a
// share and the joining of S; an even share, where CTAs have pieces of two tiles.  The costs of joining were fitted to calls timed
// each of the three ways (17 to 500 tokens x 576 to 49152 rows): 500 fp32 tokens x 4096 x 4096 80 us spread, 76 us so.
static int mu_share(int rem, int UPR, int num_sms) {
    if (!rem) return 0;
    int best = rem;
    double cost = UPR;
    for (int s = 2; s * rem <= num_sms && s <= UPR; ++s) {
        const double c = (double)((UPR + s - 1) / s) + MU_JOIN + MU_JOIN_EACH * s;
        if (c < cost) cost = c, best = s * rem;
    }
    if ((long long)rem * UPR >= num_sms) {
        const double c = (double)rem * UPR / num_sms + MU_SPREAD + MU_JOIN_EACH * ((double)num_sms / rem + 1);
        if (c < cost) best = num_sms;
    }
    return best;
}

// n >= 1, 16 R n <= 2^40 + 2^28: fewer than 2^28 tiles, as NT is 64 at least where there are two tiles of tokens
void mul_plan(int R, int UPR, int n, int type, int r16, int num_sms, MulPlan *p) {
    const int most = type == ER_F32 ? MU_REG_TOKENS : MU_MAX_TOKENS;
    p->ntl = (n + most - 1) / most;
    p->NT = ((n + p->ntl - 1) / p->ntl + 15) / 16 * 16;
    p->ntl = (n + p->NT - 1) / p->NT;
    p->MT = (R + 7) / 8;
    const long long tiles = (long long)p->MT * p->ntl;
    // whole tiles for every CTA first; of what is left each tile for a CTA, or for S of them, or all of it spread evenly
    p->waves = (int)(tiles / num_sms);
    p->rem = (int)(tiles % num_sms);
    p->share = mu_share(p->rem, UPR, num_sms);
    p->grid = p->waves ? num_sms : p->share;
    p->planes = type == ER_F32 ? 2 : 1;
    p->natoms = p->ntl * p->NT / 8;
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    p->extra = r16 && n > MU_FEW_TOKENS ? MU_EXTRA : 0;  // (mul_few adds adapters at its end)
    p->off_x = 0;
    p->off_up = up((size_t)(UPR + p->extra) * p->natoms * 1024 * p->planes);
    p->off_v = p->off_up + up((size_t)p->natoms * 8 * 2 * sizeof(float));
    p->off_part = p->off_v + up((size_t)n * r16 * sizeof(float));
    p->slices = n <= MU_FEW_TOKENS ? mul_few_slices(UPR, n, p->planes) : 0;
    if (p->slices) {
        p->waves = p->rem = p->share = 0;
        p->grid = p->slices * max(1, min((R + 1) / 2, num_sms / p->slices));
        p->off_cnt = p->off_k = p->bytes = p->off_part + (p->slices > 1 ? up((size_t)p->slices * n * 16 * R * sizeof(float)) : 0);
        return;
    }
    p->off_cnt = p->off_part + (p->rem ? up(((size_t)p->grid * 2 * p->NT + 16) * 128 * sizeof(float)) : 0);
    p->off_k = p->off_cnt + up((size_t)p->rem * sizeof(int));
    p->bytes = p->off_k + (p->extra ? up((size_t)p->ntl * (1 + 8 * p->extra) * sizeof(int)) : 0);
}

template <int QT, bool F32, int TOK>
static cudaError_t mu_attr() {
    return cudaFuncSetAttribute(mul_main_kernel<QT, F32, TOK>, cudaFuncAttributeMaxDynamicSharedMemorySize, MU_SMEM);
}
template <int QT>
static cudaError_t mu_attrs() {
    cudaError_t r[] = {mu_attr<QT, true, MU_SMALL_TOKENS>(), mu_attr<QT, true, MU_REG_TOKENS>(), mu_attr<QT, false, MU_SMALL_TOKENS>(),
                       mu_attr<QT, false, MU_REG_TOKENS>(), mu_attr<QT, false, 0>()};
    for (cudaError_t x : r)
        if (x != cudaSuccess) return x;
    return cudaSuccess;
}
cudaError_t mul_prepare() {
    const cudaError_t e = mu_attrs<Q8_0>();
    if (e != cudaSuccess) return e;
    const cudaError_t f = mu_attrs<Q4_0>();
    return f == cudaSuccess ? mul_few_prepare() : f;
}

template <class K, class... P>
static cudaError_t mu_launch(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t st, bool pdl, P... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int QT>
static cudaError_t mu_main(MulArgs &k, const MulPlan &p, cudaStream_t st) {
    const bool f32 = k.type == ER_F32;
    constexpr int SLOT = 8 * mu_rgs<QT>();
    const int bsz = k.NT * 128 * p.planes, room = MU_SMEM - 1024 - MU_STAGE * 4 - (int)sizeof(MuBars);
    // rs is even: a slot then always belongs to the same copying warp, which waits for its uses in order.  (With an odd number
    // it could wait for a use while the one before, the other's, is still on its way: a barrier's parity does not tell a phase
    // from the one two before it.)
    k.rs = min(MU_MAX_RING, (room - MU_NA * bsz) / SLOT) & ~1;
    static_assert(MU_PRODUCERS == 2, "even");
    auto go = [&](auto kernel, int threads) { return mu_launch(kernel, dim3(p.grid), threads, MU_SMEM, st, true, k); };
    constexpr int S = MU_SMALL_TOKENS, L = MU_REG_TOKENS;
    if (f32) return p.NT <= S ? go(mul_main_kernel<QT, true, S>, mu_threads<S>()) : go(mul_main_kernel<QT, true, L>, mu_threads<L>());
    if (p.NT <= S) return go(mul_main_kernel<QT, false, S>, mu_threads<S>());
    return p.NT <= L ? go(mul_main_kernel<QT, false, L>, mu_threads<L>()) : go(mul_main_kernel<QT, false, 0>, mu_threads<0>());
}

template <class T>
static cudaError_t mu_prep(const er_matrix_mul_args &a, const Mat &m, const MulArgs &k, float *up, int ncnt, cudaStream_t st) {
    if (k.ids && k.n <= MU_FRONT_TOKENS)
        return mu_launch(mul_front_kernel<T>, dim3(a.n_tokens, k.ad.r16 / 8), 256, 0, st, true, reinterpret_cast<const T *>(a.x_dev),
                         (long long)a.x_stride, m.K, m.UPR, const_cast<uint8_t *>(k.x), k.plane, k.natoms, up,
                         up + (size_t)k.natoms * 8, k.cnt, ncnt, k.ids, k.ad, const_cast<float *>(k.v), const_cast<int2 *>(k.ksteps), const_cast<int *>(k.nksteps),
                         k.flags);
    return mu_launch(mul_prep_kernel<T>, dim3(a.n_tokens), 256, 0, st, true, reinterpret_cast<const T *>(a.x_dev),
                     (long long)a.x_stride, m.K, m.UPR, const_cast<uint8_t *>(k.x), k.plane, k.natoms, up,
                     up + (size_t)k.natoms * 8, k.cnt, ncnt);
}

cudaError_t launch_matrix_mul(const Mat &m, const float *row_up, int *flags, const er_matrix_mul_args &a, const AdaptersView *ad,
                              const MulPlan &p, int shortfall, cudaStream_t st) {
    uint8_t *w = (uint8_t *)a.work_dev;
    float *up = (float *)(w + p.off_up);
    MulArgs k = {};
    k.W = m.d;
    k.row_up = row_up;
    k.R = m.R;
    k.UPR = m.UPR;
    k.rows = m.N;
    k.n = a.n_tokens;
    k.NT = p.NT;
    k.ntl = p.ntl;
    k.MT = p.MT;
    k.waves = p.waves;
    k.rem = p.rem;
    k.grid = p.grid;
    k.grem = p.share;
    k.x = w + p.off_x;
    k.natoms = p.natoms;
    k.plane = (size_t)(m.UPR + p.extra) * p.natoms * 1024;
    k.tok_up = up;
    k.tok_down = up + (size_t)p.natoms * 8;
    if (ad) {
        k.ad = *ad;
        k.ids = a.ids_dev;
    }
    k.v = (const float *)(w + p.off_v);
    k.y = a.y_dev;
    k.y_stride = a.y_stride;
    k.type = a.type;
    k.part = (float *)(w + p.off_part);
    k.cnt = (int *)(w + p.off_cnt);
    k.flags = flags;
    k.shortfall = shortfall;
    int *ks = (int *)(w + p.off_k);
    k.ksteps = (const int2 *)ks;
    k.nksteps = p.extra ? ks + (size_t)p.ntl * 8 * p.extra : nullptr;
    cudaError_t e = a.type == ER_F32   ? mu_prep<float>(a, m, k, up, p.rem, st)
                    : a.type == ER_F16 ? mu_prep<__half>(a, m, k, up, p.rem, st)
                                       : mu_prep<__nv_bfloat16>(a, m, k, up, p.rem, st);
    if (e == cudaSuccess && ad && k.n > MU_FRONT_TOKENS) {
        const dim3 grid((a.n_tokens + 7) / 8, ad->r16 / 16, min(8, a.n_tokens));
        float *v = const_cast<float *>(k.v);
        e = p.planes == 2 ? mu_launch(mul_shrink_kernel<true>, grid, 256, 0, st, true, k.x, k.plane, k.natoms, m.UPR, k.n,
                                      k.tok_down, k.ids, *ad, v)
                          : mu_launch(mul_shrink_kernel<false>, grid, 256, 0, st, true, k.x, k.plane, k.natoms, m.UPR, k.n,
                                      k.tok_down, k.ids, *ad, v);
    }
    if (e == cudaSuccess && ad && k.n > MU_FRONT_TOKENS)
        e = mu_launch(mul_expand_kernel, dim3(p.ntl, p.extra), 256, 0, st, true, const_cast<uint8_t *>(k.x), k.natoms, m.UPR, k.n,
                      k.NT, p.planes, k.tok_up, k.ids, *ad, k.v, (int2 *)ks, const_cast<int *>(k.nksteps), k.flags);
    if (p.slices) return e == cudaSuccess ? launch_mul_few(m, a, ad, p, flags, st) : e;
    if (e == cudaSuccess) e = m.qt == Q8_0 ? mu_main<Q8_0>(k, p, st) : mu_main<Q4_0>(k, p, st);
    return e;
}

cudaError_t set_wait_limit_mul(unsigned long long ns) { return set_wait_limit_here(ns); }

}  // namespace er
