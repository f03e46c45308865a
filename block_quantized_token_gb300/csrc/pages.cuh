// The paged 4-bit K/V cache: where a row's codes and scales lie in the pool, and
// the quantiser's steps.  A page of one KV head is page_rows / 16 tiles of 16
// rows, one tile 18 * HD contiguous bytes (a multiple of 128: 2304 or 1152), so
// that one bulk copy brings all that 16 rows need.
//   K codes [16 rows][HD / 2 bytes]: word t * (HD / 32) + b of a row holds dims
//     32 b + 8 t .. + 7, dim 2 i + e of those at bits 4 i + 16 e: a mask yields the
//     fp16 pair (2 i, 2 i + 1), and lane t of a tensor-core quad finds its 8 dims of
//     every block in HD / 32 consecutive words.
//   V codes [HD / 64 q][8 g][4 t][4 u] words: dims 64 q + 16 u + g (low nibbles) and
//     that + 8 (high nibbles) of rows 2 t + e + 8 i in byte i + 2 e: a mask yields the
//     pair of rows (2 t, 2 t + 1) of one dim.  A byte belongs to one row, so rows
//     written at the same time by different threads share none.
//   K scales [16][HD / 32]; V scales [4 t][HD / 32][2 i][2 e].
// Scales have 8 significant bits (rounded to bf16 first): d (c - 8) then has at
// most 8 + 3 = 11, so every value is an fp16 number and enters the tensor cores
// unrounded; (16 + c) d - 24 d is exact in one fp16 FMA because 24 d has at most
// 8 + 2 bits and |d| <= 2720 keeps it finite.
#pragma once
#include <cuda_bf16.h>

#include "common.cuh"
#include "tcgen05.cuh"

namespace er {

constexpr float PG_DMAX = 2720.f;

__host__ __device__ constexpr int pg_tile_bytes(int hd) { return 18 * hd; }
__host__ __device__ constexpr int pg_off_ks(int hd) { return 8 * hd; }
__host__ __device__ constexpr int pg_off_v(int hd) { return 9 * hd; }
__host__ __device__ constexpr int pg_off_vs(int hd) { return 17 * hd; }

// byte of a tile that holds dims d and (V) d + 8 / (K) the code of dim d of row r; nibble: its bits
__host__ __device__ inline int pg_k_word(int r, int w, int hd) { return r * (hd / 2) + 4 * w; }  // word w of row r
__host__ __device__ inline int pg_v_byte(int r, int j) {  // byte of dims 16 (j / 8) + j % 8 and + 8, j < hd / 2
    const int q = j >> 5, u = (j >> 3) & 3, g = j & 7, t = (r & 7) >> 1, e = r & 1, i = r >> 3;
    return ((((q * 8 + g) * 4 + t) * 4) + u) * 4 + i + 2 * e;
}
__host__ __device__ inline int pg_vs_half(int r, int b, int hd) {  // index of the V scale of (row r, block b)
    return ((((r & 7) >> 1) * (hd / 32) + b) * 2 + (r >> 3)) * 2 + (r & 1);
}

// a slot's tile of KV head h
ER_DEV uint8_t *pg_tile(uint8_t *pool, int page_rows, int KV, int hd, int slot, int h) {
    const int page = slot / page_rows, in = slot - page * page_rows;
    return pool + (((size_t)page * KV + h) * (page_rows >> 4) + (in >> 4)) * pg_tile_bytes(hd);
}

// fp16(bf16(-m / 8)) within +-PG_DMAX; NaN stays
ER_DEV float pg_scale(float m) {
    const float d = __bfloat162float(__float2bfloat16_rn(m * -0.125f));
    if (isnan(d)) return d;
    return __half2float(__float2half_rn(fminf(fmaxf(d, -PG_DMAX), PG_DMAX)));
}

// one value of a row of `type` (ER_F32, ER_F16, ER_BF16) by its index
template <class T>
ER_DEV float pg_ld(const T *p);
template <>
ER_DEV float pg_ld<float>(const float *p) { return *p; }
template <>
ER_DEV float pg_ld<__half>(const __half *p) { return __half2float(*p); }
template <>
ER_DEV float pg_ld<__nv_bfloat16>(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
template <class T>
ER_DEV T pg_cvt(float v);
template <>
ER_DEV float pg_cvt<float>(float v) { return v; }
template <>
ER_DEV __half pg_cvt<__half>(float v) { return __float2half_rn(v); }
template <>
ER_DEV __nv_bfloat16 pg_cvt<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Waits for what a CTA has in flight before it ends.  With a limit of its own: under the one that er_set_wait_limit_ns sets
// the CTA could end while copies still write its shared memory, by then another's.
ER_DEV void pg_drain(uint64_t *bar, uint32_t parity) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < ER_WAIT_NS) {
    }
}

ER_DEV float pg_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
ER_DEV uint32_t pg_pack(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// nibble N of each half of w (bits 4 N ..) as the fp16 pair 16 + c; fma(that, d, pg_m24(d)) are the values of scale pair d
template <int N>
ER_DEV uint32_t pg_code(uint32_t w) {
    return lop3_and_or(N == 0 ? w << 6 : N == 1 ? w << 2 : N == 2 ? w >> 2 : w >> 6, 0x03C003C0u, 0x4C004C00u);
}
ER_DEV uint32_t pg_m24(uint32_t d) {
    // (the factor written as the word 0xCE00CE00 costs the prompt kernel 16 of 572 us: another order of its code)
    const __half2 r = __hmul2(*reinterpret_cast<const __half2 *>(&d), __halves2half2(__ushort_as_half(0xCE00), __ushort_as_half(0xCE00)));
    return *reinterpret_cast<const uint32_t *>(&r);
}

constexpr int PG_MAX_LEN = 2147483647 - 1024;
// a sequence's rows at most: what its table holds, and fewer than 2^31 by so much that sums with a block or a page stay ints
ER_DEV int pg_max_len(int table_stride, int page_rows) {
    return (int)min((long long)table_stride * page_rows, (long long)PG_MAX_LEN);
}
// the first row that the token at position p attends (p < 0: none, whatever this says)
ER_DEV int pg_first(int p, int window) { return window ? max(0, max(p, 0) - (window - 1)) : 0; }

}  // namespace er
