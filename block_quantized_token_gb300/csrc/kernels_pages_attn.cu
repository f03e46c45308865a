// Attention over the paged 4-bit K/V cache (pages.cuh): o = softmax(scale q k^T) v for the rows that a
// token attends, one pass over them with the running maximum m and sum l:
//   m' = max(m, s),  l' = l e^(m - m') + e^(s - m'),  o' = o e^(m - m') + e^(s - m') v.
// One warp per (token, query head), lanes over the head's dims.
#include "internal.h"
#include "pages.cuh"

namespace er {

template <class T, int HD>
__global__ void __launch_bounds__(256) pages_attn_kernel(PagesView p, er_pages_attention_args a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.y, G = a.n_heads / p.KV;
    const int q0 = a.q_start_dev[b], q1 = a.q_start_dev[b + 1], len = a.lens_dev[b];
    if (q0 < 0 || q1 < q0 || q1 > a.n_tokens || len < 0 || (long long)len > (long long)a.table_stride * p.page_rows) {
        if (threadIdx.x == 0) atomicOr(p.flags, ER_PAGES_FLAG_RANGE);
        return;
    }
    const float scale = (a.scale != 0.f ? a.scale : 1.f / sqrtf((float)HD)) * 1.4426950408889634f;
    const long long items = (long long)(q1 - q0) * a.n_heads;
    for (long long it = (long long)blockIdx.x * 8 + warp; it < items; it += (long long)gridDim.x * 8) {
        const int i = (int)(it / a.n_heads), h = (int)(it - (long long)i * a.n_heads);
        const int row = q0 + i, pos = len - (q1 - q0) + i, kvh = h / G;
        const int first = a.window ? max(0, pos - a.window + 1) : 0;
        constexpr int NB = HD / 32;
        // lane l holds dim 32 b + l of every block b
        const T *q = (const T *)a.q_dev + row * a.q_stride + (size_t)h * HD;
        float x[NB], o[NB], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int k = 0; k < NB; ++k) {
            x[k] = pg_ld<T>(q + 32 * k + lane) * scale;
            o[k] = 0.f;
        }
        for (int r = first; r <= pos; ++r) {
            const int page = a.tables_dev[(size_t)b * a.table_stride + r / p.page_rows];
            if (page < 0 || page >= p.n_pages) {
                if (lane == 0) atomicOr(p.flags, ER_PAGES_FLAG_RANGE);
                continue;
            }
            const int slot = page * p.page_rows + r % p.page_rows, rr = (r % p.page_rows) & 15;
            const uint8_t *tile = pg_tile(p.pool, p.page_rows, p.KV, HD, slot, kvh);
            const __half *ks = reinterpret_cast<const __half *>(tile + pg_off_ks(HD));
            const __half *vs = reinterpret_cast<const __half *>(tile + pg_off_vs(HD));
            float s = 0.f, v[NB];
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                const uint32_t w = *reinterpret_cast<const uint32_t *>(tile + pg_k_word(rr, (lane >> 3) * NB + k, HD));
                const int j = lane & 7, bit = 4 * (j >> 1) + 16 * (j & 1);
                s = fmaf(x[k], __half2float(ks[rr * NB + k]) * (float)((int)((w >> bit) & 15u) - 8), s);
                const int dim = 32 * k + lane, jj = 8 * (dim >> 4) + (dim & 7);
                const int c = tile[pg_off_v(HD) + pg_v_byte(rr, jj, HD)];
                v[k] = __half2float(vs[pg_vs_half(rr, k, HD)]) * (float)(((dim & 8) ? c >> 4 : c & 15) - 8);
            }
#pragma unroll
            for (int off = 16; off; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
            const float mn = fmaxf(m, s), base = mn == -INFINITY ? 0.f : mn;
            const float corr = exp2f(m - base), e = exp2f(s - base);
            l = l * corr + e;
#pragma unroll
            for (int k = 0; k < NB; ++k) o[k] = o[k] * corr + e * v[k];
            m = mn;
        }
        T *out = (T *)a.out_dev + row * a.out_stride + (size_t)h * HD;
#pragma unroll
        for (int k = 0; k < NB; ++k) out[32 * k + lane] = pg_cvt<T>(l == 0.f ? 0.f : o[k] / l);
        if (a.lse_dev && lane == 0)
            a.lse_dev[(size_t)row * a.n_heads + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
}

template <class T>
static cudaError_t attn_t(const PagesView &p, const er_pages_attention_args &a, cudaStream_t st) {
    const long long items = (long long)a.n_tokens * a.n_heads;
    long long x = (items + 7) / 8;
    if (x > 1024) x = 1024;
    dim3 grid((unsigned)x, (unsigned)a.n_seqs);
    if (p.hd == 128) pages_attn_kernel<T, 128><<<grid, 256, 0, st>>>(p, a);
    else pages_attn_kernel<T, 64><<<grid, 256, 0, st>>>(p, a);
    return cudaGetLastError();
}

cudaError_t launch_pages_attention(const PagesView &p, const er_pages_attention_args &a, int num_sms,
                                   cudaStream_t st) {
    (void)num_sms;
    return a.type == ER_F32   ? attn_t<float>(p, a, st)
           : a.type == ER_F16 ? attn_t<__half>(p, a, st)
                              : attn_t<__nv_bfloat16>(p, a, st);
}

}  // namespace er
