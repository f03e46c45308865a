// er_matrix_mul for few tokens: y[t] = W x[t] (+ scale_a B_a v[t]) for up to 16 of them.
//
// Mathematics.  The rows' operand is that of kernels_mul.cu: fp16 times a power of two of the row, fp32 rows as hi and lo halves.
// W's codes enter the products (mma.sync, exact in fp16) without their scale: per block of 32 columns a sum in the tensor cores,
// which the block's fp16 scale then takes into a sum in fp32.
//
// Work.  W is read once, straight from global memory into registers: a unit's bytes lie in the order of the fragments of
// m16n8k16.  A CTA of 16 warps keeps the rows of a slice of the columns in shared memory; its items are pairs of row groups
// (32 rows), which share the fragments of x.  A warp works a share of the slice's units, the same for every item, with the loads
// of the next units, across items, on their way; the warps' sums of an item meet in shared memory (two buffers, a barrier an
// item), where warp t sums up token t's 32 rows, adds its adapter's share and writes them.  Columns that do not fit are cut into
// slices, each with CTAs of its own; sums of slices go to scratch, and a kernel behind this one adds them in their order.
//
// What bounds it.  Up to 8 bf16 tokens HBM: 128256 x 4096 Q8_0 90 us, 6.2 TB/s, 0.92 of a copy's rate.  16 tokens (108 us) and
// fp32 rows (173 us) the warps' own chains: four warps a scheduler, as many as 128 registers allow, issue 36 % of the time, tensor
// pipe 20 and 31 %; waiting for loads, for fragments and for products follow one another.  Loads of two steps are on their way; the
// third costs registers that the products miss (128256 x 4096 with 8 tokens 108 us).  What is further ahead is fetched into L2
// (32000 x 4096 with 16 bf16 tokens 39 to 32 us).  Two or four pairs of row groups at a time, with half or a quarter of the
// warps on each, gain nothing (fp32 176 to 183 us), nor do products of both groups of tokens in turn (+ 0 to 3 %).
// Small matrices: the two kernels' way to each other, 3.1 us for one token x 576 x 576 and 6.4 us for 16 x 4096 x 4096 (2.8 TB/s).
#include <cuda_bf16.h>

#include "gemv_core.cuh"
#include "pages.cuh"
#include "requests.h"

namespace er {

constexpr int MF_WARPS = 16, MF_THREADS = 32 * MF_WARPS;
constexpr int MF_AHEAD = 2;   // steps (a unit of two row groups) whose loads are on their way
constexpr int MF_FETCH = 8;   // steps that are fetched into L2 before their loads, about
constexpr int MF_ROW = 36;    // floats of a token's 32 rows in a warp's sums: lanes' places lie in 32 banks
constexpr int MF_SMEM = 231424;

__host__ __device__ constexpr int mf_sums(int tiles) { return 2 * MF_WARPS * 8 * tiles * MF_ROW * 4; }

struct FewArgs {
    const uint8_t *W;
    int R, UPR, rows, n;
    int pairs, slices, per;  // per: CTAs of a slice
    const uint8_t *x;
    size_t plane;
    int natoms;
    const float *tok_down;
    AdaptersView ad;
    const int32_t *ids;  // NULL: no adapters
    const float *v;
    void *y;
    long long y_stride;
    int type;
    float *part;  // slices > 1: [slice][token][16 R]
    int *flags;
};

template <int QT>
struct MfUnit {
    uint4 q[QT == Q8_0 ? 2 : 1];
    uint2 d;
};
ER_DEV uint4 mf_ld16(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
ER_DEV uint2 mf_ld8(const void *p) {
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
template <int QT>
ER_DEV void mf_load(MfUnit<QT> &w, const uint8_t *unit, int lane) {
    w.q[0] = mf_ld16(unit + 16 * lane);
    if (QT == Q8_0) w.q[QT == Q8_0 ? 1 : 0] = mf_ld16(unit + 512 + 16 * lane);
    w.d = mf_ld8(unit + QTraits<QT>::quant_bytes + 8 * (lane >> 2));
}
// fragments of 16 columns (half h of block b)
template <int QT>
ER_DEV void mf_fragment(const MfUnit<QT> &w, int b, int h, uint32_t (&A)[4]) {
    if (QT == Q8_0) {
        const uint4 c = w.q[QT == Q8_0 ? b : 0];
        q8_word_to_h2(h ? c.z : c.x, A[0], A[1]);
        q8_word_to_h2(h ? c.w : c.y, A[2], A[3]);
    } else {
        const uint4 c = w.q[0];
        q4_word_to_h2(b ? (h ? c.w : c.z) : (h ? c.y : c.x), A);
    }
}
ER_DEV void mf_ldmatrix(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
ER_DEV void mf_copy16(uint32_t to, const void *from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// the adapter's share of this lane's row: B's row times the token's v
template <bool BF16>
ER_DEV float mf_share(const uint4 *b, const float4 *v, int rank) {
    float s = 0.f, t = 0.f;
    for (int j = 0; j < rank / 8; j += 2) {
        const uint4 p = __ldg(b + j), q = __ldg(b + j + 1);
        const float4 v0 = __ldcg(v + 2 * j), v1 = __ldcg(v + 2 * j + 1), v2 = __ldcg(v + 2 * j + 2), v3 = __ldcg(v + 2 * j + 3);
        auto dot = [](uint32_t w0, uint32_t w1, const float4 &f, float a) {
            float2 x, y;
            if (BF16) {
                x = make_float2(__uint_as_float(w0 << 16), __uint_as_float(w0 & 0xFFFF0000u));
                y = make_float2(__uint_as_float(w1 << 16), __uint_as_float(w1 & 0xFFFF0000u));
            } else {
                x = __half22float2(*reinterpret_cast<const __half2 *>(&w0));
                y = __half22float2(*reinterpret_cast<const __half2 *>(&w1));
            }
            return fmaf(y.y, f.w, fmaf(y.x, f.z, fmaf(x.y, f.y, fmaf(x.x, f.x, a))));
        };
        s = dot(p.x, p.y, v0, s);
        t = dot(p.z, p.w, v1, t);
        s = dot(q.x, q.y, v2, s);
        t = dot(q.z, q.w, v3, t);
    }
    return s + t;
}

ER_DEV void mf_out(void *y, size_t at, int type, float f) {
    if (type == ER_F32) reinterpret_cast<float *>(y)[at] = f;
    else if (type == ER_BF16) reinterpret_cast<__nv_bfloat16 *>(y)[at] = __float2bfloat16(f);
    else reinterpret_cast<__half *>(y)[at] = __float2half_rn(f);
}

// PL: planes of the operand; TILES: groups of 8 tokens
template <int QT, int PL, int TILES>
__global__ void __launch_bounds__(MF_THREADS, 1) mul_few_kernel(const __grid_constant__ FewArgs a) {
    constexpr int UB = QTraits<QT>::unit_bytes, XU = PL * TILES * 1024;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int slice = blockIdx.x / a.per, first = blockIdx.x % a.per;
    // this warp's units of the slice's
    const int s0 = (int)((long long)slice * a.UPR / a.slices), ns = (int)((long long)(slice + 1) * a.UPR / a.slices) - s0;
    const int most = ns / MF_WARPS, more = ns % MF_WARPS, nu = most + (warp < more), l0 = warp * most + min(warp, more), u0 = s0 + l0;
    const int busy = min(ns, MF_WARPS);  // warps with units
    const int items = first < a.pairs ? (a.pairs - first + a.per - 1) / a.per : 0;
    float *const sums = reinterpret_cast<float *>(smem_raw);
    uint8_t *const xs = smem_raw + mf_sums(TILES) + (size_t)l0 * XU;
    const uint32_t xa = smem_u32(xs);

    // ---- W's units in the order of their use
    const int steps = items * nu;
    int lp = first, lu = 0;
    const uint8_t *src = a.W + ((size_t)2 * lp * a.UPR + u0) * UB;
    size_t second = 2 * lp + 1 < a.R ? (size_t)a.UPR * UB : 0;  // (a last pair may have one row group: its rows twice)
    // into L2 before: a pair's units of this warp
    const int ahead = nu ? (MF_FETCH + nu - 1) / nu : 0;
    auto fetch = [&](int p) {
        if (lane < 2 && p < a.pairs && 2 * p + lane < a.R)
            prefetch_l2_bulk(a.W + ((size_t)(2 * p + lane) * a.UPR + u0) * UB, (uint32_t)(nu * UB));
    };
    auto load = [&](MfUnit<QT> (&w)[2]) {
        mf_load<QT>(w[0], src, lane);
        mf_load<QT>(w[1], src + second, lane);
        src += UB;
        if (++lu == nu) {
            lu = 0;
            lp += a.per;
            src = a.W + ((size_t)2 * lp * a.UPR + u0) * UB;
            second = 2 * lp + 1 < a.R ? (size_t)a.UPR * UB : 0;
            fetch(lp + ahead * a.per);
        }
    };
    MfUnit<QT> w[MF_AHEAD][2];
#pragma unroll
    for (int i = 0; i < MF_AHEAD; ++i)
        if (i < steps) load(w[i]);
    for (int i = 1; i <= ahead; ++i) fetch(first + i * a.per);

    // ---- x: every warp its own units
    pdl_wait();
    pdl_launch_dependents();  // (after the wait: what starts now finds all before this kernel done)
    for (int i = 0; i < nu; ++i)
#pragma unroll
        for (int p = 0; p < PL; ++p)
#pragma unroll
            for (int q = 0; q < TILES; ++q) {
                const uint8_t *from = a.x + p * a.plane + ((size_t)(u0 + i) * a.natoms + q) * 1024 + lane * 16;
                const uint32_t to = xa + (uint32_t)(i * XU + (p * TILES + q) * 1024 + lane * 16);
                mf_copy16(to, from);
                mf_copy16(to + 512, from + 512);
            }
    asm volatile("cp.async.commit_group;" ::: "memory");
    // the token that this warp sums up
    const bool sums_up = warp < a.n;
    float down = 0.f;
    int id = -1, rank = 0;
    if (sums_up) {
        down = a.tok_down[warp];
        if (a.ids && slice == 0) {
            id = a.ids[warp];
            if (id >= a.ad.slots) {
                if (first == 0 && lane == 0) atomicOr(a.flags, ER_MUL_FLAG_RANGE);
                id = -1;
            }
            if (id >= 0) rank = a.ad.rank[id];
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();

    float acc[2][TILES][4];
    auto clear = [&]() {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int q = 0; q < TILES; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[r][q][i] = 0.f;
    };
    clear();
    int pair = first, cu = 0, buffer = 0;
    // an item's end
    auto finish = [&]() {
        float *const at = sums + buffer * MF_WARPS * 8 * TILES * MF_ROW;
        if (nu) {
            float *const to = at + warp * 8 * TILES * MF_ROW + 2 * t * MF_ROW + g;
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int q = 0; q < TILES; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i) to[(8 * q + (i & 1)) * MF_ROW + 16 * r + 8 * (i >> 1)] = acc[r][q][i];
            clear();
        }
        asm volatile("bar.sync 1, %0;" ::"n"(MF_THREADS) : "memory");
        if (sums_up) {
            float s = 0.f;
            const float *from = at + warp * MF_ROW + lane;
#pragma unroll
            for (int i = 0; i < MF_WARPS; ++i)
                if (i < busy) s += from[i * 8 * TILES * MF_ROW];
            s *= down;
            const int row = 32 * pair + lane;
            if (row < a.rows) {
                if (rank) {
                    const uint4 *b = reinterpret_cast<const uint4 *>(a.ad.b + ((size_t)id * a.ad.rows + row) * a.ad.r16 * 2);
                    const float4 *v = reinterpret_cast<const float4 *>(a.v + (size_t)warp * a.ad.r16);
                    s += a.ad.bf16 ? mf_share<true>(b, v, rank) : mf_share<false>(b, v, rank);
                }
                if (a.slices > 1) __stcg(a.part + ((size_t)slice * a.n + warp) * 16 * a.R + row, s);
                else mf_out(a.y, (size_t)warp * a.y_stride + row, a.type, s);
            }
        }
        buffer ^= 1;
        pair += a.per;
    };
    const uint32_t xrow = xa + (lane & 7) * 128, chunk = lane >> 3, swz = lane & 7;
    auto consume = [&](const MfUnit<QT> (&w)[2]) {
        const uint32_t xu = xrow + (uint32_t)cu * XU;
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            uint32_t B[PL][TILES][4];
#pragma unroll
            for (int p = 0; p < PL; ++p)
#pragma unroll
                for (int q = 0; q < TILES; ++q) mf_ldmatrix(xu + (p * TILES + q) * 1024 + (((4 * b + chunk) ^ swz) << 4), B[p][q]);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                uint32_t A[2][4];
                mf_fragment<QT>(w[r], b, 0, A[0]);
                mf_fragment<QT>(w[r], b, 1, A[1]);
                // (an infinite scale becomes NaN)
                const uint32_t dd = b ? w[r].d.y : w[r].d.x, d2 = h2_fma(dd, 0u, dd);
                const float d0 = h2f_lo(d2), d1 = h2f_hi(d2);
#pragma unroll
                for (int q = 0; q < TILES; ++q) {
                    float D[4];
                    const float zero[4] = {0.f, 0.f, 0.f, 0.f};
                    // lo halves first
                    mma_16816(D, A[0], B[PL - 1][q][0], B[PL - 1][q][1], zero);
                    mma_16816(D, A[1], B[PL - 1][q][2], B[PL - 1][q][3], D);
                    if (PL == 2) {
                        mma_16816(D, A[0], B[0][q][0], B[0][q][1], D);
                        mma_16816(D, A[1], B[0][q][2], B[0][q][3], D);
                    }
                    acc[r][q][0] = fmaf(d0, D[0], acc[r][q][0]);
                    acc[r][q][1] = fmaf(d0, D[1], acc[r][q][1]);
                    acc[r][q][2] = fmaf(d1, D[2], acc[r][q][2]);
                    acc[r][q][3] = fmaf(d1, D[3], acc[r][q][3]);
                }
            }
        }
        if (++cu == nu) {
            cu = 0;
            finish();
        }
    };
    if (!nu)
        for (int i = 0; i < items; ++i) finish();
    for (int s = 0; s < steps; s += MF_AHEAD) {
#pragma unroll
        for (int i = 0; i < MF_AHEAD; ++i)
            if (s + i < steps) {
                consume(w[i]);
                if (s + i + MF_AHEAD < steps) load(w[i]);
            }
    }
}

// sums of slices, in their order
__global__ void __launch_bounds__(256) mul_few_join_kernel(const float *part, int slices, int n, int R, int rows, void *y,
                                                           long long y_stride, int type) {
    pdl_wait();
    pdl_launch_dependents();
    const int row = blockIdx.x * 256 + threadIdx.x, token = blockIdx.y;
    if (row >= rows) return;
    const size_t step = (size_t)n * 16 * R;
    const float *p = part + (size_t)token * 16 * R + row;
    float s = 0.f;
    for (int i = 0; i < slices; ++i) s += __ldcg(p + i * step);
    mf_out(y, (size_t)token * y_stride + row, type, s);
}

int mul_few_slices(int UPR, int n, int planes) {
    const int tiles = n > 8 ? 2 : 1, units = (MF_SMEM - mf_sums(tiles)) / (planes * tiles * 1024);
    return (UPR + units - 1) / units;
}

template <int QT, int PL, int TILES>
static cudaError_t mf_attr() {
    return cudaFuncSetAttribute(mul_few_kernel<QT, PL, TILES>, cudaFuncAttributeMaxDynamicSharedMemorySize, MF_SMEM);
}
cudaError_t mul_few_prepare() {
    cudaError_t r[] = {mf_attr<Q8_0, 1, 1>(), mf_attr<Q8_0, 1, 2>(), mf_attr<Q8_0, 2, 1>(), mf_attr<Q8_0, 2, 2>(),
                       mf_attr<Q4_0, 1, 1>(), mf_attr<Q4_0, 1, 2>(), mf_attr<Q4_0, 2, 1>(), mf_attr<Q4_0, 2, 2>()};
    for (cudaError_t x : r)
        if (x != cudaSuccess) return x;
    return cudaSuccess;
}

template <class K, class... P>
static cudaError_t mf_launch(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t st, P... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

cudaError_t launch_mul_few(const Mat &m, const er_matrix_mul_args &a, const AdaptersView *ad, const MulPlan &p, int *flags,
                           cudaStream_t st) {
    uint8_t *work = (uint8_t *)a.work_dev;
    FewArgs k = {};
    k.W = m.d;
    k.R = m.R;
    k.UPR = m.UPR;
    k.rows = m.N;
    k.n = a.n_tokens;
    k.pairs = (m.R + 1) / 2;
    k.slices = p.slices;
    k.per = p.grid / p.slices;
    k.x = work + p.off_x;
    k.plane = (size_t)m.UPR * p.natoms * 1024;
    k.natoms = p.natoms;
    k.tok_down = (const float *)(work + p.off_up) + (size_t)p.natoms * 8;
    if (ad) {
        k.ad = *ad;
        k.ids = a.ids_dev;
    }
    k.v = (const float *)(work + p.off_v);
    k.y = a.y_dev;
    k.y_stride = a.y_stride;
    k.type = a.type;
    k.part = (float *)(work + p.off_part);
    k.flags = flags;
    const int tiles = k.n > 8 ? 2 : 1;
    const size_t smem = mf_sums(tiles) + (size_t)((m.UPR + p.slices - 1) / p.slices) * p.planes * tiles * 1024;
    auto go = [&](auto kernel) { return mf_launch(kernel, dim3(p.grid), MF_THREADS, smem, st, k); };
    const bool two = tiles == 2;
    cudaError_t e;
    if (m.qt == Q8_0) {
        if (p.planes == 2) e = two ? go(mul_few_kernel<Q8_0, 2, 2>) : go(mul_few_kernel<Q8_0, 2, 1>);
        else e = two ? go(mul_few_kernel<Q8_0, 1, 2>) : go(mul_few_kernel<Q8_0, 1, 1>);
    } else {
        if (p.planes == 2) e = two ? go(mul_few_kernel<Q4_0, 2, 2>) : go(mul_few_kernel<Q4_0, 2, 1>);
        else e = two ? go(mul_few_kernel<Q4_0, 1, 2>) : go(mul_few_kernel<Q4_0, 1, 1>);
    }
    if (e == cudaSuccess && p.slices > 1)
        e = mf_launch(mul_few_join_kernel, dim3((m.N + 255) / 256, k.n), 256, 0, st, (const float *)k.part, k.slices, k.n, m.R, m.N,
                      k.y, k.y_stride, k.type);
    return e;
}

}  // namespace er
