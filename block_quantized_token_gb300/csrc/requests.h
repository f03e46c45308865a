// Host-side declarations of what requests bring to a step (include/er_requests.h).
#pragma once

#include "../../include/er_requests.h"
#include "internal.h"

namespace er {

#define ER_MUL_FLAG_RANGE 2  // an adapter number past the slots
#define ER_MUL_FLAG_WAIT 4   // (ER_FLAG_WAIT)

cudaError_t launch_matrix_row_up(const Mat &m, float *up, cudaStream_t st);

// adapters in the layout that the products read
struct AdaptersView {
    const uint8_t *a;   // fp16 [slots][r16][Kp], rows times powers of two
    const float *down;  // [slots][r16]: what takes a row's product back, the adapter's scale in it
    const uint8_t *b;   // 16 bits [slots][rows][r16]
    const int *rank;    // [slots], multiples of 16, 0: empty
    const int *wild;    // [slots], 1: B holds what is no number, or none once a row of W brings it up (MU_WILD)
    int slots, r16, Kp, rows, bf16;
};
cudaError_t launch_adapters_set(const AdaptersView &v, int slot, int rank, int cols, float scale, const void *a, const void *b,
                                cudaStream_t st);
cudaError_t launch_adapters_clear(const AdaptersView &v, int slot, cudaStream_t st);

// scratch of a product: where its parts lie, in bytes
struct MulPlan {
    int NT, ntl, MT;           // tokens of a tile, tiles of tokens, tiles of rows
    int grid, waves, rem, share;  // CTAs; whole tiles of each; tiles left over, and the CTAs that share these
    int natoms;                // groups of 8 tokens in the operand
    int planes;                // 2: hi and lo halves of fp32 rows
    int extra;                 // steps that adapters may add to a tile
    int slices;                // few tokens (kernels_mul_few.cu): slices of the columns; else 0
    size_t off_x, off_up, off_v, off_part, off_cnt, off_k, bytes;
};
void mul_plan(int R, int UPR, int n, int type, int r16, int num_sms, MulPlan *p);
cudaError_t mul_prepare();  // kernel attributes
int mul_few_slices(int UPR, int n, int planes);
cudaError_t mul_few_prepare();
cudaError_t launch_mul_few(const Mat &m, const er_matrix_mul_args &a, const AdaptersView *ad, const MulPlan &p, int *flags,
                           cudaStream_t st);
cudaError_t launch_matrix_mul(const Mat &m, const float *row_up, int *flags, const er_matrix_mul_args &a, const AdaptersView *ad,
                              const MulPlan &p, int shortfall, cudaStream_t st);
cudaError_t launch_sample(const er_sample_args &a, cudaStream_t st);
cudaError_t set_wait_limit_mul(unsigned long long ns);

}  // namespace er

// What every er_matrix is: with the factors [16 R] that er_matrix_mul brings its rows' scales up by (behind the counters), that
// call's flags (behind the flags word) and its injected shortfall.
struct er_matrix_rows : er_matrix {
    float *row_up;
    int *mul_flags;
    int shortfall;
};

struct er_adapters {
    er_adapters_config cfg;
    int device;
    size_t bytes;
    void *mem;  // one allocation: ranks, factors, A, B
    er::AdaptersView v;
};
