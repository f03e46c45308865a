// Host-side declarations of the paged 4-bit K/V cache (include/er_pages.h).
#pragma once

#include "../../include/er_pages.h"
#include "internal.h"

namespace er {

// ---------------------------------------------------------------------------
// paged 4-bit K/V cache (pages.cuh: layout and quantiser)
// ---------------------------------------------------------------------------
#define ER_PAGES_FLAG_FULL 1   // a request was not admitted
#define ER_PAGES_FLAG_RANGE 2  // a length, position, slot or table entry out of range
#define ER_PAGES_MAX_SEQS 1024
struct PagesView {
    uint8_t *pool;  // the layer's pages
    int n_pages, page_rows, KV, hd;
    int *flags;
};
cudaError_t launch_pages_plan(const PagesView &p, const er_pages_plan_args &a, int *ticket, int num_sms,
                              cudaStream_t st);
cudaError_t launch_pages_release(const PagesView &p, int n_seqs, const int32_t *done, int32_t *lens, int32_t *tables,
                                 int table_stride, int32_t *free_list, int32_t *free_count, cudaStream_t st);
cudaError_t launch_rope_table(int hd, double base, int n, float *out, cudaStream_t st);
cudaError_t launch_pages_append(const PagesView &p, const er_pages_append_args &a, int num_sms, cudaStream_t st);
cudaError_t launch_pages_read(const PagesView &p, int n, const int32_t *slots, int type, void *k, void *v,
                              cudaStream_t st);
cudaError_t launch_pages_attention(const PagesView &p, const er_pages_attention_args &a, float *part, int *cnt,
                                   int shortfall, int num_sms, cudaStream_t st);
size_t pages_attn_part_floats(int num_sms);  // `part`; cnt: one int per SM, zero
cudaError_t pages_attn_prepare();            // kernel attributes
// sequences with at least min_rows query rows a KV head (kernels_pages_prompt.cu)
cudaError_t launch_pages_prompt(const PagesView &p, const er_pages_attention_args &a, int min_rows, int shortfall,
                                cudaStream_t st);
cudaError_t pages_prompt_prepare();
cudaError_t set_wait_limit_prompt(unsigned long long ns);
cudaError_t set_wait_limit_pages(unsigned long long ns);

}  // namespace er

struct er_pages {
    er_pages_config cfg;
    uint8_t *pool;
    size_t layer_bytes;
    int device, num_sms;
    int *flags;   // er_pages_error
    int *ticket;  // arrival counter of the plan kernel (zero between launches)
    int *cnt;     // arrival counters of the attention kernel [SMs] (zero between launches)
    int shortfall;  // er_pages_inject_wait_shortfall
    float *part;  // states of units shared by several CTAs (pages_attn_part_floats)
};
