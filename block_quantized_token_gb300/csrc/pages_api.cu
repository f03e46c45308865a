// Entry points of the paged 4-bit K/V cache (include/er_pages.h): argument checks and ownership.
#include <math.h>

#include <new>

#include "pages.cuh"
#include "pages.h"

using namespace er;

namespace {

er_status check_config(const er_pages_config *c) {
    if (!c) return er_fail_status(ER_EINVAL, "config is NULL");
    if (c->n_layers < 1 || c->n_pages < 1 || c->n_kv_heads < 1 || c->page_rows < 1 || c->head_dim < 1)
        return er_fail_status(ER_EINVAL, "config sizes must be positive");
    if (c->page_rows % 16 || c->page_rows > 1024)
        return er_fail_status(ER_EINVAL, "page_rows must be a multiple of 16 up to 1024");
    if (c->head_dim != 64 && c->head_dim != 128) return er_fail_status(ER_EUNSUPPORTED, "head_dim must be 64 or 128");
    if (c->kv_type != ER_Q4_0) {
        const bool known = c->kv_type == ER_F32 || c->kv_type == ER_F16 || c->kv_type == ER_Q8_0 || c->kv_type == ER_BF16;
        return er_fail_status(known ? ER_EUNSUPPORTED : ER_EINVAL, "kv_type must be ER_Q4_0");
    }
    if ((long long)c->n_pages * c->page_rows > 2147483647ll)
        return er_fail_status(ER_EINVAL, "n_pages * page_rows must be below 2^31");
    if (c->n_kv_heads > 1024 || c->n_layers > 65536) return er_fail_status(ER_EINVAL, "n_kv_heads or n_layers too large");
    // a layer's tiles have 32-bit numbers in the kernels
    if ((long long)c->n_pages * (c->page_rows / 16) * c->n_kv_heads > 2147483647ll)
        return er_fail_status(ER_EINVAL, "n_pages * page_rows * n_kv_heads must be below 2^35");
    return ER_OK;
}

size_t layer_bytes(const er_pages_config *c) {
    return (size_t)c->n_pages * c->n_kv_heads * (c->page_rows / 16) * pg_tile_bytes(c->head_dim);
}

bool row_type(int t) { return t == ER_F32 || t == ER_F16 || t == ER_BF16; }
int type_bytes(int t) { return t == ER_F32 ? 4 : 2; }
bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

template <class... P>
bool words(const P *...p) {  // int32 and float arrays (NULL is)
    return (((uintptr_t)p | ...) & 3) == 0;
}

// refuses memory of another device than the current one, where a kernel would reach it as a peer's or fault
er_status check_memory(const void *p, const char *what) {
    int dev = -1;
    cudaPointerAttributes a;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaPointerGetAttributes(&a, p);
    if (e != cudaSuccess) return er_fail_cuda(e, what);
    return a.type == cudaMemoryTypeDevice && a.device != dev
               ? er_fail_status(ER_EINVAL, "the memory belongs to another device than the current one")
               : ER_OK;
}
er_status check_handle(const er_pages *p) {
    if (!p) return er_fail_status(ER_EINVAL, "handle is NULL");
    int dev = -1;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return er_fail_cuda(e, "cudaGetDevice");
    if (dev != p->device) return er_fail_status(ER_EINVAL, "the handle belongs to another device than the current one");
    return ER_OK;
}
er_status check_layer(const er_pages *p, int32_t layer) {
    if (er_status s = check_handle(p); s != ER_OK) return s;
    if (layer < 0 || layer >= p->cfg.n_layers) return er_fail_status(ER_EINVAL, "layer out of range");
    return ER_OK;
}

PagesView view_of(const er_pages *p, int layer) {
    return {p->pool + (size_t)layer * p->layer_bytes, p->cfg.n_pages, p->cfg.page_rows, p->cfg.n_kv_heads,
            p->cfg.head_dim, p->flags};
}
er_status done(cudaError_t e, const char *what) { return e == cudaSuccess ? ER_OK : er_fail_cuda(e, what); }

}  // namespace

extern "C" {

size_t er_pages_pool_bytes(const er_pages_config *cfg) {
    return check_config(cfg) == ER_OK ? layer_bytes(cfg) * cfg->n_layers : 0;
}

er_status er_pages_create(const er_pages_config *cfg, void *pool, er_pages **out) {
    if (!out) return er_fail_status(ER_EINVAL, "out is NULL");
    if (er_status s = check_config(cfg); s != ER_OK) return s;
    if (!pool) return er_fail_status(ER_EINVAL, "pool is NULL");
    if (!aligned(pool, 16)) return er_fail_status(ER_EINVAL, "pool must be 16-byte aligned");
    if (er_status s = check_memory(pool, "er_pages_create"); s != ER_OK) return s;
    er_pages *p = new (std::nothrow) er_pages();
    if (!p) return er_fail_status(ER_ENOMEM, "out of host memory");
    p->cfg = *cfg;
    p->pool = (uint8_t *)pool;
    p->layer_bytes = layer_bytes(cfg);
    p->flags = p->ticket = p->cnt = nullptr;
    p->part = nullptr;
    p->shortfall = 0;
    cudaError_t e = cudaGetDevice(&p->device);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&p->num_sms, cudaDevAttrMultiProcessorCount, p->device);
    if (e == cudaSuccess) e = pages_attn_prepare();
    // one block: flags, ticket, counters (zero), then the attention kernel's states
    const size_t ints = (128 + (size_t)(p->num_sms + 63) / 64 * 64) * sizeof(int);
    void *q = nullptr;
    if (e == cudaSuccess) e = device_alloc(&q, ints + pages_attn_part_floats(p->num_sms) * sizeof(float));
    if (e == cudaSuccess) {
        p->flags = (int *)q;
        p->ticket = p->flags + 64;
        p->cnt = p->flags + 128;
        p->part = (float *)((uint8_t *)q + ints);
        e = cudaMemset(q, 0, ints);
    }
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
        er_pages_destroy(p);
        return er_fail_cuda(e, "er_pages_create");
    }
    *out = p;
    return ER_OK;
}

void er_pages_destroy(er_pages *p) {
    if (!p) return;
    device_free(p->flags);
    delete p;
}

er_status er_pages_plan(er_pages *p, const er_pages_plan_args *a, void *stream) {
    if (!p || !a) return er_fail_status(ER_EINVAL, "NULL argument");
    if (a->n_seqs < 1 || a->n_seqs > ER_PAGES_MAX_SEQS) return er_fail_status(ER_EINVAL, "n_seqs must be in 1..1024");
    if (a->max_tokens < 0 || a->table_stride < 1) return er_fail_status(ER_EINVAL, "max_tokens or table_stride out of range");
    if (!a->lens_dev || !a->new_dev || !a->free_dev || !a->free_count_dev || !a->tables_dev || !a->lens_out_dev ||
        !a->free_count_out_dev || !a->q_start_dev ||
        (a->max_tokens && (!a->positions_dev || !a->slots_dev || !a->seqs_dev)))
        return er_fail_status(ER_EINVAL, "NULL argument");
    if (!words(a->lens_dev, a->new_dev, a->free_dev, a->free_count_dev, a->tables_dev, a->lens_out_dev, a->free_count_out_dev,
               a->q_start_dev, a->positions_dev, a->slots_dev, a->seqs_dev))
        return er_fail_status(ER_EINVAL, "int arrays must be 4-byte aligned");
    if (er_status s = check_handle(p); s != ER_OK) return s;
    return done(launch_pages_plan(view_of(p, 0), *a, p->ticket, p->num_sms, (cudaStream_t)stream), "er_pages_plan");
}

er_status er_pages_release(er_pages *p, int32_t n_seqs, const int32_t *done_dev, int32_t *lens, int32_t *tables,
                           int32_t table_stride, int32_t *free_list, int32_t *free_count, void *stream) {
    if (!p || !done_dev || !lens || !tables || !free_list || !free_count) return er_fail_status(ER_EINVAL, "NULL argument");
    if (n_seqs < 1 || n_seqs > ER_PAGES_MAX_SEQS) return er_fail_status(ER_EINVAL, "n_seqs must be in 1..1024");
    if (table_stride < 1) return er_fail_status(ER_EINVAL, "table_stride must be positive");
    // (the kernel numbers the entries given back with an int, a block's width at a time)
    if ((long long)n_seqs * table_stride > 2147483648ll - 1024)
        return er_fail_status(ER_EINVAL, "n_seqs * table_stride must be at most 2^31 - 1024");
    if (!words(done_dev, lens, tables, free_list, free_count)) return er_fail_status(ER_EINVAL, "int arrays must be 4-byte aligned");
    if (er_status s = check_handle(p); s != ER_OK) return s;
    return done(launch_pages_release(view_of(p, 0), n_seqs, done_dev, lens, tables, table_stride, free_list, free_count,
                                     (cudaStream_t)stream),
                "er_pages_release");
}

er_status er_rope_table(int32_t head_dim, double base, int32_t n, float *out, void *stream) {
    if (head_dim < 2 || head_dim % 2 || head_dim > 1024) return er_fail_status(ER_EINVAL, "head_dim must be even, 2..1024");
    if (!(base > 0) || !isfinite(base)) return er_fail_status(ER_EINVAL, "base must be positive and finite");
    if (n < 0 || (n && !out)) return er_fail_status(ER_EINVAL, "n_positions negative or out NULL");
    if (!aligned(out, 4)) return er_fail_status(ER_EINVAL, "out must be 4-byte aligned");
    if (!n) return ER_OK;
    if (er_status s = check_memory(out, "er_rope_table"); s != ER_OK) return s;
    return done(launch_rope_table(head_dim, base, n, out, (cudaStream_t)stream), "er_rope_table");
}

er_status er_pages_append(er_pages *p, int32_t layer, const er_pages_append_args *a, void *stream) {
    if (!p || !a) return er_fail_status(ER_EINVAL, "NULL argument");
    if (er_status s = check_layer(p, layer); s != ER_OK) return s;
    if (!row_type(a->type)) return er_fail_status(ER_EINVAL, "type must be ER_F32, ER_F16 or ER_BF16");
    if (a->n_tokens < 0 || a->n_heads < 0 || a->n_heads > 65536) return er_fail_status(ER_EINVAL, "n_tokens or n_heads out of range");
    if (!a->n_tokens) return ER_OK;
    if (!a->k_dev || !a->v_dev || !a->slots_dev) return er_fail_status(ER_EINVAL, "k, v and slots must be given");
    if ((a->n_heads > 0) != (a->q_dev != nullptr) || (a->n_heads > 0) != (a->q_out_dev != nullptr))
        return er_fail_status(ER_EINVAL, "q and q_out must be given iff n_heads > 0");
    if (a->rope_style != ER_ROPE_PAIRS && a->rope_style != ER_ROPE_HALVES)
        return er_fail_status(ER_EINVAL, "rope_style must be ER_ROPE_PAIRS or ER_ROPE_HALVES");
    if (a->rope_dev && (!a->positions_dev || a->rope_positions < 1))
        return er_fail_status(ER_EINVAL, "a rope table needs positions and rope_positions >= 1");
    if (a->rope_dev && !aligned(a->rope_dev, 8)) return er_fail_status(ER_EINVAL, "the rope table must be 8-byte aligned");
    if (!words(a->q_gain_dev, a->k_gain_dev, a->positions_dev, a->slots_dev))
        return er_fail_status(ER_EINVAL, "gains, positions and slots must be 4-byte aligned");
    if (!(a->eps >= 0.f) || isinf(a->eps)) return er_fail_status(ER_EINVAL, "eps must be finite and >= 0");
    const int64_t row = (int64_t)a->n_heads * p->cfg.head_dim, kvd = (int64_t)p->cfg.n_kv_heads * p->cfg.head_dim;
    if (a->q_stride < row || a->q_out_stride < row || a->k_stride < kvd || a->v_stride < kvd)
        return er_fail_status(ER_EINVAL, "a stride is shorter than its row");
    const size_t n = (size_t)type_bytes(a->type);
    if (!aligned(a->q_dev, n) || !aligned(a->k_dev, n) || !aligned(a->v_dev, n) || !aligned(a->q_out_dev, n))
        return er_fail_status(ER_EINVAL, "rows must be aligned to their type");
    if (a->q_out_dev && a->q_out_dev == a->q_dev && a->q_out_stride != a->q_stride)
        return er_fail_status(ER_EINVAL, "q_out may be q only with the same stride");
    return done(launch_pages_append(view_of(p, layer), *a, p->num_sms, (cudaStream_t)stream), "er_pages_append");
}

er_status er_pages_read(er_pages *p, int32_t layer, int32_t n, const int32_t *slots, int32_t type, void *k, void *v,
                        void *stream) {
    if (er_status s = check_layer(p, layer); s != ER_OK) return s;
    if (!row_type(type)) return er_fail_status(ER_EINVAL, "type must be ER_F32, ER_F16 or ER_BF16");
    if (n < 0 || (n && !slots)) return er_fail_status(ER_EINVAL, "n negative or slots NULL");
    if (!words(slots)) return er_fail_status(ER_EINVAL, "slots must be 4-byte aligned");
    if (!aligned(k, type_bytes(type)) || !aligned(v, type_bytes(type)))
        return er_fail_status(ER_EINVAL, "rows must be aligned to their type");
    if (!n || (!k && !v)) return ER_OK;
    return done(launch_pages_read(view_of(p, layer), n, slots, type, k, v, (cudaStream_t)stream), "er_pages_read");
}

er_status er_pages_attention(er_pages *p, int32_t layer, const er_pages_attention_args *a, void *stream) {
    if (!p || !a) return er_fail_status(ER_EINVAL, "NULL argument");
    if (er_status s = check_layer(p, layer); s != ER_OK) return s;
    if (!row_type(a->type)) return er_fail_status(ER_EINVAL, "type must be ER_F32, ER_F16 or ER_BF16");
    if (a->n_seqs < 1 || a->n_seqs > ER_PAGES_MAX_SEQS) return er_fail_status(ER_EINVAL, "n_seqs must be in 1..1024");
    if (a->n_tokens < 0 || a->table_stride < 1 || a->window < 0)
        return er_fail_status(ER_EINVAL, "n_tokens, table_stride or window out of range");
    if (a->n_heads < 1 || a->n_heads % p->cfg.n_kv_heads || a->n_heads / p->cfg.n_kv_heads > 64)
        return er_fail_status(ER_EINVAL, "n_heads must be a multiple of n_kv_heads, at most 64 times it");
    if ((int64_t)a->n_tokens * (a->n_heads / p->cfg.n_kv_heads) > 2147483647ll - 1024)
        return er_fail_status(ER_EINVAL, "n_tokens * n_heads / n_kv_heads must be below 2^31 - 1024");
    if (!a->n_tokens) return ER_OK;
    if (!words(a->q_start_dev, a->lens_dev, a->tables_dev)) return er_fail_status(ER_EINVAL, "int arrays must be 4-byte aligned");
    if (!a->q_dev || !a->out_dev || !a->q_start_dev || !a->lens_dev || !a->tables_dev)
        return er_fail_status(ER_EINVAL, "NULL argument");
    const int64_t row = (int64_t)a->n_heads * p->cfg.head_dim;
    if (a->q_stride < row || a->out_stride < row) return er_fail_status(ER_EINVAL, "a stride is shorter than its row");
    if (!isfinite(a->scale)) return er_fail_status(ER_EINVAL, "scale must be finite");
    const size_t n = (size_t)type_bytes(a->type);
    if (!aligned(a->q_dev, n) || !aligned(a->out_dev, n) || !aligned(a->lse_dev, 4))
        return er_fail_status(ER_EINVAL, "rows must be aligned to their type");
    if (a->out_dev == a->q_dev && a->out_stride != a->q_stride)
        return er_fail_status(ER_EINVAL, "out may be q only with the same stride");
    return done(launch_pages_attention(view_of(p, layer), *a, p->part, p->cnt, p->shortfall, p->num_sms, (cudaStream_t)stream),
                "er_pages_attention");
}

er_status er_pages_inject_wait_shortfall(er_pages *p, int32_t extra) {
    if (!p) return er_fail_status(ER_EINVAL, "handle is NULL");
    if (extra < 0 || extra > 1024) return er_fail_status(ER_EINVAL, "extra must be in 0..1024");
    p->shortfall = extra;
    return ER_OK;
}

er_status er_pages_error(er_pages *p, int32_t *code) {
    if (!p || !code) return er_fail_status(ER_EINVAL, "NULL argument");
    if (er_status s = check_handle(p); s != ER_OK) return s;
    cudaError_t e = cudaDeviceSynchronize();
    int f = 0;
    if (e == cudaSuccess) e = cudaMemcpy(&f, p->flags, sizeof(int), cudaMemcpyDeviceToHost);
    if (e == cudaSuccess) e = cudaMemset(p->flags, 0, sizeof(int));
    // a kernel that gave up may have left its arrival counters short
    if (e == cudaSuccess && (f & ER_FLAG_WAIT)) e = cudaMemset(p->cnt, 0, (size_t)p->num_sms * sizeof(int));
    // cudaMemset returns before it is done, and a stream that does not wait for the null stream may run a call of this handle next
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return er_fail_cuda(e, "er_pages_error");
    *code = f & (ER_PAGES_FLAG_FULL | ER_PAGES_FLAG_RANGE | ER_FLAG_WAIT);
    return *code ? er_fail_status(ER_EDEVICE, "device flags set") : ER_OK;
}

}  // extern "C"
