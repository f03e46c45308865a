// Entry points of what requests bring to a step (include/er_requests.h): argument checks and ownership.
#include <math.h>

#include <new>

#include "requests.h"

using namespace er;

namespace {

bool row_type(int t) { return t == ER_F32 || t == ER_F16 || t == ER_BF16; }
bool aligned(const void *p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

er_status check_device(int device) {
    int dev = -1;
    if (cudaError_t e = cudaGetDevice(&dev); e != cudaSuccess) return er_fail_cuda(e, "cudaGetDevice");
    if (dev != device) return er_fail_status(ER_EINVAL, "the handle belongs to another device than the current one");
    return ER_OK;
}
er_status done(cudaError_t e, const char *what) { return e == cudaSuccess ? ER_OK : er_fail_cuda(e, what); }

er_status check_adapters(const er_adapters *ad, int slot) {
    if (!ad) return er_fail_status(ER_EINVAL, "adapters are NULL");
    if (slot < 0 || slot >= ad->cfg.slots) return er_fail_status(ER_EINVAL, "slot out of range");
    return check_device(ad->device);
}

// what a product's sizes must keep to, with its plan
er_status check_mul(const er_matrix *x, const er_adapters *ad, int64_t n, int type, MulPlan *p) {
    if (!x) return er_fail_status(ER_EINVAL, "matrix is NULL");
    if (!row_type(type)) return er_fail_status(ER_EINVAL, "type must be ER_F32, ER_F16 or ER_BF16");
    if (n < 0 || n >= (1 << 24)) return er_fail_status(ER_EINVAL, "n_tokens must be in 0..2^24 - 1");
    if (n * x->m.N >= 1ll << 40 || n * x->m.K >= 1ll << 40)
        return er_fail_status(ER_EINVAL, "n_tokens times rows or cols must be below 2^40");
    if (ad && (ad->cfg.rows != x->m.N || ad->cfg.cols != x->m.K))
        return er_fail_status(ER_EINVAL, "the adapters are of another shape than the matrix");
    if (ad && ad->device != x->device) return er_fail_status(ER_EINVAL, "the adapters belong to another device than the matrix");
    if (n) mul_plan(x->m.R, x->m.UPR, (int)n, type, ad ? ad->v.r16 : 0, x->num_sms, p);
    return ER_OK;
}

}  // namespace

extern "C" {

er_status er_adapters_create(const er_adapters_config *c, er_adapters **out) {
    if (!c || !out) return er_fail_status(ER_EINVAL, "NULL argument");
    if (c->rows < 1 || c->cols < 32 || c->cols % 32)
        return er_fail_status(ER_EINVAL, "rows >= 1, cols a positive multiple of 32");
    if (c->slots < 1 || c->slots > 4096) return er_fail_status(ER_EINVAL, "slots must be in 1..4096");
    if (c->max_rank < 1 || c->max_rank > 256) return er_fail_status(ER_EINVAL, "max_rank must be in 1..256");
    if (c->type != ER_F16 && c->type != ER_BF16) return er_fail_status(ER_EINVAL, "type must be ER_F16 or ER_BF16");
    er_adapters *ad = new (std::nothrow) er_adapters();
    if (!ad) return er_fail_status(ER_ENOMEM, "out of host memory");
    ad->cfg = *c;
    AdaptersView &v = ad->v;
    v.slots = c->slots;
    v.r16 = (c->max_rank + 15) / 16 * 16;
    v.Kp = (c->cols + 63) / 64 * 64;
    v.rows = c->rows;
    v.bf16 = c->type == ER_BF16;
    auto up = [](size_t b) { return (b + 255) / 256 * 256; };
    const size_t nr = up((size_t)v.slots * 2 * sizeof(int)), nd = up((size_t)v.slots * v.r16 * sizeof(float));
    const size_t na = (size_t)v.slots * v.r16 * v.Kp * 2, nb = (size_t)v.slots * v.rows * v.r16 * 2;
    ad->bytes = nr + nd + up(na) + up(nb);
    ad->mem = nullptr;
    cudaError_t e = cudaGetDevice(&ad->device);
    if (e == cudaSuccess) e = device_alloc(&ad->mem, ad->bytes);
    if (e == cudaSuccess) e = cudaMemset(ad->mem, 0, nr);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) {
        er_adapters_destroy(ad);
        return er_fail_cuda(e, "er_adapters_create");
    }
    uint8_t *m = (uint8_t *)ad->mem;
    v.rank = (const int *)m;
    v.wild = v.rank + v.slots;
    v.down = (const float *)(m + nr);
    v.a = m + nr + nd;
    v.b = m + nr + nd + up(na);
    *out = ad;
    return ER_OK;
}

void er_adapters_destroy(er_adapters *ad) {
    if (!ad) return;
    device_free(ad->mem);
    delete ad;
}

size_t er_adapters_device_bytes(const er_adapters *ad) { return ad ? ad->bytes : 0; }

er_status er_adapters_set(er_adapters *ad, int32_t slot, int32_t rank, float scale, const void *a, const void *b, void *stream) {
    if (er_status s = check_adapters(ad, slot); s != ER_OK) return s;
    if (rank < 1 || rank > ad->cfg.max_rank) return er_fail_status(ER_EINVAL, "rank must be in 1..max_rank");
    if (!isfinite(scale)) return er_fail_status(ER_EINVAL, "scale must be finite");
    if (!a || !b) return er_fail_status(ER_EINVAL, "NULL argument");
    if (!aligned(a, 2) || !aligned(b, 2)) return er_fail_status(ER_EINVAL, "a and b must be 2-byte aligned");
    return done(launch_adapters_set(ad->v, slot, rank, ad->cfg.cols, scale, a, b, (cudaStream_t)stream), "er_adapters_set");
}

er_status er_adapters_clear(er_adapters *ad, int32_t slot, void *stream) {
    if (er_status s = check_adapters(ad, slot); s != ER_OK) return s;
    return done(launch_adapters_clear(ad->v, slot, (cudaStream_t)stream), "er_adapters_clear");
}

size_t er_matrix_mul_work_bytes(const er_matrix *x, const er_adapters *ad, int32_t n, int32_t type) {
    MulPlan p;
    return check_mul(x, ad, n, type, &p) == ER_OK ? (n ? p.bytes : 256) : 0;
}

er_status er_matrix_mul(const er_matrix *x, const er_matrix_mul_args *a, void *stream) {
    if (!x || !a) return er_fail_status(ER_EINVAL, "NULL argument");
    MulPlan p;
    if (er_status s = check_mul(x, a->adapters, a->n_tokens, a->type, &p); s != ER_OK) return s;
    if (er_status s = check_device(x->device); s != ER_OK) return s;
    if ((a->adapters != nullptr) != (a->ids_dev != nullptr))
        return er_fail_status(ER_EINVAL, "adapters and ids must be given together");
    if (!a->n_tokens) return ER_OK;
    if (!a->x_dev || !a->y_dev || !a->work_dev) return er_fail_status(ER_EINVAL, "x, y and work must be given");
    if (a->x_stride < x->m.K || a->y_stride < x->m.N) return er_fail_status(ER_EINVAL, "a stride is shorter than its row");
    const size_t n = a->type == ER_F32 ? 4 : 2;
    if (!aligned(a->x_dev, n) || !aligned(a->y_dev, n)) return er_fail_status(ER_EINVAL, "rows must be aligned to their type");
    if (!aligned(a->ids_dev, 4)) return er_fail_status(ER_EINVAL, "ids must be 4-byte aligned");
    if (!aligned(a->work_dev, 256)) return er_fail_status(ER_EINVAL, "work must be 256-byte aligned");
    if (a->work_bytes < p.bytes) return er_fail_status(ER_EINVAL, "work is smaller than er_matrix_mul_work_bytes");
    const er_matrix_rows *y = static_cast<const er_matrix_rows *>(x);
    return done(launch_matrix_mul(x->m, y->row_up, y->mul_flags, *a, a->adapters ? &a->adapters->v : nullptr, p, y->shortfall,
                                  (cudaStream_t)stream),
                "er_matrix_mul");
}

er_status er_matrix_mul_error(er_matrix *x, int32_t *code) {
    if (!x || !code) return er_fail_status(ER_EINVAL, "NULL argument");
    if (er_status s = check_device(x->device); s != ER_OK) return s;
    int f = 0, *w = static_cast<er_matrix_rows *>(x)->mul_flags;
    cudaError_t e = cudaDeviceSynchronize();
    if (e == cudaSuccess) e = cudaMemcpy(&f, w, sizeof(int), cudaMemcpyDeviceToHost);
    if (e == cudaSuccess) e = cudaMemset(w, 0, sizeof(int));
    // the memset returns before it is done; a call on another stream may set a flag next
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) return er_fail_cuda(e, "er_matrix_mul_error");
    *code = f & (ER_MUL_FLAG_RANGE | ER_MUL_FLAG_WAIT);
    return *code ? er_fail_status(ER_EDEVICE, "device flags set") : ER_OK;
}

er_status er_matrix_mul_inject_wait_shortfall(er_matrix *x, int32_t extra) {
    if (!x) return er_fail_status(ER_EINVAL, "matrix is NULL");
    if (extra < 0 || extra > 1024) return er_fail_status(ER_EINVAL, "extra must be in 0..1024");
    static_cast<er_matrix_rows *>(x)->shortfall = extra;
    return ER_OK;
}

er_status er_sample(const er_sample_args *a, void *stream) {
    if (!a) return er_fail_status(ER_EINVAL, "NULL argument");
    if (!row_type(a->type)) return er_fail_status(ER_EINVAL, "type must be ER_F32, ER_F16 or ER_BF16");
    if (a->n_rows < 0 || a->n_rows > 1 << 20) return er_fail_status(ER_EINVAL, "n_rows must be in 0..2^20");
    if (a->vocab < 1) return er_fail_status(ER_EINVAL, "vocab must be positive");
    if (a->vocab > ER_SAMPLE_MAX_VOCAB) return er_fail_status(ER_EUNSUPPORTED, "vocab above ER_SAMPLE_MAX_VOCAB");
    if (!a->n_rows) return ER_OK;
    if (!a->logits_dev || !a->uniform_dev || !a->tokens_dev)
        return er_fail_status(ER_EINVAL, "logits, uniform and tokens must be given");
    if (a->stride < a->vocab) return er_fail_status(ER_EINVAL, "the stride is shorter than a row");
    if (!aligned(a->logits_dev, a->type == ER_F32 ? 4 : 2)) return er_fail_status(ER_EINVAL, "rows must be aligned to their type");
    const uintptr_t words = (uintptr_t)a->temperature_dev | (uintptr_t)a->top_k_dev | (uintptr_t)a->top_p_dev |
                            (uintptr_t)a->min_p_dev | (uintptr_t)a->uniform_dev | (uintptr_t)a->tokens_dev |
                            (uintptr_t)a->logprobs_dev;
    if (words & 3) return er_fail_status(ER_EINVAL, "int and float arrays must be 4-byte aligned");
    if (!aligned(a->top_k64_dev, 8)) return er_fail_status(ER_EINVAL, "top_k64 must be 8-byte aligned");
    if (a->top_k_dev && a->top_k64_dev) return er_fail_status(ER_EINVAL, "top_k and top_k64 must not be given together");
    return done(launch_sample(*a, (cudaStream_t)stream), "er_sample");
}

}  // extern "C"
