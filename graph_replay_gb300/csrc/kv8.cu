// kv8.cu -- the C ABI of the 8-bit K/V cache: argument checks and launches on
// the caller's stream.  No handle, no allocation, no wait: each call only
// launches kernels, so it can be recorded into a graph, and calls from several
// threads do not meet.
#include <limits.h>
#include <stdarg.h>
#include <stdio.h>

#include <cmath>

#include "graphdec.h"
#include "internal.h"

using namespace gd;

namespace {

constexpr int64_t KV8_MAX_CAP = 1 << 30;

int refuse(int code, const char* fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_call_message(buf);
    return code;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// the caller's current device is put back when the call ends
struct OnDevice {
    int prev = -1, dev;
    cudaError_t e;
    explicit OnDevice(int device) : dev(device) {
        e = cudaGetDevice(&prev);
        if (e == cudaSuccess && prev != dev) e = cudaSetDevice(dev);
    }
    ~OnDevice() {
        if (prev >= 0 && prev != dev) cudaSetDevice(prev);
    }
};

int check_cache(const dec_kv8_cache* c, Kv8Cache* out) {
    if (!c) return refuse(DEC_E_INVALID, "cache is NULL");
    if (!c->k || !c->v || !c->k_scale || !c->v_scale) return refuse(DEC_E_INVALID, "k, v, k_scale and v_scale are required");
    if (!aligned16(c->k) || !aligned16(c->v)) return refuse(DEC_E_INVALID, "k and v must be 16-byte aligned");
    if (c->rows < 1 || c->pages_per_row < 1 || c->page_size < 1 || c->num_pages < 1 || c->n_kv_heads < 1)
        return refuse(DEC_E_INVALID, "rows, pages_per_row, page_size, num_pages and n_kv_heads must be >= 1");
    if (c->rows > KV8_MAX_ROWS) return refuse(DEC_E_UNSUPPORTED, "rows = %d: at most %d", c->rows, KV8_MAX_ROWS);
    if (c->n_kv_heads > 1024) return refuse(DEC_E_UNSUPPORTED, "n_kv_heads = %d: at most 1024", c->n_kv_heads);
    if (c->head_dim != 64 && c->head_dim != 128)
        return refuse(DEC_E_UNSUPPORTED, "head_dim %d unsupported (64 or 128)", c->head_dim);
    if (c->scale_block != 16 && c->scale_block != 32 && c->scale_block != 64 && c->scale_block != 128)
        return refuse(DEC_E_UNSUPPORTED, "scale_block %d unsupported (16, 32, 64 or 128)", c->scale_block);
    if (c->page_size % c->scale_block) return refuse(DEC_E_INVALID, "page_size must be a multiple of scale_block");
    if ((int64_t)c->pages_per_row * c->page_size > KV8_MAX_CAP)
        return refuse(DEC_E_UNSUPPORTED, "pages_per_row * page_size: at most 2^30 positions");
    if (!c->pages && (int64_t)c->rows * c->pages_per_row > c->num_pages)
        return refuse(DEC_E_INVALID, "without a page table num_pages must be at least rows * pages_per_row");
    if (c->device < 0) return refuse(DEC_E_INVALID, "device must be >= 0");
    *out = Kv8Cache{(uint8_t*)c->k, (uint8_t*)c->v, c->k_scale, c->v_scale, c->pages, c->rows, c->pages_per_row,
                    c->page_size, c->num_pages, c->n_kv_heads, c->head_dim, c->scale_block,
                    kv8_log2(c->scale_block), FastDiv((unsigned)c->page_size)};
    return DEC_OK;
}

int check_batch(const dec_kv8_batch* b, const Kv8Cache& c, Kv8Batch* out) {
    if (!b) return refuse(DEC_E_INVALID, "batch is NULL");
    if (!b->kv_len || !b->err) return refuse(DEC_E_INVALID, "kv_len and err are required");
    if (b->total < 0 || b->max_new < 1) return refuse(DEC_E_INVALID, "total must be >= 0 and max_new >= 1");
    if (!b->q_start && (b->total != c.rows || b->max_new != 1))
        return refuse(DEC_E_INVALID, "without q_start each row has one token: total = rows, max_new = 1");
    if (b->max_new > (1 << 24)) return refuse(DEC_E_UNSUPPORTED, "max_new = %d: at most 2^24", b->max_new);
    *out = Kv8Batch{b->q_start, b->kv_len, b->total, b->max_new, b->err, 0};
    return DEC_OK;
}

int check_dtype(int dtype, int* out) {
    if (dtype != DEC_DTYPE_F32 && dtype != DEC_DTYPE_BF16)
        return refuse(DEC_E_INVALID, "dtype must be DEC_DTYPE_F32 or DEC_DTYPE_BF16");
    *out = dtype == DEC_DTYPE_BF16 ? W_BF16 : W_F32;
    return DEC_OK;
}

// a [total, heads, head_dim] operand: heads side by side, any 16-byte aligned token stride
int check_tokens(const char* what, const void* p, int64_t stride, int heads, int hd, int wt, int total) {
    const int es = wt == W_BF16 ? 2 : 4;
    if (!p && total > 0) return refuse(DEC_E_INVALID, "%s is NULL", what);
    if (!aligned16(p)) return refuse(DEC_E_INVALID, "%s must be 16-byte aligned", what);
    if (stride < (int64_t)heads * hd || (stride * es) % 16)
        return refuse(DEC_E_INVALID, "%s: the token stride must hold all heads and be a multiple of 16 bytes", what);
    return DEC_OK;
}

int check_attend(const dec_kv8_cache* cache, const dec_kv8_batch* batch, const dec_kv8_attn* a, Kv8Attend* p) {
    int rc;
    if ((rc = check_cache(cache, &p->c)) != DEC_OK) return rc;
    if ((rc = check_batch(batch, p->c, &p->b)) != DEC_OK) return rc;
    if (!a) return refuse(DEC_E_INVALID, "attn is NULL");
    if ((rc = check_dtype(a->dtype, &p->dtype)) != DEC_OK) return rc;
    if (a->n_heads < 1 || a->n_heads % p->c.Hkv) return refuse(DEC_E_INVALID, "n_kv_heads must divide n_heads");
    if (a->n_heads / p->c.Hkv > 128) return refuse(DEC_E_UNSUPPORTED, "n_heads / n_kv_heads: at most 128");
    if ((int64_t)p->b.max_new * a->n_heads > (1 << 30)) return refuse(DEC_E_UNSUPPORTED, "max_new * n_heads: at most 2^30");
    if (a->window < 0 || a->sinks < 0) return refuse(DEC_E_INVALID, "window and sinks must be >= 0");
    if (!(a->scale >= 0.0) || !std::isfinite((float)a->scale))
        return refuse(DEC_E_INVALID, "scale must be finite and >= 0");
    if ((rc = check_tokens("q", a->q, a->q_stride, a->n_heads, p->c.hd, p->dtype, p->b.total)) != DEC_OK) return rc;
    if ((rc = check_tokens("out", a->out, a->out_stride, a->n_heads, p->c.hd, p->dtype, p->b.total)) != DEC_OK) return rc;
    p->q = a->q;
    p->out = a->out;
    p->q_stride = a->q_stride;
    p->out_stride = a->out_stride;
    p->heads(a->n_heads);
    p->window = a->window ? a->window : INT_MAX;
    p->sinks = a->window ? a->sinks : 0;
    p->scale = a->scale > 0.0 ? (float)a->scale : (float)(1.0 / std::sqrt((double)p->c.hd));
    return DEC_OK;
}

// the counters, then the floats
size_t counter_bytes(const Kv8Cache& c) { return ((size_t)c.rows * c.Hkv * sizeof(int) + 255) / 256 * 256; }
size_t attend_bytes(const Kv8Attend& p, int sms) {
    return counter_bytes(p.c) + sizeof(float) * (kv8_decode_takes(p, sms) ? kv8_decode_floats(p, sms) : kv8_prompt_floats(p, sms));
}

int sms_of(int device, int* n) {
    const cudaError_t e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, device);
    if (e == cudaSuccess) return DEC_OK;
    cudaGetLastError();
    return refuse(DEC_E_CUDA, "device %d: %s", device, cudaGetErrorString(e));
}

int launched(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return DEC_OK;
    cudaGetLastError();
    return refuse(DEC_E_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

}  // namespace

extern "C" {

int dec_kv8_append(const dec_kv8_cache* cache, const dec_kv8_batch* batch, const dec_kv8_new* t, void* stream) {
    Kv8Append p{};
    int rc;
    if ((rc = check_cache(cache, &p.c)) != DEC_OK) return rc;
    if ((rc = check_batch(batch, p.c, &p.b)) != DEC_OK) return rc;
    if (!t) return refuse(DEC_E_INVALID, "tokens is NULL");
    if ((rc = check_dtype(t->dtype, &p.dtype)) != DEC_OK) return rc;
    if ((rc = check_tokens("k", t->k, t->k_stride, p.c.Hkv, p.c.hd, p.dtype, p.b.total)) != DEC_OK) return rc;
    if ((rc = check_tokens("v", t->v, t->v_stride, p.c.Hkv, p.c.hd, p.dtype, p.b.total)) != DEC_OK) return rc;
    if (p.b.total == 0) return DEC_OK;
    p.k = t->k;
    p.v = t->v;
    p.k_stride = t->k_stride;
    p.v_stride = t->v_stride;
    OnDevice on(cache->device);
    if ((rc = launched(on.e, "cudaSetDevice")) != DEC_OK) return rc;
    return launched(kv8_append_launch(p, (cudaStream_t)stream), "dec_kv8_append");
}

int dec_kv8_workspace(const dec_kv8_cache* cache, const dec_kv8_batch* batch, const dec_kv8_attn* attn, size_t* bytes) {
    if (!bytes) return refuse(DEC_E_INVALID, "bytes is NULL");
    Kv8Attend p{};
    int rc, sms;
    if ((rc = check_attend(cache, batch, attn, &p)) != DEC_OK) return rc;
    if ((rc = sms_of(cache->device, &sms)) != DEC_OK) return rc;
    *bytes = attend_bytes(p, sms);
    return DEC_OK;
}

int dec_kv8_attend(const dec_kv8_cache* cache, const dec_kv8_batch* batch, const dec_kv8_attn* attn, void* stream) {
    Kv8Attend p{};
    int rc, sms;
    if ((rc = check_attend(cache, batch, attn, &p)) != DEC_OK) return rc;
    if (p.b.total == 0) return DEC_OK;
    if ((rc = sms_of(cache->device, &sms)) != DEC_OK) return rc;
    const size_t need = attend_bytes(p, sms);
    if (!attn->workspace || attn->workspace_bytes < need)
        return refuse(DEC_E_OOM, "workspace of %zu bytes is smaller than the %zu needed",
                      attn->workspace ? attn->workspace_bytes : (size_t)0, need);
    if (!aligned16(attn->workspace)) return refuse(DEC_E_INVALID, "workspace must be 16-byte aligned");
    p.counters = (int*)attn->workspace;
    p.ws = (float*)((char*)attn->workspace + counter_bytes(p.c));
    OnDevice on(cache->device);
    if ((rc = launched(on.e, "cudaSetDevice")) != DEC_OK) return rc;
    const cudaStream_t s = (cudaStream_t)stream;
    return launched(kv8_decode_takes(p, sms) ? kv8_decode_launch(p, sms, s) : kv8_prompt_launch(p, sms, s), "dec_kv8_attend");
}

}  // extern "C"
