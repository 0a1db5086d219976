// w4.cu -- the C ABI of the 4-bit weights: argument checks and launches on the
// caller's stream.  No handle, no allocation, no wait: each call only launches
// kernels, so it can be recorded into a graph.
#include <limits.h>
#include <stdarg.h>
#include <stdio.h>

#include <cmath>

#include "graphdec.h"
#include "internal.h"

using namespace gd;

namespace {

int refuse(int code, const char* fmt, ...) {
    char buf[256];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_call_message(buf);
    return code;
}

bool aligned(const void* p, unsigned to) { return ((uintptr_t)p & (to - 1)) == 0; }

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

int launched(cudaError_t e, const char* what) {
    if (e == cudaSuccess) return DEC_OK;
    cudaGetLastError();
    return refuse(DEC_E_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

int sms_of(int device, int* n) {
    const cudaError_t e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, device);
    if (e == cudaSuccess) return DEC_OK;
    cudaGetLastError();
    return refuse(DEC_E_CUDA, "device %d: %s", device, cudaGetErrorString(e));
}

}  // namespace

namespace gd {
int w4_check(const char* what, const dec_w4_weight* w, W4Matrix* out) {
    if (!w) return refuse(DEC_E_INVALID, "%s is NULL", what);
    if (!w->codes || !w->scales) return refuse(DEC_E_INVALID, "%s: codes and scales are required", what);
    if (!aligned(w->codes, 16) || !aligned(w->scales, 2))
        return refuse(DEC_E_INVALID, "%s: codes must be 16-byte, scales 2-byte aligned", what);
    if (w->n < 1 || w->k < 1) return refuse(DEC_E_INVALID, "%s: n and k must be >= 1", what);
    if (w->group != 32 && w->group != 64 && w->group != 128)
        return refuse(DEC_E_UNSUPPORTED, "%s: group %d unsupported (32, 64 or 128)", what, w->group);
    if (w->k % w->group) return refuse(DEC_E_INVALID, "%s: k must be a multiple of group", what);
    if (w->k > (1 << 20) || (int64_t)w->n * w->k > (1ll << 33))
        return refuse(DEC_E_UNSUPPORTED, "%s: at most 2^20 columns and 2^33 weights", what);
    if (w->device < 0) return refuse(DEC_E_INVALID, "%s: device must be >= 0", what);
    *out = W4Matrix{w->codes, w->scales, w->n, w->k, w->group};
    return DEC_OK;
}
}  // namespace gd

namespace {

int check_dtype(const char* what, int dtype, bool* f32) {
    if (dtype != DEC_DTYPE_F32 && dtype != DEC_DTYPE_BF16)
        return refuse(DEC_E_INVALID, "%s must be DEC_DTYPE_F32 or DEC_DTYPE_BF16", what);
    *f32 = dtype == DEC_DTYPE_F32;
    return DEC_OK;
}

// a matrix that is read or written in 16-byte pieces
int check_rows(const char* what, const void* p, int64_t stride, int64_t cols, bool f32) {
    if (!p) return refuse(DEC_E_INVALID, "%s is NULL", what);
    if (!aligned(p, 16)) return refuse(DEC_E_INVALID, "%s must be 16-byte aligned", what);
    if (stride < cols || stride > (1ll << 40) || (stride * (f32 ? 4 : 2)) % 16)
        return refuse(DEC_E_INVALID, "%s: the stride must hold a row and be a multiple of 16 bytes", what);
    return DEC_OK;
}

// a matrix that is read or written one value at a time
int check_values(const char* what, const void* p, int64_t stride, int64_t cols, bool f32) {
    if (!p) return refuse(DEC_E_INVALID, "%s is NULL", what);
    if (!aligned(p, f32 ? 4 : 2)) return refuse(DEC_E_INVALID, "%s must be aligned to its type", what);
    if (stride < cols || stride > (1ll << 40)) return refuse(DEC_E_INVALID, "%s: the stride must hold a row", what);
    return DEC_OK;
}

// whether rows of two matrices with as many rows meet: x and out may be columns of one wider matrix
bool meet(const void* a, int64_t a_stride, int64_t a_bytes, const void* b, int64_t b_stride, int64_t b_bytes, int64_t rows) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    if (x + (uint64_t)((rows - 1) * a_stride + a_bytes) <= y || y + (uint64_t)((rows - 1) * b_stride + b_bytes) <= x) return false;
    if (rows == 1 || a_stride != b_stride) return true;
    const int64_t off = (int64_t)((y - x) % (uint64_t)a_stride);   // y's column in a's rows
    const int64_t at = y >= x ? off : (int64_t)(a_stride - (int64_t)((x - y) % (uint64_t)a_stride)) % a_stride;
    return at < a_bytes || at + b_bytes > a_stride;
}

// whether one of `rows` rows, `bytes` each and `stride` bytes apart, has a byte of [q, q + qbytes)
bool rows_touch(const void* p, int64_t stride, int64_t bytes, int64_t rows, const void* q, int64_t qbytes) {
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    if (b + (uint64_t)qbytes <= a) return false;
    const uint64_t i = b > a ? (b - a) / (uint64_t)stride : 0;   // the last row that starts at or before q, or the first
    if (i < (uint64_t)rows && a + i * stride + bytes > b) return true;
    return i + 1 < (uint64_t)rows && a + (i + 1) * stride < b + (uint64_t)qbytes;
}

int check_apart(const char* what, const dec_w4_weight* w, const void* p, int64_t stride, bool f32) {
    const int64_t size = f32 ? 4 : 2, codes = (int64_t)w->n * w->k / 2, scales = (int64_t)w->n * (w->k / w->group) * 2;
    if (rows_touch(p, stride * size, w->k * size, w->n, w->codes, codes) || rows_touch(p, stride * size, w->k * size, w->n, w->scales, scales) ||
        rows_touch(w->codes, codes, codes, 1, w->scales, scales))
        return refuse(DEC_E_INVALID, "%s, codes and scales overlap", what);
    return DEC_OK;
}

// sizes, types and whether there is a gain: what a plan follows from
int check_sizes(const dec_w4_weight* w, const dec_w4_weight* up, bool glu, const dec_w4_call* c, W4Call* p) {
    int rc;
    *p = W4Call{};
    if ((rc = w4_check(glu ? "gate" : "w", w, &p->w[0])) != DEC_OK) return rc;
    p->nw = 1;
    p->glu = glu;
    if (glu) {
        if ((rc = w4_check("up", up, &p->w[1])) != DEC_OK) return rc;
        if (up->n != w->n || up->k != w->k || up->group != w->group || up->device != w->device)
            return refuse(DEC_E_INVALID, "gate and up must have one shape, group and device");
        p->nw = 2;
    }
    if (!c) return refuse(DEC_E_INVALID, "call is NULL");
    if (c->tokens < 0) return refuse(DEC_E_INVALID, "tokens must be >= 0");
    if ((int64_t)c->tokens * w->n > INT_MAX) return refuse(DEC_E_UNSUPPORTED, "tokens * n: at most 2^31 - 1");
    if (c->tokens > (1 << 21)) return refuse(DEC_E_UNSUPPORTED, "tokens = %d: at most 2^21", c->tokens);
    if ((int64_t)c->tokens * w->k > INT_MAX) return refuse(DEC_E_UNSUPPORTED, "tokens * k: at most 2^31 - 1");
    if ((rc = check_dtype("x_dtype", c->x_dtype, &p->x_f32)) != DEC_OK) return rc;
    if ((rc = check_dtype("out_dtype", c->out_dtype, &p->out_f32)) != DEC_OK) return rc;
    if (c->gain) {
        if ((rc = check_dtype("gain_dtype", c->gain_dtype, &p->gain_f32)) != DEC_OK) return rc;
        if (!(c->eps >= 0.0) || !std::isfinite((float)c->eps)) return refuse(DEC_E_INVALID, "eps must be finite and >= 0");
    }
    if (glu) {
        if (c->act != DEC_ACT_SILU && c->act != DEC_ACT_GELU_TANH)
            return refuse(DEC_E_INVALID, "act must be DEC_ACT_SILU or DEC_ACT_GELU_TANH");
        if (c->residual) return refuse(DEC_E_INVALID, "dec_w4_glu takes no residual");
    }
    p->act = c->act;
    p->tokens = c->tokens;
    p->gain = c->gain;
    p->eps = (float)c->eps;
    return DEC_OK;
}

// the pointers, strides and overlaps of a call whose sizes are checked
int check_tensors(const dec_w4_weight* w, const dec_w4_call* c, W4Call* p) {
    int rc;
    if (!aligned(c->gain, 16)) return refuse(DEC_E_INVALID, "gain must be 16-byte aligned");
    if (!c->err || !aligned(c->err, 4)) return refuse(DEC_E_INVALID, "err is required");
    if (c->tokens > 0) {
        if ((rc = check_rows("x", c->x, c->x_stride, w->k, p->x_f32)) != DEC_OK) return rc;
        if ((rc = check_values("out", c->out, c->out_stride, w->n, p->out_f32)) != DEC_OK) return rc;
        if (c->residual) {
            if ((rc = check_values("residual", c->residual, c->residual_stride, w->n, p->out_f32)) != DEC_OK) return rc;
            if (c->residual == c->out && c->residual_stride != c->out_stride)
                return refuse(DEC_E_INVALID, "a residual that is out must have its stride");
        }
        const int64_t xs = p->x_f32 ? 4 : 2, os = p->out_f32 ? 4 : 2, n = w->n, k = w->k;
        if (meet(c->x, c->x_stride * xs, k * xs, c->out, c->out_stride * os, n * os, c->tokens) ||
            (c->gain && meet(c->gain, k * 4, k * (p->gain_f32 ? 4 : 2), c->out, c->out_stride * os,
                             ((int64_t)c->tokens - 1) * c->out_stride * os + n * os, 1)) ||
            (c->residual && c->residual != c->out &&
             meet(c->residual, c->residual_stride * os, n * os, c->out, c->out_stride * os, n * os, c->tokens)))
            return refuse(DEC_E_INVALID, "out overlaps x, the gain or the residual (it may be the residual itself)");
    }
    p->x = c->x;
    p->residual = c->residual;
    p->out = c->out;
    p->x_stride = c->x_stride;
    p->residual_stride = c->residual_stride;
    p->out_stride = c->out_stride;
    p->err = c->err;
    return DEC_OK;
}

// how a call runs, and what it needs of workspace
struct Plan {
    bool few;
    W4Gemv gemv;
    W4Gemm gemm;
    size_t bytes;
};

// Few tokens (at most 16 columns of activation parts) go to w4_gemv.cu: 8 fp32 tokens, 14336 -> 4096, take 22 us there and
// 40 in w4_gemm.cu; 9 bf16 ones as long in both, 16 longer.  Columns too many for its shared memory go there too
cudaError_t plan_of(const W4Call& c, int sms, Plan* p) {
    p->few = c.tokens * c.parts() <= 16;
    p->bytes = 0;
    if (p->few) {
        p->gemv = W4Gemv{};
        p->gemv.c = c;
        if (w4_gemv_plan(&p->gemv, sms) == cudaSuccess) return cudaSuccess;
        cudaGetLastError();
        p->few = false;
    }
    p->gemm = W4Gemm{};
    p->gemm.c = c;
    const cudaError_t e = w4_gemm_plan(&p->gemm, sms);
    p->bytes = w4_gemm_bytes(p->gemm);
    return e;
}

int run(const dec_w4_weight* w, const dec_w4_weight* up, bool glu, const dec_w4_call* call, void* stream) {
    W4Call c;
    int rc, sms;
    if ((rc = check_sizes(w, up, glu, call, &c)) != DEC_OK || (rc = check_tensors(w, call, &c)) != DEC_OK) return rc;
    if (c.tokens == 0) return DEC_OK;
    const char* what = glu ? "dec_w4_glu" : "dec_w4_linear";
    OnDevice on(w->device);
    if ((rc = launched(on.e, "cudaSetDevice")) != DEC_OK) return rc;
    if ((rc = sms_of(w->device, &sms)) != DEC_OK) return rc;
    Plan p;
    if ((rc = launched(plan_of(c, sms, &p), what)) != DEC_OK) return rc;
    if (p.bytes && (!call->workspace || call->workspace_bytes < p.bytes))
        return refuse(DEC_E_OOM, "workspace of %zu bytes is smaller than the %zu needed",
                      call->workspace ? call->workspace_bytes : (size_t)0, p.bytes);
    if (!aligned(call->workspace, 256)) return refuse(DEC_E_INVALID, "workspace must be 256-byte aligned");
    if (!p.few) {
        p.gemm.ws = call->workspace;
        return launched(w4_gemm_launch(p.gemm, (cudaStream_t)stream), what);
    }
    return launched(w4_gemv_launch(p.gemv, (cudaStream_t)stream, false), what);
}

}  // namespace

extern "C" {

int dec_w4_quantize(const dec_w4_weight* w, const void* src, int64_t src_stride, int32_t dtype, void* stream) {
    W4Matrix m;
    bool f32;
    int rc, sms;
    if ((rc = w4_check("w", w, &m)) != DEC_OK) return rc;
    if ((rc = check_dtype("dtype", dtype, &f32)) != DEC_OK) return rc;
    if ((rc = check_rows("src", src, src_stride, w->k, f32)) != DEC_OK) return rc;
    if ((rc = check_apart("src", w, src, src_stride, f32)) != DEC_OK) return rc;
    OnDevice on(w->device);
    if ((rc = launched(on.e, "cudaSetDevice")) != DEC_OK) return rc;
    if ((rc = sms_of(w->device, &sms)) != DEC_OK) return rc;
    return launched(w4_quantize_launch(m, src, src_stride, f32, sms, (cudaStream_t)stream), "dec_w4_quantize");
}

int dec_w4_dequantize(const dec_w4_weight* w, void* dst, int64_t dst_stride, int32_t dtype, void* stream) {
    W4Matrix m;
    bool f32;
    int rc, sms;
    if ((rc = w4_check("w", w, &m)) != DEC_OK) return rc;
    if ((rc = check_dtype("dtype", dtype, &f32)) != DEC_OK) return rc;
    if ((rc = check_rows("dst", dst, dst_stride, w->k, f32)) != DEC_OK) return rc;
    if ((rc = check_apart("dst", w, dst, dst_stride, f32)) != DEC_OK) return rc;
    OnDevice on(w->device);
    if ((rc = launched(on.e, "cudaSetDevice")) != DEC_OK) return rc;
    if ((rc = sms_of(w->device, &sms)) != DEC_OK) return rc;
    return launched(w4_values_launch(m, dst, dst_stride, f32, sms, (cudaStream_t)stream), "dec_w4_dequantize");
}

int dec_w4_workspace(const dec_w4_weight* w, const dec_w4_weight* up, const dec_w4_call* call, size_t* bytes) {
    if (!bytes) return refuse(DEC_E_INVALID, "bytes is NULL");
    W4Call c;
    int rc, sms;
    if ((rc = check_sizes(w, up, up != nullptr, call, &c)) != DEC_OK) return rc;
    *bytes = 0;
    if (c.tokens == 0) return DEC_OK;
    OnDevice on(w->device);
    if ((rc = launched(on.e, "cudaSetDevice")) != DEC_OK) return rc;
    if ((rc = sms_of(w->device, &sms)) != DEC_OK) return rc;
    Plan p;
    if ((rc = launched(plan_of(c, sms, &p), "dec_w4_workspace")) != DEC_OK) return rc;
    *bytes = p.bytes;
    return DEC_OK;
}

int dec_w4_linear(const dec_w4_weight* w, const dec_w4_call* call, void* stream) { return run(w, nullptr, false, call, stream); }

int dec_w4_glu(const dec_w4_weight* gate, const dec_w4_weight* up, const dec_w4_call* call, void* stream) {
    return run(gate, up, true, call, stream);
}

}  // extern "C"
