// kv8_attend.cu -- attention over the 8-bit K/V cache: one warp for each token
// and query head, a running softmax over the positions that the token sees.
#include "kv8.cuh"

namespace gd {

namespace {

template <typename T>
__global__ void k_kv8_attend(const Kv8Attend p) {
    const int warp = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
    const Kv8Cache& c = p.c;
    const int t = warp / p.Hq, hq = warp % p.Hq, h = hq / (p.Hq / c.Hkv);
    if (t >= p.b.total) return;
    Kv8Row row{0, 0, 0};
    int r = 0;
    for (; r < c.rows; ++r)
        if (kv8_row(p.b, c.ppr * c.page, r, &row) && t >= row.t0 && t < row.t0 + row.n) break;
    if (r == c.rows) return;
    const int pos = row.len - row.n + t - row.t0, per = c.hd / 32;
    float q[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
    for (int i = 0; i < per; ++i)
        q[i] = Elem<T>::load1(static_cast<const T*>(p.q) + t * p.q_stride + hq * c.hd + lane * per + i);
    for (int j = 0; j <= pos; ++j) {
        if (!kv8_sees(pos, j, p.window, p.sinks)) continue;
        const int page = kv8_page(c, p.b.err, r, j / c.page);
        if (page < 0) continue;
        const size_t at = ((size_t)page * c.Hkv + h) * c.page + j % c.page;
        const size_t sc = ((size_t)page * c.Hkv + h) * (c.page / c.block) + j % c.page / c.block;
        float s = 0.f, f[4];
        for (int i = 0; i < per; ++i) {
            e4m3x4_to_f32(c.k[at * c.hd + lane * per + i], f);
            s += q[i] * f[0];
        }
        s = warp_sum(s) * pow2i(c.ks[sc] - 127) * p.scale;
        const float m2 = fmaxf(m, s), a = expf(m - m2), w = expf(s - m2);
        l = l * a + w;
        for (int i = 0; i < per; ++i) {
            e4m3x4_to_f32(c.v[at * c.hd + lane * per + i], f);
            o[i] = o[i] * a + w * (f[0] * pow2i(c.vs[sc] - 127));
        }
        m = m2;
    }
    for (int i = 0; i < per; ++i)
        Elem<T>::round_store(l == 0.f ? 0.f : o[i] / l, static_cast<T*>(p.out) + t * p.out_stride + hq * c.hd + lane * per + i);
}

}  // namespace

size_t kv8_attend_floats(const Kv8Attend& p, int num_sms) { return kv8_decode_takes(p) ? kv8_decode_floats(p, num_sms) : 0; }

cudaError_t kv8_attend_launch(const Kv8Attend& p, int num_sms, cudaStream_t s) {
    if (kv8_decode_takes(p)) return kv8_decode_launch(p, num_sms, s);
    const int blocks = (p.b.total * p.Hq + 3) / 4;
    if (p.dtype == W_BF16) k_kv8_attend<__nv_bfloat16><<<blocks, 128, 0, s>>>(p);
    else k_kv8_attend<float><<<blocks, 128, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace gd
