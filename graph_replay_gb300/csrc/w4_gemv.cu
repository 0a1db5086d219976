// w4_gemv.cu -- planning and launch of the few-token products with 4-bit weights
// (w4_gemv.cuh; instantiated in w4_gemv_g32.cu, w4_gemv_g64.cu, w4_gemv_g128.cu).
#include "w4_gemv.cuh"

namespace gd {

const void* w4_gemv_kernel_32(int parts, int nb, int kind);
const void* w4_gemv_kernel_64(int parts, int nb, int kind);
const void* w4_gemv_kernel_128(int parts, int nb, int kind);

namespace {

constexpr size_t SMEM_MOST = 220 * 1024;       // dynamic shared memory of a CTA

int kind_of(const W4Call& c) { return c.glu ? W4_GLU : c.nw > 1 ? W4_STACK : W4_ONE; }
int blocks_of(const W4Gemv& g) { return g.block * g.c.parts() <= 8 ? 1 : 2; }

const void* kernel_of(const W4Gemv& g) {
    const int nb = blocks_of(g), P = g.c.parts(), kind = kind_of(g.c);
    switch (g.c.group()) {
        case 32: return w4_gemv_kernel_32(P, nb, kind);
        case 64: return w4_gemv_kernel_64(P, nb, kind);
        default: return w4_gemv_kernel_128(P, nb, kind);
    }
}

size_t smem_of(const W4Gemv& g) {
    const int P = g.c.parts(), chunks = (g.c.k() + 127) / 128, most = (chunks + g.ks - 1) / g.ks;
    const size_t ring = (size_t)WG_WARPS * g.stages * WG_STEP, x = (size_t)most * g.block * P * 256;
    const size_t f = ((size_t)most * g.block + 3) / 4 * 16 + (g.c.gain ? (size_t)most * 512 : 0);
    const size_t sums = g.ks > 1 ? sizeof(float) * (g.c.glu ? 2 : 1) * g.block * g.rows : 0;
    return ring + x + f + sums + sizeof(float) * g.bufs * WG_WARPS * wg_tokens(P, blocks_of(g)) * WG_PITCH;
}

}  // namespace

// how many clusters of ks CTAs, one an SM, run at a time: they do not cross the chip's SM groups, so it may be less than
// the SMs hold (asked once for each size; devices of one process are alike)
int w4_clusters(int ks, int num_sms) {
    if (ks == 1) return num_sms;
    static std::atomic<int> known[4];
    const int i = ks == 2 ? 1 : ks == 4 ? 2 : 3;
    int n = known[i].load(std::memory_order_relaxed);
    if (n == 0) {
        const void* fn = w4_gemv_kernel_128(2, 1, W4_ONE);
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = (unsigned)ks;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.gridDim = dim3((unsigned)(num_sms / ks * ks));
        cfg.blockDim = dim3(WG_THREADS);
        cfg.dynamicSmemBytes = SMEM_MOST;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        if (raise_smem_cap(fn) != cudaSuccess || cudaOccupancyMaxActiveClusters(&n, fn, &cfg) != cudaSuccess || n < 1) {
            cudaGetLastError();
            n = num_sms / ks;
        }
        if (n > num_sms / ks) n = num_sms / ks;
        if (n < 1) n = 1;
        known[i].store(n, std::memory_order_relaxed);
    }
    return n;
}

cudaError_t w4_gemv_plan(W4Gemv* g, int num_sms) {
    const W4Call& c = g->c;
    const int P = c.parts(), N = c.n(), chunks = (c.k() + 127) / 128, most = WG_MAX_TOKENS / P;
    // as many tokens a CTA as its shared memory holds; the rest in further rows of the grid
    for (g->block = c.tokens < most ? c.tokens : most;; g->block = (g->block + 1) / 2) {
        // rows evenly over the SMs, at least 8 a CTA: a tile has 16, and a CTA of fewer saves nothing
        const int gr = c.glu ? 16 : 32;
        // CTAs along k: the fewest (a cluster: 1, 2, 4 or 8) whose shared memory holds the activations beside a ring of four
        // steps or two
        for (g->ks = 1; g->ks <= 8 && g->ks <= chunks; g->ks *= 2) {
            const int places = w4_clusters(g->ks, num_sms);
            g->rows = (N + places - 1) / places;
            if (g->rows < 8) g->rows = 8;
            g->grid = (N + g->rows - 1) / g->rows;
            const int groups = (g->rows + gr - 1) / gr;
            const int own = (chunks + g->ks - 1) / g->ks;
            // warps along k: as many as have a chunk, but no more than leave each set of warps a row group
            g->wk = WG_WARPS;
            while (g->wk > 1 && (own < g->wk || (groups >= 2 * (WG_WARPS / g->wk) && own < 8 * g->wk))) g->wk /= 2;
            const int sets = WG_WARPS / g->wk, iters = (groups + sets - 1) / sets;
            g->bufs = iters > 1 ? 2 : 1;
            g->stages = WG_STAGES;
            if (smem_of(*g) > SMEM_MOST) g->stages = 2;
            if (smem_of(*g) <= SMEM_MOST) break;
        }
        if (g->ks <= 8 && g->ks <= chunks) break;
        if (g->block == 1) return cudaErrorInvalidValue;
    }
    g->smem = smem_of(*g);
    // the cap once for each kernel and device
    static OncePerDevice once[3][2][2][3];
    const void* fn = kernel_of(*g);
    if (!fn) return cudaErrorInvalidValue;
    return once[c.group() == 32 ? 0 : c.group() == 64 ? 1 : 2][P - 1][blocks_of(*g) - 1][kind_of(c)].run([&] { return raise_smem_cap(fn); });
}

cudaError_t w4_gemv_launch(const W4Gemv& g, cudaStream_t s, bool pdl) {
    const W4Call& c = g.c;
    W4GemvArgs a{};
    int end = 0;
    for (int i = 0; i < 3; ++i) {
        const W4Matrix& w = c.w[i < c.nw ? i : c.nw - 1];
        a.codes[i] = (const uint8_t*)w.codes;
        a.scales[i] = (const __nv_bfloat16*)w.scales;
        end += i < c.nw ? w.n : 0;
        a.end[i] = end;
    }
    a.N = c.n();
    a.K = c.k();
    a.tokens = c.tokens;
    a.block = g.block;
    a.wk = g.wk;
    a.ks = g.ks;
    a.rows = g.rows;
    a.stages = g.stages;
    a.bufs = g.bufs;
    a.act = c.act;
    a.x_f32 = c.x_f32;
    a.gain_f32 = c.gain_f32;
    a.out_f32 = c.out_f32;
    a.x = c.x;
    a.gain = c.gain;
    a.residual = c.residual;
    a.out = c.out;
    a.x_stride = c.x_stride;
    a.residual_stride = c.residual_stride;
    a.out_stride = c.out_stride;
    a.eps = c.eps;
    a.pdl = pdl;
    a.amax = g.amax;
    a.nonfinite = g.nonfinite;
    a.trace = g.trace;
    a.trace_id = g.trace_id;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(g.grid * g.ks, (c.tokens + g.block - 1) / g.block);
    cfg.blockDim = dim3(WG_THREADS);
    cfg.dynamicSmemBytes = g.smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    cfg.attrs = attr;
    if (pdl) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[cfg.numAttrs++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (g.ks > 1) {
        attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
        attr[cfg.numAttrs].val.clusterDim.x = (unsigned)g.ks;
        attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
        ++cfg.numAttrs;
    }
    void* args[] = {&a};
    return cudaLaunchKernelExC(&cfg, kernel_of(g), args);
}

}  // namespace gd
