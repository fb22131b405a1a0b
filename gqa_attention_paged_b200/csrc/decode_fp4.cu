// decode_fp4.cu -- GQA decode over a paged cache held in 4 bits (fp4.cuh: e2m1 codes, an e4m3
// scale per token, kv head and 16 dims, an fp32 factor per kv head).
//
// One CTA per (query head, sequence); its warps take the sequence's tokens in turn, lane l
// holds dims l, l + 32, ...; the softmax is the online form, the warps' states are merged
// through shared memory at the end.
#include "fp4.cuh"
#include "quant_kv.h"

namespace gqa {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float fp4_value(uint32_t code) {
    const float m = (code & 7u) < 5u ? 0.5f * (float)(code & 7u) : ((code & 7u) == 5u ? 3.f : 2.f * (float)(code & 7u) - 8.f);
    return code & 8u ? -m : m;
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps) decode_fp4_kernel(const Fp4DecodeArgs a) {
    constexpr int V = D / 32, C = D / 8;
    __shared__ float part[kWarps][D];
    __shared__ float ms[kWarps], ls[kWarps];
    const int h = blockIdx.x, b = blockIdx.y;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    grid_dependents_launch();
    const int kvh = h / (a.Hq / a.Hk);
    int L = a.seq_lens[b];
    if (L < 0 || L > a.pt_stride * a.P) {
        if (threadIdx.x == 0) set_error(a.err, GQA_ERR_BAD_PAGE);
        L = L < 0 ? 0 : a.pt_stride * a.P;
    }
    const size_t row = (size_t)b * a.Hq + h;
    const float kf = (a.k_scale ? a.k_scale[kvh] : 1.f) * a.scale, vf = a.v_scale ? a.v_scale[kvh] : 1.f;
    float q[V], o[V], m = -INFINITY, l = 0.f;
    for (int v = 0; v < V; ++v) {
        q[v] = __bfloat162float(static_cast<const __nv_bfloat16 *>(a.q)[row * D + lane + 32 * v]) * kf;
        o[v] = 0.f;
    }
    for (int t = warp; t < L; t += kWarps) {
        const int phys = a.page_table[(size_t)b * a.pt_stride + t / a.P];
        if (phys < 0 || phys >= a.num_pages) {
            if (lane == 0) set_error(a.err, GQA_ERR_BAD_PAGE);
            continue;
        }
        const size_t tile = fp4_tile_offset(phys, a.Hk, kvh, a.P, t % a.P, D);
        const uint8_t *kt = a.k_pages + tile, *vt = a.v_pages + tile;
        const int tok = t % kFp4Tile, pair = tok / 2;
        float s = 0.f;
        for (int v = 0; v < V; ++v) {
            const int d = lane + 32 * v;
            const uint32_t byte = kt[tok * (D / 2) + d / 2];
            s += q[v] * fp4_value(d & 1 ? byte >> 4 : byte & 15u) * e4m3_to_f32(kt[8 * D + tok * (D / 16) + d / 16]);
        }
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        const float mn = fmaxf(m, s), alpha = mn == -INFINITY ? 1.f : expf(m - mn), p = mn == -INFINITY ? 0.f : expf(s - mn);
        l = l * alpha + p;
        for (int v = 0; v < V; ++v) {
            const int d = lane + 32 * v;
            const uint32_t byte = vt[(pair >> 2) * (4 * D) + (d / C) * (4 * C) + (pair & 3) * C + d % C];
            o[v] = o[v] * alpha + p * fp4_value(tok & 1 ? byte >> 4 : byte & 15u) *
                                      e4m3_to_f32(vt[8 * D + pair * (D / 8) + d / 16 * 2 + (tok & 1)]);
        }
        m = mn;
    }
    for (int v = 0; v < V; ++v) part[warp][lane + 32 * v] = o[v];
    if (lane == 0) {
        ms[warp] = m;
        ls[warp] = l;
    }
    __syncthreads();
    float M = -INFINITY, W = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, ms[w]);
    for (int w = 0; w < kWarps; ++w) W += ms[w] == -INFINITY ? 0.f : ls[w] * expf(ms[w] - M);
    for (int d = threadIdx.x; d < D; d += blockDim.x) {
        float s = 0.f;
        for (int w = 0; w < kWarps; ++w)
            if (ms[w] != -INFINITY) s += part[w][d] * expf(ms[w] - M);
        const float r = W > 0.f ? s / W * vf : W == 0.f ? 0.f : W;
        if (a.out_f32) static_cast<float *>(a.out)[row * D + d] = r;
        else static_cast<__nv_bfloat16 *>(a.out)[row * D + d] = __float2bfloat16(r);
    }
    if (threadIdx.x == 0 && a.lse) a.lse[row] = M + logf(W);
}

}  // namespace

size_t fp4_decode_piece_bytes(int, int, int) { return 0; }

cudaError_t launch_decode_fp4(const Fp4DecodeArgs &a, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.Hq, a.B);
    cfg.blockDim = dim3(32 * kWarps);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return a.D == 128 ? cudaLaunchKernelEx(&cfg, decode_fp4_kernel<128>, a) : cudaLaunchKernelEx(&cfg, decode_fp4_kernel<64>, a);
}

}  // namespace gqa
