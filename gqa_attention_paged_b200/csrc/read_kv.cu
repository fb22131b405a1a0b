// read_kv.cu -- reads a stretch of every sequence's cached tokens back as bf16 values, from
// 4-bit, e4m3 or bf16 pools, through the page table ("TensorRT-LLM与TensorRT核心差异解析",
// section 4.2.2 PageAttention): into rows [token][kv head][dim], or into bf16 pages in the
// pools' own layout (what a kernel that takes bf16 pages then runs on).
//
// A value is code * scale (exact) * factor in fp32, rounded once to bf16.  Bound by HBM: 4-bit
// or 8-bit in, 16-bit out.  A CTA takes a run of output rows: first a thread per row finds the
// row's place in the pool (the page table is read once per row, not once per element), then a
// warp takes 16 rows of one kv head at a time, a lane 16 dims of a row at once: all its loads
// go out before the first conversion, and every store is a whole 32-byte sector.  80K tokens of
// e4m3 pages: 79.7 us, 6.3 TB/s (96.8 with 16-byte stores and a look-up per thread); 8 contexts up
// to 4096 of 4-bit pages, 66 MB: 13.9 us, 785 CTAs of which 592 are
// resident, so a wave and a third of another.
#include "fp4.cuh"
#include "quant_kv.h"

namespace gqa {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = 128;  // output rows of a CTA
constexpr int kGroup = 16;     // rows a warp takes at a time

// Eight f16x2 -> 16 values times g as bf16.
__device__ __forceinline__ void scaled_bf16(const uint32_t (&h)[8], float g, uint32_t (&w)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        w[i] = pack_bf16(f.x * g, f.y * g);
    }
}

__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
    const __half2 d = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&d);
}

// The raw bytes of 16 dims (block c) of one cached row, keys or values.
template <int KIND>
struct Raw {
    uint4 a, b;
    float s;
    uint32_t sc;
};

// `q`: the row's index in the pool, ((page * Hk + kv head) * P + slot).
template <int KIND, int D, bool IS_V>
__device__ __forceinline__ void fetch(Raw<KIND> &x, const void *pages, const float *scale, int q, int c, int pshift) {
    if constexpr (KIND == GQA_KV_BF16) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(pages) + (size_t)q * D + c * 16);
        x.a = __ldg(p);
        x.b = __ldg(p + 1);
    } else if constexpr (KIND == GQA_KV_FP8_E4M3) {
        x.a = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(pages) + (size_t)q * D + c * 16));
        x.s = __ldg(scale + (q >> pshift));
    } else {
        const uint8_t *tile = static_cast<const uint8_t *>(pages) + (size_t)(q / kFp4Tile) * fp4_tile_bytes(D);
        const int tok = q % kFp4Tile;
        if constexpr (!IS_V) {
            const uint2 w = __ldg(reinterpret_cast<const uint2 *>(tile + tok * (D / 2) + c * 8));
            x.a.x = w.x;
            x.a.y = w.y;
            x.sc = __ldg(tile + 8 * D + tok * (D / 16) + c);
        } else {
            // both tokens of the pair; the other one's row reads the same bytes
            constexpr int C = D / 8;
            const int pair = tok / 2;
            const uint8_t *codes = tile + (pair >> 2) * (4 * D) + (pair & 3) * C;
            if constexpr (C == 16) {
                x.a = __ldg(reinterpret_cast<const uint4 *>(codes + c * (4 * C)));
            } else {
                const uint2 u = __ldg(reinterpret_cast<const uint2 *>(codes + (2 * c) * (4 * C)));
                const uint2 v = __ldg(reinterpret_cast<const uint2 *>(codes + (2 * c + 1) * (4 * C)));
                x.a = make_uint4(u.x, u.y, v.x, v.y);
            }
            x.sc = __ldg(tile + 8 * D + pair * (D / 8) + c * 2 + (tok & 1));
        }
    }
}

template <int KIND, bool IS_V>
__device__ __forceinline__ void convert(const Raw<KIND> &x, int q, float g, uint32_t (&w)[8]) {
    if constexpr (KIND == GQA_KV_BF16) {
        const uint32_t u[8] = {x.a.x, x.a.y, x.a.z, x.a.w, x.b.x, x.b.y, x.b.z, x.b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = u[i];
    } else if constexpr (KIND == GQA_KV_FP8_E4M3) {
        const uint32_t u[4] = {x.a.x, x.a.y, x.a.z, x.a.w};
        uint32_t h[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) e4m3x4_to_f16x4(u[i], h[2 * i], h[2 * i + 1]);
        scaled_bf16(h, x.s, w);
    } else {
        const uint32_t one = e4m3x2_to_f16(x.sc), sc = __byte_perm(one, one, 0x1010);
        uint32_t h[8];
        if constexpr (!IS_V) {
            const uint32_t u[2] = {x.a.x, x.a.y};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t t[4];
                e2m1x8_to_f16(u[i], t);
#pragma unroll
                for (int k = 0; k < 4; ++k) h[4 * i + k] = t[k];
            }
        } else {
            // this token's nibbles of 16 bytes, gathered into 8 bytes
            const uint32_t u[4] = {x.a.x, x.a.y, x.a.z, x.a.w};
            const int shift = (q & 1) * 4;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t n = (u[i] >> shift) & 0x0f0f0f0fu;  // 0a 0b 0c 0d
                const uint32_t m = (n | (n >> 4)) & 0x00ff00ffu;   // ba in byte 0, dc in byte 2
                uint32_t t[4];
                e2m1x8_to_f16(m, t);
                h[2 * i] = t[0];
                h[2 * i + 1] = t[2];
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = f16x2_mul(h[i], sc);
        scaled_bf16(h, g, w);
    }
}

template <int KIND, int D>
__global__ void __launch_bounds__(kThreads) read_kv_kernel(const ReadArgs a, const int rows, const long long total_rows,
                                                           const int pshift, const bool wide) {
    constexpr int G = D / 16, kAt = 32 / G, kIts = kGroup / kAt;  // rows of a warp at once, and how often
    __shared__ int place[kMaxRows];
    __shared__ Sequences<int64_t> seqs;
    const long long r0 = (long long)blockIdx.x * rows;
    const int P = 1 << pshift;
    grid_dependency_wait();
    grid_dependents_launch();

    // ---- where the CTA's rows lie in the pool (head 0; -1: not read)
    seqs.load(a.cu_out, a.seq_lens, a.B);
    __syncthreads();
    if (threadIdx.x < rows) {
        const long long r = r0 + threadIdx.x;
        int at = -1;
        if (r < total_rows) {
            const long long unit = a.paged ? r >> pshift : r;
            const int b = sequence_of(seqs.cu, a.B, unit);
            const long long u0 = seqs.cu[b], u1 = seqs.cu[b + 1];
            const int L = seqs.lens[b], s0 = a.starts ? __ldg(a.starts + b) : 0;
            if (unit >= u0 && unit < u1) {
                const bool ok = L >= 0 && L <= a.pt_stride * P && s0 >= 0;
                const long long t = a.paged ? (((s0 >> pshift) + (unit - u0)) << pshift) + (r & (P - 1)) : s0 + (unit - u0);
                if (ok && t >= s0 && t < L) {
                    const int phys = __ldg(a.page_table + (size_t)b * a.pt_stride + (t >> pshift));
                    if (phys >= 0 && phys < a.num_pages) at = phys * a.Hk * P + (int)(t & (P - 1));
                    else set_error(a.err, GQA_ERR_BAD_PAGE);
                } else if (!ok || !a.paged || L == 0 || (t >> pshift) > ((L - 1) >> pshift)) {
                    // (a page's slots outside the stretch are no error)
                    set_error(a.err, GQA_ERR_BAD_PAGE);
                }
            }
        }
        place[threadIdx.x] = at;
    }
    __syncthreads();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % G;
    const int tasks = rows / kGroup * a.Hk;
#pragma unroll 1
    for (int task = warp; task < tasks; task += kThreads / 32) {
        const int grp = task / a.Hk, j = task - grp * a.Hk;
        const int row = grp * kGroup + lane / G;
        const float gk = KIND == GQA_KV_FP4 && a.k_scale ? __ldg(a.k_scale + j) : 1.f;
        const float gv = KIND == GQA_KV_FP4 && a.v_scale ? __ldg(a.v_scale + j) : 1.f;
        Raw<KIND> k[kIts], v[kIts];
        int q[kIts];
#pragma unroll
        for (int i = 0; i < kIts; ++i) {
            const int at = place[row + i * kAt];
            q[i] = at < 0 ? -1 : at + (j << pshift);
            if (at < 0) continue;
            fetch<KIND, D, false>(k[i], a.k_pages, a.k_scale, q[i], c, pshift);
            fetch<KIND, D, true>(v[i], a.v_pages, a.v_scale, q[i], c, pshift);
        }
#pragma unroll
        for (int i = 0; i < kIts; ++i) {
            if (q[i] < 0) continue;
            const long long r = r0 + row + i * kAt;
            const size_t dst = (size_t)(a.paged ? (((r >> pshift) * a.Hk + j) << pshift) + (r & (P - 1)) : r * a.Hk + j) * D + c * 16;
            uint32_t w[8];
            convert<KIND, false>(k[i], q[i], gk, w);
            store32(static_cast<uint16_t *>(a.k_out) + dst, w, wide);
            convert<KIND, true>(v[i], q[i], gv, w);
            store32(static_cast<uint16_t *>(a.v_out) + dst, w, wide);
        }
    }
}

}  // namespace

cudaError_t launch_read_kv(const ReadArgs &a, cudaStream_t stream) {
    if (a.B == 0 || a.total == 0) return cudaSuccess;
    // enough groups of 16 rows for a warp each, over the kv heads
    const int rows = kGroup * (a.Hk >= 8 ? 1 : (8 + a.Hk - 1) / a.Hk);
    const int pshift = a.P == 16 ? 4 : (a.P == 32 ? 5 : 6);
    const long long total_rows = a.paged ? a.total << pshift : a.total;
    const long long blocks = (total_rows + rows - 1) / rows;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    const bool wide = ((reinterpret_cast<uintptr_t>(a.k_out) | reinterpret_cast<uintptr_t>(a.v_out)) & 31) == 0;
    void (*k)(const ReadArgs, int, long long, int, bool);
    if (a.kv_dtype == GQA_KV_FP4) k = a.D == 128 ? read_kv_kernel<GQA_KV_FP4, 128> : read_kv_kernel<GQA_KV_FP4, 64>;
    else if (a.kv_dtype == GQA_KV_FP8_E4M3)
        k = a.D == 128 ? read_kv_kernel<GQA_KV_FP8_E4M3, 128> : read_kv_kernel<GQA_KV_FP8_E4M3, 64>;
    else k = a.D == 128 ? read_kv_kernel<GQA_KV_BF16, 128> : read_kv_kernel<GQA_KV_BF16, 64>;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k, a, rows, total_rows, pshift, wide);
}

}  // namespace gqa
