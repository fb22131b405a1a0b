// read_kv.cu -- reads a stretch of every sequence's cached tokens back as bf16 values, from
// 4-bit, e4m3 or bf16 pools, through the page table ("TensorRT-LLM与TensorRT核心差异解析",
// section 4.2.2 PageAttention): into rows [token][kv head][dim], or into bf16 pages in the
// pools' own layout (what a kernel that takes bf16 pages then runs on).
//
// A value is code * scale (exact) * factor in fp32, rounded once to bf16.  Bound by HBM: 4-bit
// in, 16-bit out.  One thread per (token, kv head, 16 dims).
#include "fp4.cuh"
#include "quant_kv.h"

namespace gqa {
namespace {

__device__ __forceinline__ void store_bf16x16(uint16_t *dst, const float (&x)[16]) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
    uint4 *d = reinterpret_cast<uint4 *>(dst);
    d[0] = make_uint4(w[0], w[1], w[2], w[3]);
    d[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

__device__ __forceinline__ void f16x2_to_f32(uint32_t h, float &lo, float &hi) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    lo = f.x;
    hi = f.y;
}

// 16 dims (block c) of one token's K row.
template <int D>
__device__ __forceinline__ void read_fp4_k(const uint8_t *tile, int tok, int c, float g, float (&x)[16]) {
    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(tile + tok * (D / 2) + c * 8));
    const float s = e4m3_to_f32(__ldg(tile + 8 * D + tok * (D / 16) + c));
    const uint32_t u[2] = {w.x, w.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t h[4];
        e2m1x8_to_f16(u[i], h);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            f16x2_to_f32(h[k], x[8 * i + 2 * k], x[8 * i + 2 * k + 1]);
            x[8 * i + 2 * k] = x[8 * i + 2 * k] * s * g;
            x[8 * i + 2 * k + 1] = x[8 * i + 2 * k + 1] * s * g;
        }
    }
}

// The same of its V row: the token's nibble of 16 bytes.
template <int D>
__device__ __forceinline__ void read_fp4_v(const uint8_t *tile, int tok, int c, float g, float (&x)[16]) {
    constexpr int C = D / 8;
    const int pair = tok / 2;
    const uint8_t *codes = tile + (pair >> 2) * (4 * D) + (pair & 3) * C;
    const float s = e4m3_to_f32(__ldg(tile + 8 * D + pair * (D / 8) + c * 2 + (tok & 1)));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int d = c * 16 + 4 * i;
        const uint32_t w = __ldg(reinterpret_cast<const uint32_t *>(codes + (d / C) * (4 * C) + d % C));
        uint32_t h[4];
        e2m1x8_to_f16(w, h);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float lo, hi;
            f16x2_to_f32(h[k], lo, hi);
            x[4 * i + k] = ((tok & 1) ? hi : lo) * s * g;
        }
    }
}

template <int KIND, int D>
__global__ void __launch_bounds__(256) read_kv_kernel(const ReadArgs a) {
    constexpr int G = D / 16;
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const int c = (int)(i % G), j = (int)(i / G % a.Hk);
    const long long r = i / G / a.Hk;  // output row, or slot of the output pages
    const long long unit = a.paged ? r / a.P : r;
    if (unit >= a.total) return;
    const int b = sequence_of(a.cu_out, a.B, unit);
    const long long u0 = __ldg(a.cu_out + b), u1 = __ldg(a.cu_out + b + 1);
    if (unit < u0 || unit >= u1) return;
    const int L = __ldg(a.seq_lens + b), s0 = a.starts ? __ldg(a.starts + b) : 0;
    if (L < 0 || L > a.pt_stride * a.P || s0 < 0) {
        set_error(a.err, GQA_ERR_BAD_PAGE);
        return;
    }
    const long long t = a.paged ? (s0 / a.P + (unit - u0)) * a.P + r % a.P : s0 + (unit - u0);
    if (t < s0 || t >= L) {
        // a page's slots outside the stretch are no error, a row past the sequence is
        if (!a.paged || t / a.P > (L - 1) / a.P || L == 0) set_error(a.err, GQA_ERR_BAD_PAGE);
        return;
    }
    const int phys = __ldg(a.page_table + (size_t)b * a.pt_stride + t / a.P);
    if (phys < 0 || phys >= a.num_pages) {
        set_error(a.err, GQA_ERR_BAD_PAGE);
        return;
    }
    const int slot = (int)(t % a.P);
    const size_t dst = (a.paged ? ((size_t)unit * a.Hk + j) * a.P + slot : (size_t)unit * a.Hk + j) * D + c * 16;
    uint16_t *ko = static_cast<uint16_t *>(a.k_out) + dst, *vo = static_cast<uint16_t *>(a.v_out) + dst;
    const size_t row = (((size_t)phys * a.Hk + j) * a.P + slot) * D + c * 16;
    if constexpr (KIND == GQA_KV_BF16) {
        const uint4 *k = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.k_pages) + row);
        const uint4 *v = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.v_pages) + row);
        const uint4 k0 = __ldg(k), k1 = __ldg(k + 1), v0 = __ldg(v), v1 = __ldg(v + 1);
        reinterpret_cast<uint4 *>(ko)[0] = k0;
        reinterpret_cast<uint4 *>(ko)[1] = k1;
        reinterpret_cast<uint4 *>(vo)[0] = v0;
        reinterpret_cast<uint4 *>(vo)[1] = v1;
    } else if constexpr (KIND == GQA_KV_FP8_E4M3) {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            const uint4 w = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(kv ? a.v_pages : a.k_pages) + row));
            const float s = __ldg((kv ? a.v_scale : a.k_scale) + (size_t)phys * a.Hk + j);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
            float x[16];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t h0, h1;
                e4m3x4_to_f16x4(u[e], h0, h1);
                f16x2_to_f32(h0, x[4 * e], x[4 * e + 1]);
                f16x2_to_f32(h1, x[4 * e + 2], x[4 * e + 3]);
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) x[e] *= s;
            store_bf16x16(kv ? vo : ko, x);
        }
    } else {
        const size_t tile = fp4_tile_offset(phys, a.Hk, j, a.P, slot, D);
        float x[16];
        read_fp4_k<D>(static_cast<const uint8_t *>(a.k_pages) + tile, slot % kFp4Tile, c,
                      a.k_scale ? __ldg(a.k_scale + j) : 1.f, x);
        store_bf16x16(ko, x);
        read_fp4_v<D>(static_cast<const uint8_t *>(a.v_pages) + tile, slot % kFp4Tile, c,
                      a.v_scale ? __ldg(a.v_scale + j) : 1.f, x);
        store_bf16x16(vo, x);
    }
}

}  // namespace

cudaError_t launch_read_kv(const ReadArgs &a, cudaStream_t stream) {
    if (a.B == 0 || a.total == 0) return cudaSuccess;
    const long long rows = a.paged ? a.total * a.P : a.total;
    const long long blocks = (rows * a.Hk * (a.D / 16) + 255) / 256;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    void (*k)(const ReadArgs);
    if (a.kv_dtype == GQA_KV_FP4) k = a.D == 128 ? read_kv_kernel<GQA_KV_FP4, 128> : read_kv_kernel<GQA_KV_FP4, 64>;
    else if (a.kv_dtype == GQA_KV_FP8_E4M3)
        k = a.D == 128 ? read_kv_kernel<GQA_KV_FP8_E4M3, 128> : read_kv_kernel<GQA_KV_FP8_E4M3, 64>;
    else k = a.D == 128 ? read_kv_kernel<GQA_KV_BF16, 128> : read_kv_kernel<GQA_KV_BF16, 64>;
    k<<<(unsigned)blocks, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace gqa
