// write_kv.cu -- writes the newest tokens of every sequence into the paged cache: a prefill
// chunk's, or a decode step's one token ("TensorRT对Grouped Query Attention的支持进展", sections
// "动态形状与KV Cache管理" and "与动态批处理协同"), quantised on the way for 4-bit and e4m3 pools.
//
// 4-bit pools (write_fp4_kernel).  A block of 16 dims of one token, with g the head's factor:
//   a = max |x|,  sf = e4m3(min(fl(a / fl(6 g)), 448)),  s = fl(sf g),  code = e2m1(fl(x / s))
// (fl: fp32 rounding).  The quotients are IEEE divisions: a reciprocal would move values off
// the exact ties that bf16 inputs hit.  A block whose scale rounds to 0 stores zeros, one that
// holds a NaN stores a NaN scale (it reads back as NaN), infinities saturate.  One thread per
// (row, kv head, block): 32 bytes in, 8 code bytes and a scale byte out for K.  V bytes hold
// two tokens, so the thread of the even token takes both (a chunk's first token may be the odd
// one alone; half-written bytes keep their other nibble).
//
// e4m3 and bf16 pools (write_page_kernel).  One CTA per (page of the chunk, kv head,
// sequence).  A page whose first slot is in the chunk takes its scale from the chunk's tokens
// in it, absmax / 448 (1 when they are all zero); a page that was begun earlier keeps its
// scale.  A chunk of one token is gqa_paged_append_kv()'s rule.
#include "fp4.cuh"
#include "quant_kv.h"

namespace gqa {
namespace {

// Where sequence b's rows go: first row, number of rows, first token.  False (and the error
// word set) when the lengths do not fit one another.
__device__ __forceinline__ bool chunk_of(const WriteArgs &a, int b, int &row0, int &n, int &tok0) {
    const int L = __ldg(a.seq_lens + b);
    if (a.cu_q) {
        row0 = __ldg(a.cu_q + b);
        n = __ldg(a.cu_q + b + 1) - row0;
    } else {
        row0 = b;
        n = L > 0 ? 1 : 0;
    }
    tok0 = L - n;
    if (n < 0 || n > a.max_q_len || row0 < 0 || (long long)row0 + n > a.total_q || tok0 < 0 ||
        L > a.pt_stride * a.P) {
        set_error(a.err, GQA_ERR_BAD_PAGE);
        return false;
    }
    return true;
}

// Scale code of a block of 16 and its values over the scale; zeros where the scale is 0 or NaN.
__device__ __forceinline__ uint32_t quantise_block(float (&x)[16], float g) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) a = max_nan(a, fabsf(x[i]));
    const uint32_t sf = f32_to_e4m3(a / (6.f * g));
    const float s = e4m3_to_f32(sf) * g;
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = s > 0.f ? x[i] / s : 0.f;
    return sf;
}

__device__ __forceinline__ void load_block(const void *rows, long long stride, long long r, int at,
                                           float (&x)[16]) {
    const uint4 *p = reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(rows) + r * stride + at);
    unpack_bf16x8(__ldg(p), x);
    unpack_bf16x8(__ldg(p + 1), x + 8);
}

template <int D>
__global__ void __launch_bounds__(256) write_fp4_kernel(const WriteArgs a) {
    constexpr int G = D / 16, C = D / 8;
    grid_dependency_wait();
    grid_dependents_launch();
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const int c = (int)(i % G), j = (int)(i / G % a.Hk);
    const long long r = i / G / a.Hk;
    if (r >= a.total_q) return;
    const int b = a.cu_q ? sequence_of(a.cu_q, a.B, r) : (int)r;
    int row0, n, tok0;
    if (!chunk_of(a, b, row0, n, tok0) || r < row0 || r >= row0 + n) return;
    const int t = tok0 + (int)(r - row0);
    const int phys = __ldg(a.page_table + (size_t)b * a.pt_stride + t / a.P);
    if (phys < 0 || phys >= a.num_pages) {
        set_error(a.err, GQA_ERR_BAD_PAGE);
        return;
    }
    const size_t tile = fp4_tile_offset(phys, a.Hk, j, a.P, t % a.P, D);
    const int tok = t % kFp4Tile, pair = tok / 2;
    const int at = j * D + c * 16;

    // ---- K: this token's block
    float x[16];
    load_block(a.k_new, a.k_stride, r, at, x);
    const uint32_t ks = quantise_block(x, a.k_scale ? __ldg(a.k_scale + j) : 1.f);
    {
        uint8_t *kt = static_cast<uint8_t *>(a.k_pages) + tile;
        const float l0[4] = {x[0], x[2], x[4], x[6]}, h0[4] = {x[1], x[3], x[5], x[7]};
        const float l1[4] = {x[8], x[10], x[12], x[14]}, h1[4] = {x[9], x[11], x[13], x[15]};
        *reinterpret_cast<uint2 *>(kt + tok * (D / 2) + c * 8) =
            make_uint2(f32_to_e2m1x8(l0, h0), f32_to_e2m1x8(l1, h1));
        kt[8 * D + tok * G + c] = (uint8_t)ks;
    }

    // ---- V: the pair's blocks, by the even token's thread (or the odd one's, when it is the
    // chunk's first)
    const bool odd = tok & 1;
    if (odd && r != row0) return;
    const bool both = !odd && r + 1 < row0 + n;
    const float gv = a.v_scale ? __ldg(a.v_scale + j) : 1.f;
    float y[16];
    uint32_t s0, s1 = 0;
    load_block(a.v_new, a.v_stride, r, at, x);
    s0 = quantise_block(x, gv);
    if (both) {
        load_block(a.v_new, a.v_stride, r + 1, at, y);
        s1 = quantise_block(y, gv);
    } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = 0.f;
    }
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float l[4] = {x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]};
        const float h[4] = {y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]};
        w[e] = f32_to_e2m1x8(l, h);
    }
    uint8_t *vt = static_cast<uint8_t *>(a.v_pages) + tile;
    uint8_t *sc = vt + 8 * D + pair * (2 * G) + c * 2;
    uint8_t *codes = vt + (pair >> 2) * (4 * D) + (pair & 3) * C;
    if (both) {
        *reinterpret_cast<uint16_t *>(sc) = (uint16_t)(s0 | (s1 << 8));
    } else {
        sc[tok & 1] = (uint8_t)s0;
        const uint32_t keep = odd ? 0x0f0f0f0fu : 0xf0f0f0f0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int d = c * 16 + 4 * e;
            const uint32_t old = *reinterpret_cast<const uint32_t *>(codes + (d / C) * (4 * C) + d % C);
            w[e] = (old & keep) | ((odd ? w[e] << 4 : w[e]) & ~keep);
        }
    }
    if constexpr (C == 16) {
        *reinterpret_cast<uint4 *>(codes + c * (4 * C)) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        *reinterpret_cast<uint2 *>(codes + (2 * c) * (4 * C)) = make_uint2(w[0], w[1]);
        *reinterpret_cast<uint2 *>(codes + (2 * c + 1) * (4 * C)) = make_uint2(w[2], w[3]);
    }
}

constexpr int kPageThreads = 256;
constexpr int kPageMaxChunks = 64 * 128 / 8 / kPageThreads;  // 16-byte loads a thread holds

template <bool FP8>
__device__ __forceinline__ void write_page(const WriteArgs &a, const void *rows, long long stride,
                                           void *pages, float *scales, long long row, int ntok, int slot,
                                           int phys, int j, float *red) {
    const int per = a.D / 8, chunks = ntok * per;  // 8 elements each
    uint4 w[kPageMaxChunks];
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kPageMaxChunks; ++i) {
        const int e = i * kPageThreads + threadIdx.x;
        if (e >= chunks) continue;
        w[i] = __ldg(reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(rows) +
                                                     (row + e / per) * stride + (size_t)j * a.D + (e % per) * 8));
        if (FP8) {
            float x[8];
            unpack_bf16x8(w[i], x);
#pragma unroll
            for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(x[k]));
        }
    }
    const size_t block = (size_t)phys * a.Hk + j;
    float s = 1.f;
    if (FP8) {
        if (slot == 0) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
            __syncthreads();
            m = 0.f;
            for (int k = 0; k < kPageThreads / 32; ++k) m = fmaxf(m, red[k]);
            s = m > 0.f ? m / 448.f : 1.f;
            if (threadIdx.x == 0) scales[block] = s;
        } else {
            s = scales[block];
        }
    }
#pragma unroll
    for (int i = 0; i < kPageMaxChunks; ++i) {
        const int e = i * kPageThreads + threadIdx.x;
        if (e >= chunks) continue;
        const size_t at = (block * a.P + slot + e / per) * a.D + (e % per) * 8;
        if (!FP8) {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(pages) + at) = w[i];
        } else {
            float x[8];
            unpack_bf16x8(w[i], x);
            uint32_t c[2] = {0u, 0u};
#pragma unroll
            for (int k = 0; k < 8; ++k)
                c[k / 4] |= (uint32_t)__nv_cvt_float_to_fp8(x[k] / s, __NV_SATFINITE, __NV_E4M3) << (8 * (k % 4));
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(pages) + at) = make_uint2(c[0], c[1]);
        }
    }
}

template <bool FP8>
__global__ void __launch_bounds__(kPageThreads) write_page_kernel(const WriteArgs a) {
    __shared__ float red[2][kPageThreads / 32];
    const int j = blockIdx.y, b = blockIdx.z;
    grid_dependency_wait();
    grid_dependents_launch();
    int row0, n, tok0;
    if (!chunk_of(a, b, row0, n, tok0) || n == 0) return;  // uniform for the CTA
    const long long page = (long long)tok0 / a.P + blockIdx.x;
    const long long t0 = blockIdx.x == 0 ? tok0 : page * a.P;
    const long long t1 = min((page + 1) * a.P, (long long)tok0 + n);
    if (t0 >= t1) return;
    const int phys = __ldg(a.page_table + (size_t)b * a.pt_stride + page);
    if (phys < 0 || phys >= a.num_pages) {
        if (threadIdx.x == 0) set_error(a.err, GQA_ERR_BAD_PAGE);
        return;
    }
    const long long row = row0 + (t0 - tok0);
    const int slot = (int)(t0 - page * a.P), ntok = (int)(t1 - t0);
    write_page<FP8>(a, a.k_new, a.k_stride, a.k_pages, a.k_scale, row, ntok, slot, phys, j, red[0]);
    write_page<FP8>(a, a.v_new, a.v_stride, a.v_pages, a.v_scale, row, ntok, slot, phys, j, red[1]);
}

}  // namespace

cudaError_t launch_write_kv(const WriteArgs &a, cudaStream_t stream) {
    if (a.B == 0 || a.total_q == 0 || a.max_q_len == 0) return cudaSuccess;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (a.kv_dtype == GQA_KV_FP4) {
        const long long blocks = ((long long)a.total_q * a.Hk * (a.D / 16) + 255) / 256;
        if (blocks > INT32_MAX) return cudaErrorInvalidValue;
        cfg.gridDim = dim3((unsigned)blocks);
        cfg.blockDim = dim3(256);
        return a.D == 128 ? cudaLaunchKernelEx(&cfg, write_fp4_kernel<128>, a)
                          : cudaLaunchKernelEx(&cfg, write_fp4_kernel<64>, a);
    }
    // pages that max_q_len tokens can touch, wherever they begin
    cfg.gridDim = dim3((unsigned)(((long long)a.max_q_len + a.P - 2) / a.P + 1), a.Hk, a.B);
    cfg.blockDim = dim3(kPageThreads);
    return a.kv_dtype == GQA_KV_FP8_E4M3 ? cudaLaunchKernelEx(&cfg, write_page_kernel<true>, a)
                                         : cudaLaunchKernelEx(&cfg, write_page_kernel<false>, a);
}

}  // namespace gqa
