// fp4.cuh -- the 4-bit cache's element format and page layout, shared by the kernels that
// write it (write_kv.cu), read it back (read_kv.cu) and attend to it (decode_fp4.cu).
//
// A value is code * scale * factor: an e2m1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign), an
// e4m3 scale per (token, kv head, 16 dims), an fp32 factor per kv head.  Every code * scale is
// an f16 value exactly (at most 2 + 4 significant bits, between 2^-10 and 2688), so the
// tensor-core kernels multiply exact operands.
//
// Layout.  A (page, kv head) block is P / 16 tiles; a tile holds 16 tokens in 9 D contiguous
// bytes: 8 D code bytes, then D scale bytes.  The order inside a tile is the one the m16n8k16
// fragments want, so that a warp fetches a tile's codes with two 16-byte shared-memory loads
// per lane, no bank conflict and no transpose:
//   K (tokens are M, dims are the contraction): codes [16 tokens][D / 2], a byte holds dims
//     2i and 2i + 1; lane (gq, cq) reads D / 4 dims of rows gq and gq + 8.  Scales
//     [16 tokens][D / 16].
//   V (dims are M, tokens are the contraction): a byte holds one dim of tokens 2i and 2i + 1.
//     With C = D / 8, pair i and dim d sit at (i / 4) 4D + (d / C) 4C + (i % 4) C + d % C;
//     lane (gq, cq) reads dims gq C .. gq C + C - 1 of pairs cq and cq + 4.  Scales
//     [8 pairs][D / 16][2 tokens].
// The even dim (K) or token (V) of a byte is in its low nibble.
#pragma once

#include <stdint.h>

#include "gqa_device.cuh"

namespace gqa {

constexpr int kFp4Tile = 16;  // tokens of a tile

__host__ __device__ constexpr int fp4_tile_bytes(int D) { return 9 * D; }

// Two codes of a byte (low nibble first) -> f16x2, exact.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(w));
}

// Two e4m3 bytes (low byte first) -> f16x2, exact (0x7f and 0xff are NaN).
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
    uint32_t h;
    const uint16_t s = (uint16_t)two;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(s));
    return h;
}

__device__ __forceinline__ float e4m3_to_f32(uint32_t byte) {
    const uint32_t h = e4m3x2_to_f16(byte & 0xffu);
    return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}

// Nearest e4m3 code (ties to even, saturating at 448; NaN stays NaN).
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
    return r & 0xffu;
}

__device__ __forceinline__ uint32_t f32_to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four pairs of fp32 values -> four bytes of e2m1 codes (nearest, ties to even, saturating at
// 6), lo[i] in the low nibble of byte i.
__device__ __forceinline__ uint32_t f32_to_e2m1x8(const float (&lo)[4], const float (&hi)[4]) {
    uint32_t w;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %5, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %6, %2;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %7, %3;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %4;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(w)
        : "f"(lo[0]), "f"(lo[1]), "f"(lo[2]), "f"(lo[3]), "f"(hi[0]), "f"(hi[1]), "f"(hi[2]), "f"(hi[3]));
    return w;
}

__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

__device__ __forceinline__ void unpack_bf16x8(const uint4 &w, float *x) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

// x / s for many bf16 values x over one s, rounded to fp32 as a division is, in 3 operations instead of
// its dozen and its slow path: with r = RN(1 / s) and q = RN(x r), RN(q - (q s - x) r).
//   That this is RN(x / s) was checked by going through all pairs of significands, 2^23 of s and 128 of x
// (the remainder q s - x is exact in all but 0.13% of them); powers of two change none of it while the
// steps neither overflow nor lose bits below the normal range.
// fits(): that they do not for |x| <= m, as far as |x / s| >= 2^-10, half the smallest positive code of
// either kind: the bits of the remainder are then multiples of 2^-116.  What is lost of a smaller quotient
// leaves it a code of 0 with the sign of x.  If it does not fit, the caller divides.
struct Quotient {
    float s, minus_r;
    __device__ __forceinline__ explicit Quotient(float s_) : s(s_), minus_r(-1.f / s_) {}
    __device__ __forceinline__ bool fits(float m) const { return s >= 0x1p-60f && s <= 0x1p60f && m < 0x1p20f * s; }
    __device__ __forceinline__ float operator()(float x) const {
        const float q = x * -minus_r;
        return fmaf(fmaf(q, s, -x), minus_r, q);  // (a zero keeps its sign)
    }
};
static __device__ __noinline__ float divide(float x, float s) { return x / s; }

// 32 bytes: one 256-bit store where the address allows it, which `wide` says.
__device__ __forceinline__ void store32(void *dst, const uint32_t (&w)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        uint4 *d = static_cast<uint4 *>(dst);
        d[0] = make_uint4(w[0], w[1], w[2], w[3]);
        d[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// Index of the sequence whose run of rows holds row r: the last b with cu[b] <= r, in
// [0, B - 1] whatever cu holds.
template <typename T>
__device__ __forceinline__ int sequence_of(const T *cu, int B, long long r) {
    int lo = 0, hi = B - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((long long)cu[mid] <= r) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The first rows and lengths of a batch: a copy in shared memory for up to kMax sequences, so that a
// row's search costs one trip to memory and not one per level; the caller's arrays beyond.
template <typename T>
struct Sequences {
    static constexpr int kMax = 256;
    T cu_s[kMax + 1];
    int len_s[kMax];
    const T *cu;
    const int32_t *lens;

    // By all threads of the CTA; a barrier has to follow.
    __device__ __forceinline__ void load(const T *cu_g, const int32_t *lens_g, int B) {
        const bool here = B <= kMax;
        if (threadIdx.x == 0) {
            cu = here ? cu_s : cu_g;
            lens = here ? len_s : lens_g;
        }
        if (!here) return;
        for (int b = threadIdx.x; b <= B; b += blockDim.x) {
            if (cu_g) cu_s[b] = __ldg(cu_g + b);
            if (b < B) len_s[b] = __ldg(lens_g + b);
        }
    }
};

}  // namespace gqa
