// write_kv.cu -- writes the newest tokens of every sequence into the paged cache: a prefill
// chunk's, or a decode step's one token ("TensorRT对Grouped Query Attention的支持进展", sections
// "动态形状与KV Cache管理" and "与动态批处理协同"), quantised on the way for 4-bit and e4m3 pools.
// Bound by HBM (16 bits in, 4 to 16 out) and, as it stands, by the look-ups before a CTA's first
// load: 4096 tokens into 4-bit pages 7.4 us (21 MB), 15421 ragged ones into 4-bit pages 21 us
// (3.8 TB/s), into e4m3 pages 24 us (3.9 TB/s).  The grid runs over the rows of the input, so that no CTA
// is idle however ragged the chunks are; a thread per row first finds where the row goes.
//
// 4-bit pools (write_fp4_kernel).  A block of 16 dims of one token, with g the head's factor:
//   a = max |x|,  sf = e4m3(min(fl(a / fl(6 g)), 448)),  s = fl(sf g),  code = e2m1(fl(x / s))
// (fl: fp32 rounding).  The quotients are rounded as a division's: a reciprocal alone would move
// values off the exact ties that bf16 inputs hit.  A block whose scale rounds to 0 stores zeros, one
// that holds a NaN stores a NaN scale (it reads back as NaN), infinities saturate.  A V byte holds
// two tokens, so a thread takes the blocks of a pair of tokens, of keys or of values (a chunk may
// begin or end inside a pair; half-written bytes keep their other nibble).
//
// e4m3 and bf16 pools (write_page_kernel).  Work is (page of a chunk, kv head, K or V): a team of a
// warp per 16 slots holds its tokens in registers, so the input is read once.  A page whose first
// slot is in the chunk takes its scale from the chunk's tokens in it, absmax / 448 (1 when they are
// all zero); a page that was begun earlier keeps its scale.  A chunk of one token is
// gqa_paged_append_kv()'s rule.
#include "fp4.cuh"
#include "quant_kv.h"

namespace gqa {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRows = 128;  // input rows of a CTA

// A row of the input: its sequence's first row, number of rows and first token, and the row's own
// token; `page` < 0: not written (the error word says so unless the row is of no sequence).
struct Row {
    int row0, n, t, page;
};

__device__ __forceinline__ Row find_row(const WriteArgs &a, const Sequences<int32_t> &seqs, long long r) {
    Row x = {0, 0, 0, -1};
    if (r >= a.total_q) return x;
    const int b = a.cu_q ? sequence_of(seqs.cu, a.B, r) : (int)r, L = seqs.lens[b];
    if (a.cu_q) {
        x.row0 = seqs.cu[b];
        x.n = seqs.cu[b + 1] - x.row0;
    } else {
        x.row0 = b;
        x.n = L > 0 ? 1 : 0;
    }
    const int tok0 = L - x.n;
    if (x.n < 0 || x.n > a.max_q_len || x.row0 < 0 || (long long)x.row0 + x.n > a.total_q || tok0 < 0 ||
        L > a.pt_stride * a.P) {
        set_error(a.err, GQA_ERR_BAD_PAGE);
        return x;
    }
    if (r < x.row0 || r >= x.row0 + x.n) return x;
    x.t = tok0 + (int)(r - x.row0);
    const int phys = __ldg(a.page_table + (size_t)b * a.pt_stride + x.t / a.P);
    if (phys < 0 || phys >= a.num_pages) set_error(a.err, GQA_ERR_BAD_PAGE);
    else x.page = phys;
    return x;
}

// Sequences none of whose rows are looked at (negative counts, rows past total_q) and that do not
// fit are recorded here, each by one thread of the grid's x.
__device__ __forceinline__ void check_sequences(const WriteArgs &a) {
    if (!a.cu_q) return;
    for (long long b = (long long)blockIdx.x * kThreads + threadIdx.x; b < a.B; b += (long long)gridDim.x * kThreads) {
        const int L = __ldg(a.seq_lens + b), row0 = __ldg(a.cu_q + b), n = __ldg(a.cu_q + b + 1) - row0;
        if (n < 0 || n > a.max_q_len || row0 < 0 || (long long)row0 + n > a.total_q || n > L || L > a.pt_stride * a.P)
            set_error(a.err, GQA_ERR_BAD_PAGE);
    }
}

__device__ __forceinline__ void load_block(const void *rows, long long stride, long long r, int at, float (&x)[16]) {
    const uint4 *p = reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(rows) + r * stride + at);
    const uint4 lo = __ldg(p), hi = __ldg(p + 1);
    unpack_bf16x8(lo, x);
    unpack_bf16x8(hi, x + 8);
}

// Scale code of a block of 16 and its values over the scale; zeros where the scale is 0 or NaN.
// `over6` divides by 6 g.
__device__ __forceinline__ uint32_t quantise_block(float (&x)[16], float g, const Quotient &over6) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) a = max_nan(a, fabsf(x[i]));
    const uint32_t sf = f32_to_e4m3(over6.fits(a) ? over6(a) : divide(a, over6.s));
    const Quotient over(e4m3_to_f32(sf) * g);
    if (over.fits(a)) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = over(x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = over.s > 0.f ? divide(x[i], over.s) : 0.f;
    }
    return sf;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 4) write_fp4_kernel(const WriteArgs a, const int rows) {
    constexpr int G = D / 16, C = D / 8;
    struct Pair {
        int row, place, kind;  // first row, its pool row of head 0; 0: both tokens, 1: the even one, 2: the odd one
    };
    __shared__ Sequences<int32_t> seqs;
    __shared__ Pair list[kMaxRows];
    __shared__ int pairs;
    const long long r0 = (long long)blockIdx.x * rows;
    if (threadIdx.x == 0) pairs = 0;
    grid_dependency_wait();
    grid_dependents_launch();
    seqs.load(a.cu_q, a.seq_lens, a.B);
    __syncthreads();
    if (threadIdx.x < rows) {
        const long long r = r0 + threadIdx.x;
        const Row x = find_row(a, seqs, r);
        // a pair is its even token's, or the odd one's when that is the chunk's first
        if (x.page >= 0) {
            const bool odd = x.t & 1, both = !odd && r + 1 < x.row0 + x.n;
            if (!odd || r == x.row0)
                list[atomicAdd(&pairs, 1)] = {(int)r, x.page * a.Hk * a.P + x.t % a.P, both ? 0 : odd ? 2 : 1};
        }
    }
    __syncthreads();

    // ---- the threads run over blocks, then pairs, then heads, then K and V
    const int np = pairs, units = np * G * a.Hk;
#pragma unroll 1
    for (int u = threadIdx.x; u < 2 * units; u += kThreads) {
        const bool is_v = u >= units;
        const int i = (is_v ? u - units : u) / G, c = u % G, j = i / np;
        const Pair e = list[i - j * np];
        const int q = e.place + j * a.P, tok = q % kFp4Tile;
        const void *src = is_v ? a.v_new : a.k_new;
        const long long stride = is_v ? a.v_stride : a.k_stride;
        const float *factor = is_v ? a.v_scale : a.k_scale;
        float x[16], y[16];
        load_block(src, stride, e.row, j * D + c * 16, x);
        load_block(src, stride, e.row + (e.kind == 0), j * D + c * 16, y);
        const float g = factor ? __ldg(factor + j) : 1.f;
        const Quotient over6(6.f * g);
        const uint32_t s0 = quantise_block(x, g, over6), s1 = quantise_block(y, g, over6);
        uint8_t *tile = static_cast<uint8_t *>(is_v ? a.v_pages : a.k_pages) + (size_t)(q / kFp4Tile) * fp4_tile_bytes(D);
        if (!is_v) {
            uint8_t *codes = tile + tok * (D / 2) + c * 8, *sc = tile + 8 * D + tok * G + c;
            const float l0[4] = {x[0], x[2], x[4], x[6]}, h0[4] = {x[1], x[3], x[5], x[7]};
            const float l1[4] = {x[8], x[10], x[12], x[14]}, h1[4] = {x[9], x[11], x[13], x[15]};
            *reinterpret_cast<uint2 *>(codes) = make_uint2(f32_to_e2m1x8(l0, h0), f32_to_e2m1x8(l1, h1));
            *sc = (uint8_t)s0;
            if (e.kind != 0) continue;
            const float m0[4] = {y[0], y[2], y[4], y[6]}, n0[4] = {y[1], y[3], y[5], y[7]};
            const float m1[4] = {y[8], y[10], y[12], y[14]}, n1[4] = {y[9], y[11], y[13], y[15]};
            *reinterpret_cast<uint2 *>(codes + D / 2) = make_uint2(f32_to_e2m1x8(m0, n0), f32_to_e2m1x8(m1, n1));
            sc[G] = (uint8_t)s1;
            continue;
        }
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float l[4] = {x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]};
            const float h[4] = {y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]};
            w[k] = f32_to_e2m1x8(l, h);  // alone, a token is in both nibbles
        }
        const int pair = tok / 2;
        uint8_t *sc = tile + 8 * D + pair * (2 * G) + c * 2;
        uint8_t *codes = tile + (pair >> 2) * (4 * D) + (pair & 3) * C;
        if (e.kind == 0) {
            *reinterpret_cast<uint16_t *>(sc) = (uint16_t)(s0 | (s1 << 8));
        } else {
            sc[e.kind == 2] = (uint8_t)s0;
            const uint32_t keep = e.kind == 2 ? 0x0f0f0f0fu : 0xf0f0f0f0u;  // the other token's
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int d = c * 16 + 4 * k;
                const uint32_t old = *reinterpret_cast<const uint32_t *>(codes + (d / C) * (4 * C) + d % C);
                w[k] = (old & keep) | (w[k] & ~keep);
            }
        }
        if constexpr (C == 16) {
            *reinterpret_cast<uint4 *>(codes + c * (4 * C)) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            *reinterpret_cast<uint2 *>(codes + (2 * c) * (4 * C)) = make_uint2(w[0], w[1]);
            *reinterpret_cast<uint2 *>(codes + (2 * c + 1) * (4 * C)) = make_uint2(w[2], w[3]);
        }
    }
    check_sequences(a);
}

// A lane's `count` eights of a page by division: read again, out of the way of the others.
__device__ __noinline__ void divide_eights(const uint16_t *src, long long src_step, uint8_t *dst, int dst_step, int count, float s) {
#pragma unroll 1
    for (int i = 0; i < 8 * count; ++i) {
        const float x = __uint_as_float((uint32_t)src[(i >> 3) * src_step + (i & 7)] << 16);
        dst[(i >> 3) * dst_step + (i & 7)] = (uint8_t)f32_to_e4m3(x / s);
    }
}

// One CTA per (run of `rows` input rows, kv head): the pages whose first row of the chunk is in the
// run, K and V of each.  TEAM warps hold a page's 16 TEAM slots.
template <bool FP8, int D, int TEAM>
__global__ void __launch_bounds__(kThreads, 4) write_page_kernel(const WriteArgs a, const int rows) {
    constexpr int P = 16 * TEAM, kPer = D / 8, kAt = 32 / kPer, kIts = 16 / kAt;  // rows of a warp at once
    struct Page {
        int row, ntok, slot, phys;
    };
    __shared__ Sequences<int32_t> seqs;
    __shared__ Page list[64];
    __shared__ int pages;
    __shared__ float red[kWarps];
    const long long r0 = (long long)blockIdx.x * rows;
    const int j = blockIdx.y;
    if (threadIdx.x == 0) pages = 0;
    grid_dependency_wait();
    grid_dependents_launch();
    // the run's lines set out for L2 while its pages are looked up
    for (int i = threadIdx.x; i < rows * (D / 64) * 2; i += kThreads) {
        const long long r = r0 + i / (D / 64 * 2);
        if (r < a.total_q)
            prefetch_l2(static_cast<const uint16_t *>(i & 1 ? a.v_new : a.k_new) + r * (i & 1 ? a.v_stride : a.k_stride) + j * D +
                        (i >> 1) % (D / 64) * 64);
    }
    seqs.load(a.cu_q, a.seq_lens, a.B);
    __syncthreads();
    if (threadIdx.x < rows) {
        const long long r = r0 + threadIdx.x;
        const Row x = find_row(a, seqs, r);
        if (x.page >= 0 && (x.t % P == 0 || r == x.row0)) {
            const int left = (int)(x.row0 + x.n - r);
            list[atomicAdd(&pages, 1)] = {(int)r, min(P - x.t % P, left), x.t % P, x.page};
        }
    }
    __syncthreads();

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, team = warp / TEAM, part = warp % TEAM;
#pragma unroll 1
    for (int task = team; task < 2 * pages; task += kWarps / TEAM) {
        const Page pg = list[task >> 1];
        const bool is_v = task & 1;
        const uint16_t *src = static_cast<const uint16_t *>(is_v ? a.v_new : a.k_new) + (size_t)j * D + (lane % kPer) * 8;
        const long long stride = is_v ? a.v_stride : a.k_stride;
        const int t0 = part * 16 + lane / kPer;  // this lane's first token of the page's
        uint4 w[kIts];
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < kIts; ++i)
            w[i] = t0 + i * kAt < pg.ntok ? __ldg(reinterpret_cast<const uint4 *>(src + (pg.row + t0 + i * kAt) * stride))
                                          : make_uint4(0u, 0u, 0u, 0u);
        const size_t block = (size_t)pg.phys * a.Hk + j;
        float s = 1.f;
        if (FP8) {
            float *scales = is_v ? a.v_scale : a.k_scale;
            // magnitudes order as integers, two at once; a NaN, which the scale takes no notice of, is
            // above infinity
            uint32_t big = 0;
#pragma unroll
            for (int i = 0; i < kIts; ++i) {
                const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) big = __vmaxu2(big, u[k] & 0x7fff7fffu);
            }
            big = max(big >> 16, big & 0xffffu);
            m = __uint_as_float(big << 16);
            if (big > 0x7f80u) {
                m = 0.f;
#pragma unroll
                for (int i = 0; i < kIts; ++i) {
                    float x[8];
                    unpack_bf16x8(w[i], x);
#pragma unroll
                    for (int k = 0; k < 8; ++k) m = fmaxf(m, fabsf(x[k]));
                }
            }
            if (pg.slot == 0) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                if (TEAM > 1) {
                    if (lane == 0) red[warp] = m;
                    asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * TEAM) : "memory");
#pragma unroll
                    for (int k = 0; k < TEAM; ++k) m = fmaxf(m, red[team * TEAM + k]);
                    // (the next page of the team is written after all have read this one's)
                    asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * TEAM) : "memory");
                }
                s = m > 0.f ? m / 448.f : 1.f;
                if (part == 0 && lane == 0) scales[block] = s;
            } else {
                s = scales[block];
            }
        }
        const size_t at = (block * P + pg.slot + t0) * D + (lane % kPer) * 8;
        void *dst = is_v ? a.v_pages : a.k_pages;
        if (!FP8) {
#pragma unroll
            for (int i = 0; i < kIts; ++i)
                if (t0 + i * kAt < pg.ntok) *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(dst) + at + i * kAt * D) = w[i];
            continue;
        }
        const Quotient over(s);
        if (!over.fits(m)) {
            const int count = min(kIts, (pg.ntok - t0 + kAt - 1) / kAt);
            divide_eights(src + (pg.row + t0) * stride, kAt * stride, static_cast<uint8_t *>(dst) + at, kAt * D, count, s);
            continue;
        }
#pragma unroll
        for (int i = 0; i < kIts; ++i) {
            if (t0 + i * kAt >= pg.ntok) continue;
            float x[8];
            unpack_bf16x8(w[i], x);
            uint32_t c[2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
                c[k] = f32_to_e4m3x2(over(x[4 * k]), over(x[4 * k + 1])) |
                       f32_to_e4m3x2(over(x[4 * k + 2]), over(x[4 * k + 3])) << 16;
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(dst) + at + i * kAt * D) = make_uint2(c[0], c[1]);
        }
    }
    if (j == 0) check_sequences(a);
}

template <bool FP8, int D>
void (*page_kernel(int P))(const WriteArgs, int) {
    return P == 16 ? write_page_kernel<FP8, D, 1> : P == 32 ? write_page_kernel<FP8, D, 2> : write_page_kernel<FP8, D, 4>;
}

}  // namespace

cudaError_t launch_write_kv(const WriteArgs &a, cudaStream_t stream) {
    if (a.B == 0 || a.total_q == 0 || a.max_q_len == 0) return cudaSuccess;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void (*k)(const WriteArgs, int);
    int rows;
    if (a.kv_dtype == GQA_KV_FP4) {
        // as few rows as give every thread a block, more once that fills the GPU several times
        rows = 2;
        while (rows < kMaxRows && rows * a.Hk * (a.D / 16) < kThreads) rows *= 2;
        while (rows < 32 && a.total_q / rows > 592) rows *= 2;
        cfg.gridDim = dim3((unsigned)(((long long)a.total_q + rows - 1) / rows));
        k = a.D == 128 ? write_fp4_kernel<128> : write_fp4_kernel<64>;
    } else {
        // chunks of some length: a page or a few per CTA; single tokens are a page each, which a CTA
        // takes 8 / TEAM at a time
        rows = a.total_q >= 16LL * a.B ? 64 : 8;
        cfg.gridDim = dim3((unsigned)(((long long)a.total_q + rows - 1) / rows), a.Hk);
        if (a.kv_dtype == GQA_KV_FP8_E4M3) k = a.D == 128 ? page_kernel<true, 128>(a.P) : page_kernel<true, 64>(a.P);
        else k = a.D == 128 ? page_kernel<false, 128>(a.P) : page_kernel<false, 64>(a.P);
    }
    return cudaLaunchKernelEx(&cfg, k, a, rows);
}

}  // namespace gqa
