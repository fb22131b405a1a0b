// decode_fp4.cu -- GQA decode over a paged cache held in 4 bits (fp4.cuh: e2m1 codes, an e4m3
// scale per token, kv head and 16 dims, an fp32 factor per kv head).
//
// All query heads of a group are packed into one unit (PackGQA: "解锁GQA性能潜力：从批量大小敏感性到高
// 效优化实践", section "核心参数调优：PackGQA与NumSplits的协同舞蹈"), so every cached byte crosses HBM
// once; the softmax is the online form ("TensorRT-LLM与TensorRT核心差异解析", section 4.2.1).
//
// Schedule.  The 16-token tiles of all (sequence, kv head [, block of heads]) units are laid end
// to end and cut into equal contiguous shares, one per warp of a fixed grid.  A warp streams its
// share through a private shared-memory ring: the lane that holds a tile's page index issues its
// two bulk copies (a tile's codes and scales are contiguous), the warp waits on the slot's mbarrier,
// takes the tile into registers and hands the slot to the copy of the tile kStages further on.  No
// warp waits for another until the end.  Units cut between the warps of a CTA are then merged
// through shared memory; those cut between CTAs leave one piece per CTA in the workspace, and the
// last CTA to arrive merges them, in the order of the CTAs.
//
// Tile.  S^T = K q^T and O^T += V^T P^T on m16n8k16 f16 tensor-core fragments: tokens (dims) are M,
// 8 packed heads N.  The operands code * scale are exact f16 values; q is bf16 scaled per head by
// a power of two into f16 range (exact but for elements 2^-30 of the head's largest), P is rounded
// to f16 (2^-11 of each weight, or 2^-32 of the largest); sums, the running reference and the running sum are fp32.
#include "fp4.cuh"
#include "quant_kv.h"

namespace gqa {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The softmax reference of a head is its running maximum less kRefBelow (log2 units) and moves only
// when a score passes it by kLazyRef: weights stay below 2^15, inside f16, and the largest is at
// least 2^kRefBelow, so that f16's subnormal step costs a small weight 2^-32 of the largest.
constexpr float kRefBelow = 7.0f, kLazyRef = 15.0f;
constexpr int kMinTilesPerWarp = 4;
constexpr int kRuns = kThreads;   // the sequences' tile prefix is kept per run of ceil(B / kRuns)

template <int NT>
constexpr int ctas_per_sm() { return NT == 1 ? 2 : 1; }

template <int D, int NT>
struct Cfg {
    static constexpr int KS = D / 16;         // k steps of the scores, 16-dim tiles of the output
    static constexpr int C = D / 8;           // dims of a lane's V codes
    static constexpr int kTile = fp4_tile_bytes(D);
    static constexpr int kStages = D == 128 ? 4 : 8;
    static constexpr int HW = 8 * NT;         // packed head columns
    static constexpr int RS = D + 4;          // padded row of a dumped state
    static constexpr int kDump = HW * (RS + 2);  // floats: O rows, then m and l
};

template <int D, int NT>
struct alignas(128) Smem {
    using C = Cfg<D, NT>;
    uint8_t ring[kWarps][C::kStages][2][C::kTile];  // at the end: the state of the unit begun last
    float head[kWarps][C::kDump];                   // the state of a unit begun by an earlier warp
    uint64_t full[kWarps][C::kStages];
    long long pre[kRuns + 1];                       // tiles before each run of sequences
    long long wsum[kWarps];
    int head_unit[kWarps], tail_unit[kWarps];       // unit indices, -1: none
    int empty[kWarps];
    int abort_flag, last[2];
    static_assert(sizeof(float) * C::kDump <= sizeof(ring[0]), "a state fits the warp's ring");
};

__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar,
                                          uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1], %2, [%3], %4;" ::"r"(smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

__device__ __forceinline__ int clamped_len(const Fp4DecodeArgs &a, int b) {
    const int L = __ldg(a.seq_lens + b), most = a.pt_stride * a.P;
    return L < 0 ? 0 : (L > most ? most : L);
}
__device__ __forceinline__ int tiles_of(int L) { return (L + kFp4Tile - 1) / kFp4Tile; }

// A tile's place: sequence, unit within it (kv head * head blocks + block), tile of nt.
struct Pos {
    int b, y, tile, nt;
};

// Step n tiles on (not past the last tile of the batch).
__device__ __forceinline__ void advance(Pos &p, int n, const Fp4DecodeArgs &a, int U) {
    p.tile += n;
    while (p.tile >= p.nt) {
        p.tile -= p.nt;
        if (++p.y < U) continue;
        p.y = 0;
        do {
            if (++p.b >= a.B) {
                p.b = a.B - 1;
                p.tile = 0;
                p.nt = 1;
                return;
            }
            p.nt = tiles_of(clamped_len(a, p.b));
        } while (p.nt == 0);
    }
}

// The place of flat tile f (a whole warp calls it with the same f).
__device__ __forceinline__ Pos locate(long long f, const long long *pre, const Fp4DecodeArgs &a, int U,
                                      int lane) {
    int lo = 0, hi = kRuns - 1;  // first run with U * pre[run + 1] > f
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (U * pre[mid + 1] > f) hi = mid;
        else lo = mid + 1;
    }
    const int per = (a.B + kRuns - 1) / kRuns;
    long long local = f - U * pre[lo];
    int b = lo * per;
    Pos p;
    if (per > 1) {
        for (const int end = min(a.B, b + per); b < end; b += 32) {
            const int nt = b + lane < end ? tiles_of(clamped_len(a, b + lane)) : 0;
            long long incl = nt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long t = __shfl_up_sync(kFull, incl, o);
                if (lane >= o) incl += t;
            }
            const unsigned past = __ballot_sync(kFull, U * incl > local);
            if (past) {
                const int src = __ffs(past) - 1;
                local -= U * __shfl_sync(kFull, incl - nt, src);
                b += src;
                break;
            }
            local -= U * __shfl_sync(kFull, incl, 31);
        }
    }
    p.b = b;
    p.nt = tiles_of(clamped_len(a, b));
    p.y = (int)(local / p.nt);
    p.tile = (int)(local % p.nt);
    return p;
}

// One warp's attention over part of a unit: lane (gq = lane / 4, cq = lane % 4).
template <int D, int NT>
struct State {
    using C = Cfg<D, NT>;
    uint32_t qf[NT][C::KS][2];   // q^T fragments: head 8 nt + gq, dims (D / 4) cq + 4 ks ..
    float kmul[NT][2];           // to log2 units, for heads 8 nt + 2 cq and + 1
    float o[NT][C::KS][4];       // dims gq C + 2 dt (e = 0, 1) and + 1 (e = 2, 3); heads 2 cq + (e & 1)
    float m[NT][2], l[NT][2];

    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int dt = 0; dt < C::KS; ++dt) o[nt][dt][0] = o[nt][dt][1] = o[nt][dt][2] = o[nt][dt][3] = 0.f;
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.f;
        }
    }

    __device__ __forceinline__ void load_q(const __nv_bfloat16 *rows, int nh, float mul, int lane) {
        const int gq = lane >> 2, cq = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int h = nt * 8 + gq;
            const bool ok = h < nh;
            const uint4 *src = reinterpret_cast<const uint4 *>(rows + (size_t)(ok ? h : 0) * D + cq * (D / 4));
            float x[D / 4];
            float big = 0.f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) unpack_bf16x8(ok ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u), x + 8 * i);
#pragma unroll
            for (int i = 0; i < D / 4; ++i) big = fmaxf(big, fabsf(x[i]));
            big = fmaxf(big, __shfl_xor_sync(kFull, big, 1));
            big = fmaxf(big, __shfl_xor_sync(kFull, big, 2));
            // the head's power of two: the largest |q| into [2^14, 2^15)
            int e = 0;
            if (big > 0.f && big < INFINITY) e = 14 - ilogbf(big);
            e = max(-126, min(126, e));
            const float up = __int_as_float((127 + e) << 23), down = __int_as_float((127 - e) << 23);
#pragma unroll
            for (int ks = 0; ks < C::KS; ++ks) {
                qf[nt][ks][0] = pack_f16(x[4 * ks] * up, x[4 * ks + 1] * up);
                qf[nt][ks][1] = pack_f16(x[4 * ks + 2] * up, x[4 * ks + 3] * up);
            }
            kmul[nt][0] = mul * __shfl_sync(kFull, down, 8 * cq);
            kmul[nt][1] = mul * __shfl_sync(kFull, down, 8 * cq + 4);
        }
    }

    // Fold in one tile at kt / vt, its first `valid` tokens.  `release` runs once the tile is in
    // registers.
    template <typename F>
    __device__ __forceinline__ void tile(const uint8_t *kt, const uint8_t *vt, int valid, int lane, F release) {
        constexpr int KS = C::KS, W = D / 32;  // 32-bit words of a lane's codes per token row / pair
        const int gq = lane >> 2, cq = lane & 3;
        uint32_t kr[2][W], vr[2][W], ksc[2], vsc[2];
        const uint8_t *kp = kt + gq * (D / 2) + cq * (D / 8);
        const uint8_t *vp = vt + gq * (4 * C::C) + cq * C::C;
        if constexpr (W == 4) {
            *reinterpret_cast<uint4 *>(kr[0]) = *reinterpret_cast<const uint4 *>(kp);
            *reinterpret_cast<uint4 *>(kr[1]) = *reinterpret_cast<const uint4 *>(kp + 8 * (D / 2));
            *reinterpret_cast<uint4 *>(vr[0]) = *reinterpret_cast<const uint4 *>(vp);
            *reinterpret_cast<uint4 *>(vr[1]) = *reinterpret_cast<const uint4 *>(vp + 4 * D);
        } else {
            *reinterpret_cast<uint2 *>(kr[0]) = *reinterpret_cast<const uint2 *>(kp);
            *reinterpret_cast<uint2 *>(kr[1]) = *reinterpret_cast<const uint2 *>(kp + 8 * (D / 2));
            *reinterpret_cast<uint2 *>(vr[0]) = *reinterpret_cast<const uint2 *>(vp);
            *reinterpret_cast<uint2 *>(vr[1]) = *reinterpret_cast<const uint2 *>(vp + 4 * D);
        }
        // K scales: of the lane's dims, two blocks per row (D = 128) or one
        const uint8_t *ks0 = kt + 8 * D + gq * (D / 16);
        if constexpr (D == 128) {
            ksc[0] = *reinterpret_cast<const uint16_t *>(ks0 + 2 * cq);
            ksc[1] = *reinterpret_cast<const uint16_t *>(ks0 + 8 * (D / 16) + 2 * cq);
        } else {
            ksc[0] = ks0[cq] * 0x0101u;
            ksc[1] = ks0[8 * (D / 16) + cq] * 0x0101u;
        }
        // V scales: of block (gq C) / 16, tokens 2 cq and + 1, and 8 further
        const uint8_t *vs0 = vt + 8 * D + cq * (D / 8) + (gq * C::C / 16) * 2;
        vsc[0] = *reinterpret_cast<const uint16_t *>(vs0);
        vsc[1] = *reinterpret_cast<const uint16_t *>(vs0 + 4 * (D / 8));
        __syncwarp();
        release();

        // ---- scores; even and odd k steps in two chains
        float s[NT][4], s2[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][e] = s2[nt][e] = 0.f;
        uint32_t ka = e4m3x2_to_f16(ksc[0]), kb = e4m3x2_to_f16(ksc[1]);
        const uint32_t sa[2] = {__byte_perm(ka, ka, 0x1010), __byte_perm(ka, ka, 0x3232)};
        const uint32_t sb[2] = {__byte_perm(kb, kb, 0x1010), __byte_perm(kb, kb, 0x3232)};
#pragma unroll
        for (int i = 0; i < W; ++i) {
            uint32_t ha[4], hb[4];
            e2m1x8_to_f16(kr[0][i], ha);
            e2m1x8_to_f16(kr[1][i], hb);
            const int blk = i / 2;  // 16 dims
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t af[4] = {hmul2(ha[2 * k], sa[blk]), hmul2(hb[2 * k], sb[blk]),
                                        hmul2(ha[2 * k + 1], sa[blk]), hmul2(hb[2 * k + 1], sb[blk])};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16(k ? s2[nt] : s[nt], af, qf[nt][2 * i + k][0], qf[nt][2 * i + k][1]);
            }
        }

        // ---- online softmax in log2 units; only the tiles that move the reference m take the
        // column maxima and a rescale
        float x[NT][4];
        bool need = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) x[nt][e] = (s[nt][e] + s2[nt][e]) * kmul[nt][e & 1];
            if (valid < kFp4Tile) {
                if (gq >= valid) x[nt][0] = x[nt][1] = -INFINITY;
                if (gq + 8 >= valid) x[nt][2] = x[nt][3] = -INFINITY;
            }
            need |= fmaxf(x[nt][0], x[nt][2]) > m[nt][0] + kLazyRef;
            need |= fmaxf(x[nt][1], x[nt][3]) > m[nt][1] + kLazyRef;
        }
        if (valid < kFp4Tile) {  // what follows the sequence may be anything: its scales become 0
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (2 * cq + 8 * i >= valid) vsc[i] = 0u;
                if (2 * cq + 8 * i + 1 >= valid) vsc[i] &= 0xffu;
            }
        }
        if (__any_sync(kFull, need)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float alpha[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    float mx = fmaxf(x[nt][e], x[nt][e + 2]);
                    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
                    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
                    mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
                    mx = fmaxf(mx - kRefBelow, m[nt][e]);
                    alpha[e] = mx == -INFINITY ? 1.f : ex2_approx(m[nt][e] - mx);
                    m[nt][e] = mx;
                    l[nt][e] *= alpha[e];
                }
#pragma unroll
                for (int dt = 0; dt < KS; ++dt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[nt][dt][e] *= alpha[e & 1];
            }
        }
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float ref = m[nt][e & 1] == -INFINITY ? 0.f : m[nt][e & 1];
                p[e] = ex2_approx(x[nt][e] - ref);
            }
            l[nt][0] += p[0] + p[2];
            l[nt][1] += p[1] + p[3];
            pb[nt][0] = movmatrix_trans(pack_f16(p[0], p[1]));
            pb[nt][1] = movmatrix_trans(pack_f16(p[2], p[3]));
        }

        // ---- O^T += V^T P^T
        const uint32_t va = e4m3x2_to_f16(vsc[0]), vb = e4m3x2_to_f16(vsc[1]);
#pragma unroll
        for (int i = 0; i < W; ++i) {
            uint32_t ha[4], hb[4];
            e2m1x8_to_f16(vr[0][i], ha);
            e2m1x8_to_f16(vr[1][i], hb);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t af[4] = {hmul2(ha[2 * k], va), hmul2(ha[2 * k + 1], va), hmul2(hb[2 * k], vb),
                                        hmul2(hb[2 * k + 1], vb)};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma_f16(o[nt][2 * i + k], af, pb[nt][0], pb[nt][1]);
            }
        }
    }

    // Sum l over the lanes that share a head column.
    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float v = l[nt][e];
                v += __shfl_xor_sync(kFull, v, 4);
                v += __shfl_xor_sync(kFull, v, 8);
                v += __shfl_xor_sync(kFull, v, 16);
                l[nt][e] = v;
            }
    }

    __device__ __forceinline__ void dump(float *dst, int lane) const {
        const int gq = lane >> 2, cq = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int h = nt * 8 + 2 * cq + e;
                float4 *row = reinterpret_cast<float4 *>(dst + h * C::RS + gq * C::C);
#pragma unroll
                for (int i = 0; i < C::C / 4; ++i)
                    row[i] = make_float4(o[nt][2 * i][e], o[nt][2 * i][e + 2], o[nt][2 * i + 1][e], o[nt][2 * i + 1][e + 2]);
                if (gq == 0) {
                    dst[C::HW * C::RS + h] = m[nt][e];
                    dst[C::HW * C::RS + C::HW + h] = l[nt][e];
                }
            }
    }
};

__device__ __forceinline__ void store4(void *out, int f32, size_t idx, float4 v) {
    if (f32) {
        reinterpret_cast<float4 *>(out)[idx / 4] = v;
    } else {
        reinterpret_cast<uint2 *>(out)[idx / 4] = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
    }
}

// The output of a finished unit from its merged state: O / l times the values' factor.
__device__ __forceinline__ float4 normalised(float4 o, float l, float vf) {
    const float r = l == 0.f ? 0.f : vf / l;
    return make_float4(o.x * r, o.y * r, o.z * r, o.w * r);
}

__device__ __forceinline__ void add4(float4 &acc, float w, const float4 &o) {
    acc.x += w * o.x;
    acc.y += w * o.y;
    acc.z += w * o.z;
    acc.w += w * o.w;
}

// Weight of a state with reference m in a merge with reference M.
__device__ __forceinline__ float weight(float m, float M) { return m == -INFINITY ? 0.f : ex2_approx(m - M); }

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, ctas_per_sm<NT>())
    decode_fp4_kernel(const Fp4DecodeArgs a, const int hpc, const int blocks) {
    using CF = Cfg<D, NT>;
    constexpr int S = CF::kStages;
    extern __shared__ uint8_t smem_raw[];
    Smem<D, NT> &sm = *reinterpret_cast<Smem<D, NT> *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = a.Hq / a.Hk, U = a.Hk * blocks;

    if (lane < S) mbar_init(&sm.full[warp][lane], 1);
    if (threadIdx.x == 0) sm.abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    // launched with programmatic stream serialization: everything above may overlap the previous
    // kernel of the stream, nothing below reads or writes before that kernel is complete
    grid_dependency_wait();
    grid_dependents_launch();

    // ---- tiles before each run of sequences
    {
        const int per = (a.B + kRuns - 1) / kRuns;
        const int b0 = min(a.B, (int)threadIdx.x * per), b1 = min(a.B, b0 + per);
        long long sum = 0;
        for (int b = b0; b < b1; ++b) {
            const int L = __ldg(a.seq_lens + b);
            if (L < 0 || L > a.pt_stride * a.P) {
                if (blockIdx.x == 0) set_error(a.err, GQA_ERR_BAD_PAGE);
            }
            sum += tiles_of(clamped_len(a, b));
        }
        long long incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long t = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += t;
        }
        if (lane == 31) sm.wsum[warp] = incl;
        __syncthreads();
        for (int w = 0; w < warp; ++w) incl += sm.wsum[w];
        sm.pre[threadIdx.x + 1] = incl;
        if (threadIdx.x == 0) sm.pre[0] = 0;
        __syncthreads();
    }
    const long long T = (long long)U * sm.pre[kRuns];

    // sequences without tokens: zeros and -inf
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        if (clamped_len(a, b) != 0) continue;
        for (int e = threadIdx.x; e < a.Hq * D / 4; e += kThreads)
            store4(a.out, a.out_f32, (size_t)b * a.Hq * D + 4 * e, make_float4(0.f, 0.f, 0.f, 0.f));
        if (a.lse)
            for (int e = threadIdx.x; e < a.Hq; e += kThreads) a.lse[(size_t)b * a.Hq + e] = -INFINITY;
    }
    const long long NC = max(1LL, min((long long)gridDim.x, T / (kWarps * kMinTilesPerWarp)));  // CTAs with work
    if (T == 0 || blockIdx.x >= NC) return;

    // ---- this warp's share [s_w, s_w + n)
    const long long s_w = ((long long)blockIdx.x * kWarps + warp) * T / (NC * kWarps);
    const long long n = ((long long)blockIdx.x * kWarps + warp + 1) * T / (NC * kWarps) - s_w;
    int head_unit = -1, tail_unit = -1;
    bool fail = false;
    if (n > 0) {
        const uint64_t policy = policy_evict_first();
        const int tpp = a.P / kFp4Tile;  // tiles of a page: 1, 2 or 4
        Pos p = locate(s_w, sm.pre, a, U, lane);

        // window of 32 tiles: lane i holds the pool tile of the share's tile 32 w + i (-1: bad page)
        Pos wp = p;
        advance(wp, lane, a, U);
        auto resolve = [&](long long r) {
            if (r >= n) return -1;
            const int phys = __ldg(a.page_table + (size_t)wp.b * a.pt_stride + wp.tile / tpp);
            if (phys < 0 || phys >= a.num_pages) return -1;
            return (phys * a.Hk + wp.y / blocks) * tpp + wp.tile % tpp;
        };
        auto issue = [&](int idx, int slot) {  // one lane
            uint64_t *bar = &sm.full[warp][slot];
            if (idx < 0) {
                set_error(a.err, GQA_ERR_BAD_PAGE);
                mbar_arrive(bar);  // the tile computes on stale data
                return;
            }
            mbar_arrive_expect_tx(bar, 2 * CF::kTile);
            bulk_load(sm.ring[warp][slot][0], a.k_pages + (size_t)idx * CF::kTile, CF::kTile, bar, policy);
            bulk_load(sm.ring[warp][slot][1], a.v_pages + (size_t)idx * CF::kTile, CF::kTile, bar, policy);
        };
        int win = resolve(lane), next_win = -1;
        if (lane < S && lane < n) issue(win, lane);
        if (n > 32) {
            advance(wp, 32, a, U);
            next_win = resolve(32 + lane);
        }

        State<D, NT> st;
        bool fresh = true, began = p.tile == 0;
        int L = 0;
        int slot = 0;
        uint32_t parity = 0;
        long long r = 0;
        for (; r < n; ++r) {
            const int kvh = p.y / blocks, blk = p.y % blocks;
            const size_t row0 = (size_t)p.b * a.Hq + kvh * g + blk * hpc;
            const int nh = min(hpc, g - blk * hpc);
            if (fresh) {
                st.reset();
                L = clamped_len(a, p.b);
                st.load_q(static_cast<const __nv_bfloat16 *>(a.q) + row0 * D, nh,
                          a.scale * kLog2e * (a.k_scale ? __ldg(a.k_scale + kvh) : 1.f), lane);
                fresh = false;
            }
            const bool ok = mbar_wait(&sm.full[warp][slot], parity);
            if (__any_sync(kFull, !ok)) {
                fail = true;
                break;
            }
            st.tile(sm.ring[warp][slot][0], sm.ring[warp][slot][1], L - p.tile * kFp4Tile, lane, [&] {
                const long long ri = r + S;
                if (ri >= n) return;
                if ((ri & 31) == 0) {
                    win = next_win;
                    if (ri + 32 < n) {
                        advance(wp, 32, a, U);
                        next_win = resolve(ri + 32 + lane);
                    }
                }
                if (lane == (int)(ri & 31)) issue(win, slot);
            });
            if (++slot == S) {
                slot = 0;
                parity ^= 1u;
            }
            const bool ended = p.tile == p.nt - 1;
            if (ended || r == n - 1) {
                st.finish();
                const int unit = p.b * U + p.y;
                if (began && ended) {
                    const float vf = a.v_scale ? __ldg(a.v_scale + kvh) : 1.f;
                    const int gq = lane >> 2, cq = lane & 3;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int h = nt * 8 + 2 * cq + e;
                            if (h >= nh) continue;
#pragma unroll
                            for (int i = 0; i < CF::C / 4; ++i)
                                store4(a.out, a.out_f32, (row0 + h) * D + gq * CF::C + 4 * i,
                                       normalised(make_float4(st.o[nt][2 * i][e], st.o[nt][2 * i][e + 2],
                                                              st.o[nt][2 * i + 1][e], st.o[nt][2 * i + 1][e + 2]),
                                                  st.l[nt][e], vf));
                            if (gq == 0 && a.lse) a.lse[row0 + h] = (st.m[nt][e] + log2f(st.l[nt][e])) * kLn2;
                        }
                } else if (!began) {
                    st.dump(sm.head[warp], lane);
                    head_unit = unit;
                } else {
                    // the share ends inside the unit; the ring is free: every copy has been waited for
                    st.dump(reinterpret_cast<float *>(sm.ring[warp]), lane);
                    tail_unit = unit;
                }
                fresh = began = true;
            }
            if (r < n - 1) advance(p, 1, a, U);
        }
        if (fail) {
            // give up: no copy may outlive the CTA
            if (lane == 0) {
                set_error(a.err, GQA_ERR_TIMEOUT);
                sm.abort_flag = 1;
            }
            for (long long k = r; k < n && k < r + S; ++k) {
                mbar_wait(&sm.full[warp][slot], parity);
                if (++slot == S) {
                    slot = 0;
                    parity ^= 1u;
                }
            }
        }
    }
    if (lane == 0) {
        sm.head_unit[warp] = head_unit;
        sm.tail_unit[warp] = tail_unit;
        sm.empty[warp] = n == 0;
    }
    __syncthreads();
    if (sm.abort_flag) return;

    // ---- units cut between warps.  Task w: the unit that warp w began and did not end; task -1: the
    // unit that an earlier CTA began.  Its states lie in warp order; each thread owns 4 dims of a head.
    constexpr int V4 = D / 4;
    const long long c_start = blockIdx.x * T / NC, c_end = (blockIdx.x + 1) * T / NC;
    const int slot_floats = hpc * (D + 2);
    int open[2] = {-1, -1};  // units that continue in other CTAs: begun before / in this one
    for (int w = -1; w < kWarps; ++w) {
        int unit;
        if (w < 0) {
            int f = 0;
            while (sm.empty[f]) ++f;  // some warp of a CTA with work has tiles
            unit = sm.head_unit[f];
        } else {
            unit = sm.tail_unit[w];
        }
        if (unit < 0) continue;
        int w1 = w;  // last warp with a state of the unit
        for (int k = w + 1; k < kWarps; ++k) {
            if (sm.empty[k]) continue;
            if (sm.head_unit[k] != unit) break;
            w1 = k;
        }
        const int b = unit / U, y = unit % U;
        const int kvh = y / blocks, blk = y % blocks, nh = min(hpc, g - blk * hpc);
        const size_t row0 = (size_t)b * a.Hq + kvh * g + blk * hpc;
        // where the unit ends: known to the warp that ended it
        const int per = (a.B + kRuns - 1) / kRuns;
        long long us = sm.pre[b / per];
        for (int k = b / per * per; k < b; ++k) us += tiles_of(clamped_len(a, k));
        const int nt_b = tiles_of(clamped_len(a, b));
        us = us * U + (long long)y * nt_b;
        const bool whole = us >= c_start && us + nt_b <= c_end;
        const int side = us >= c_start ? 1 : 0;
        float *piece = a.pieces + ((size_t)blockIdx.x * 2 + side) * slot_floats;
        const float vf = a.v_scale ? __ldg(a.v_scale + kvh) : 1.f;
        for (int e = threadIdx.x; e < nh * V4; e += kThreads) {
            const int h = e / V4, d = (e % V4) * 4;
            float M = -INFINITY, Ls = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k = w < 0 ? 0 : w; k <= w1; ++k) {
                if (sm.empty[k]) continue;
                const float *s = k == w ? reinterpret_cast<const float *>(sm.ring[k]) : sm.head[k];
                M = fmaxf(M, s[CF::HW * CF::RS + h]);
            }
            for (int k = w < 0 ? 0 : w; k <= w1; ++k) {
                if (sm.empty[k]) continue;
                const float *s = k == w ? reinterpret_cast<const float *>(sm.ring[k]) : sm.head[k];
                const float f = weight(s[CF::HW * CF::RS + h], M);
                Ls += f * s[CF::HW * CF::RS + CF::HW + h];
                add4(acc, f, *reinterpret_cast<const float4 *>(s + h * CF::RS + d));
            }
            if (whole) {
                store4(a.out, a.out_f32, (row0 + h) * D + d, normalised(acc, Ls, vf));
                if (d == 0 && a.lse) a.lse[row0 + h] = (M + log2f(Ls)) * kLn2;
            } else {
                float2 *dst = reinterpret_cast<float2 *>(piece + h * D + d);
                dst[0] = make_float2(acc.x, acc.y);
                dst[1] = make_float2(acc.z, acc.w);
                if (d == 0) {
                    piece[hpc * D + h] = M;
                    piece[hpc * D + hpc + h] = Ls;
                }
            }
        }
        if (!whole) open[side] = unit;
    }
    if (open[0] < 0 && open[1] < 0) return;

    // ---- units cut between CTAs: the last to arrive merges the pieces
    __threadfence();
    __syncthreads();
    if (threadIdx.x < 2) {
        const int side = threadIdx.x;
        int last = 0;
        if (open[side] >= 0) {
            const int unit = open[side], b = unit / U, y = unit % U;
            const int per = (a.B + kRuns - 1) / kRuns;
            long long us = sm.pre[b / per];
            for (int k = b / per * per; k < b; ++k) us += tiles_of(clamped_len(a, k));
            const int nt_b = tiles_of(clamped_len(a, b));
            us = us * U + (long long)y * nt_b;
            const int c0 = (int)(((us + 1) * NC + T - 1) / T - 1), c1 = (int)(((us + nt_b) * NC + T - 1) / T - 1);
            if (atomicAdd(a.counters + unit, 1) == c1 - c0) {
                a.counters[unit] = 0;  // ready for the next launch
                last = c1 - c0 + 1;
                sm.head_unit[side] = c0;
            }
        }
        sm.last[side] = last;
    }
    __syncthreads();
    for (int side = 0; side < 2; ++side) {
        const int np = sm.last[side];
        if (np == 0) continue;
        __threadfence();
        const int unit = open[side], b = unit / U, y = unit % U;
        const int kvh = y / blocks, blk = y % blocks, nh = min(hpc, g - blk * hpc);
        const size_t row0 = (size_t)b * a.Hq + kvh * g + blk * hpc;
        const float vf = a.v_scale ? __ldg(a.v_scale + kvh) : 1.f;
        const int c0 = sm.head_unit[side];
        // the unit begins in its first CTA (side 1) and runs on in the others (side 0)
        auto piece = [&](int k) { return a.pieces + ((size_t)(c0 + k) * 2 + (k == 0 ? 1 : 0)) * slot_floats; };
        for (int e = threadIdx.x; e < nh * V4; e += kThreads) {
            const int h = e / V4, d = (e % V4) * 4;
            float M = -INFINITY, Ls = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
            for (int k = 0; k < np; ++k) M = fmaxf(M, __ldcg(piece(k) + hpc * D + h));
#pragma unroll 4
            for (int k = 0; k < np; ++k) {
                const float *s = piece(k);
                const float f = weight(__ldcg(s + hpc * D + h), M);
                Ls += f * __ldcg(s + hpc * D + hpc + h);
                const float2 lo = __ldcg(reinterpret_cast<const float2 *>(s + h * D + d));
                const float2 hi = __ldcg(reinterpret_cast<const float2 *>(s + h * D + d) + 1);
                add4(acc, f, make_float4(lo.x, lo.y, hi.x, hi.y));
            }
            store4(a.out, a.out_f32, (row0 + h) * D + d, normalised(acc, Ls, vf));
            if (d == 0 && a.lse) a.lse[row0 + h] = (M + log2f(Ls)) * kLn2;
        }
    }
}

template <int D, int NT>
cudaError_t launch_t(const Fp4DecodeArgs &a, cudaStream_t stream) {
    const int g = a.Hq / a.Hk;
    const int hpc = a.pack_gqa ? (g < 8 * NT ? g : 8 * NT) : 1;
    const size_t smem = sizeof(Smem<D, NT>) + 128;
    auto kern = decode_fp4_kernel<D, NT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.sms * ctas_per_sm<NT>());
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a, hpc, (g + hpc - 1) / hpc);
}

}  // namespace

// Two pieces per CTA of the largest grid, each a state of up to 16 heads.
size_t fp4_decode_piece_bytes(int Hq, int Hk, int D) {
    const int g = Hq / Hk, hpc = g < 16 ? g : 16;
    return (size_t)kStreamMaxSms * 2 * 2 * hpc * (D + 2) * sizeof(float);
}

cudaError_t launch_decode_fp4(const Fp4DecodeArgs &a, cudaStream_t stream) {
    const bool wide = a.pack_gqa && a.Hq / a.Hk > 8;
    if (a.D == 128) return wide ? launch_t<128, 2>(a, stream) : launch_t<128, 1>(a, stream);
    return wide ? launch_t<64, 2>(a, stream) : launch_t<64, 1>(a, stream);
}

}  // namespace gqa
