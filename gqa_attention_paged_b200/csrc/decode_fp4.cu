// decode_fp4.cu -- GQA decode over a paged cache held in 4 bits (fp4.cuh: e2m1 codes, an e4m3
// scale per token, kv head and 16 dims, an fp32 factor per kv head).
//
// All query heads of a group are packed into one unit (PackGQA: "解锁GQA性能潜力：从批量大小敏感性到高
// 效优化实践", section "核心参数调优：PackGQA与NumSplits的协同舞蹈"), so every cached byte crosses HBM
// once; the softmax is the online form ("TensorRT-LLM与TensorRT核心差异解析", section 4.2.1).
//
// Schedule.  The 32-token steps of all (sequence, kv head [, block of heads]) units are laid end
// to end and cut into equal contiguous shares, one per warp of a fixed grid; units that are few and
// short have a CTA each instead.  Going on to a unit (its q, the last one's results) takes as long as
// a step, so with several steps a warp a unit counts one place more than its steps; without that,
// warps with many short units came last (64 sequences of 0 .. 4096 tokens: 43.0 us, 38.5 with it).
// A warp streams its share through a private shared-memory ring of 16-byte asynchronous copies (a
// tile's codes and scales are contiguous; a bulk copy per tile, 1152 bytes, was bound by the copies
// an SM can start, about one in 32 cycles): the step is taken into registers and its slot handed to
// the step kStages further on.  No warp waits for another until the end.  Units cut between the warps
// of a CTA are then merged through shared memory; those cut between CTAs leave one piece per CTA in
// the workspace, and the last CTA to arrive merges them, in the order of the CTAs.
//
// Tile.  S^T = K q^T and O^T += V^T P^T on m16n8k16 f16 tensor-core fragments: tokens (dims) are M,
// 8 packed heads N.  The operands code * scale are exact f16 values; q is bf16 scaled per head by
// a power of two into f16 range (exact but for elements 2^-30 of the head's largest), P is rounded
// to f16 (2^-11 of each weight, or 2^-32 of the largest); sums, the running reference and the
// running sum are fp32.  Groups above 8 run as blocks of 8 heads, whose second read of a tile is an
// L2 hit (groups of 16, 48 x 0 .. 3000 tokens: 26.8 us; one block of 16 heads took 5 more).
//
// What bounds it.  At 64 x 2048 tokens and 8 kv heads a step of 32 tokens comes to 645 instructions a
// warp with all that is around it, 128 conversions and 128 scale multiplications among them.  Issue is
// active 56% of the time and no pipe above 46%: it is the latency of a step's chain at 15 warps an SM.
// 37 us there, of which 3 go before the first keys and 4 into the merges; 1 x 2048: 10.2 us; 256 x 2048:
// 112 us (607 MB, 5.4 TB/s; copies alone 98), 129 once the power cap holds the clock.
#include <atomic>

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
constexpr int kCtasPerSm = 2;
constexpr int kHeads = 8;  // packed heads of a unit at most: the columns of a product
constexpr float kNoRef = -3e38f;  // below every reference
constexpr int kStep = 2 * kFp4Tile;  // tokens of a step: two tiles
// Steps a warp from which on a unit counts one place more than its steps.  Ragged lengths, us without
// and with: 13 steps a warp 34.3 and 28.8, 7.1 30.5 and 26.9, 4.2 19.8 and 20.3, 2.0 14.9 and 15.3;
// uniform ones 1 to 3% slower with it (64 x 2048: 36.9 and 37.1, 256 x 2048: 109 and 112).
constexpr int kWeighted = 5;
// Steps of the longest unit up to which, when there are no more units than CTAs, each has a CTA of its
// own and nothing is merged between CTAs (us, without and with: 8 units of 7 steps 9.5 and 5.8, of 22
// 10.6 and 8.0, of 32 9.4 and 9.3, of 47 11.3 and 11.9; 288 units of 32 steps 17.7 and 14.2).
constexpr int kWhole = 32;
constexpr int kRuns = kThreads;      // the sequences' step prefix is kept per run of ceil(B / kRuns)
constexpr int kMaxCtas = kStreamMaxSms * kCtasPerSm;
constexpr int kPieceLine = 32;       // floats: a piece begins on a line of 128 bytes

__host__ __device__ constexpr int piece_floats(int heads, int D) {
    return (heads * (D + 2) + kPieceLine - 1) / kPieceLine * kPieceLine;
}

// The count of a unit's CTAs that have left their pieces.  It lies in the workspace's header, behind the
// error word, where no call of the library keeps scratch, so that a zeroed workspace serves calls of any
// kind in turn.  That is room for 5 bits a CTA, six fields a word.  A unit from CTA c0 to c1 counts in
// c0's field, which is its alone because no other such unit begins in c0; if 5 bits are too few, the unit
// covers the 11 CTAs behind c0, in whose fields no other unit counts, and with them the next whole word.
struct Arrivals {
    static constexpr int kBits = 5, kFields = 32 / kBits;
    static constexpr int kWords = (kMaxCtas - 1) / kFields + 2;
    int word, shift;
    unsigned mask;
    __device__ __forceinline__ Arrivals(int c0, int c1) {
        const bool small = c1 - c0 + 1 < 1 << kBits;
        word = c0 / kFields + (small ? 0 : 1);
        shift = small ? c0 % kFields * kBits : 0;
        mask = small ? (1u << kBits) - 1 : ~0u;
    }
};
static_assert(sizeof(int) * (1 + Arrivals::kWords) <= kWorkspaceHeader, "the counts fit the header");
static_assert((1 << Arrivals::kBits) > 2 * Arrivals::kFields, "a unit that needs a word covers one");

template <int D>
struct Cfg {
    static constexpr int KS = D / 16;         // k steps of the scores, 16-dim tiles of the output
    static constexpr int C = D / 8;           // dims of a lane's V codes
    static constexpr int kTile = fp4_tile_bytes(D);
    static constexpr int kStages = D == 128 ? 2 : 4;
    static constexpr int RS = D + 4;          // padded row of a dumped state
    static constexpr int kDump = kHeads * (RS + 2);  // floats: O rows, then m and l
};

// The unit that a dumped state belongs to (-1: no state): the place of its first step, its steps, kv
// head, first row of q and heads.
struct Cut {
    int unit, first, steps, kvh, row0, n;
};

template <int D>
struct alignas(128) Smem {
    using C = Cfg<D>;
    uint8_t ring[kWarps][C::kStages][4][C::kTile];  // K, K, V, V; at the end: the state of the unit begun last
    float head[kWarps][C::kDump];                   // the state of a unit begun by an earlier warp
    int pre[kRuns + 1];                             // steps before each run of sequences
    int len[kRuns];                                 // tokens, when a run is one sequence
    int wsum[kWarps];
    Cut cut[2][kWarps];                             // of head and ring
    int empty[kWarps];
    int last[2];  // pieces to merge, of the unit begun earlier and of the one begun here
    static_assert(sizeof(float) * C::kDump <= sizeof(ring[0]), "a state fits the warp's ring");
};

// 16 bytes into shared memory, or zeros when `bytes` is 0.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t *src, uint32_t bytes, uint64_t policy) {
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src), "r"(bytes),
                 "l"(policy)
                 : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Not volatile, so that the compiler may move them (64 x 2048: 39.4 -> 38.7 us).
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

template <int W>
__device__ __forceinline__ void load_words(uint32_t (&r)[W], const uint8_t *p) {
    if constexpr (W == 4) *reinterpret_cast<uint4 *>(r) = *reinterpret_cast<const uint4 *>(p);
    else *reinterpret_cast<uint2 *>(r) = *reinterpret_cast<const uint2 *>(p);
}

__device__ __forceinline__ int clamped(const Fp4DecodeArgs &a, int L) {
    const int most = a.pt_stride * a.P;
    return L < 0 ? 0 : (L > most ? most : L);
}
__device__ __forceinline__ int clamped_len(const Fp4DecodeArgs &a, int b) { return clamped(a, __ldg(a.seq_lens + b)); }
__device__ __forceinline__ int steps_of(int L) { return (int)(((unsigned)L + kStep - 1) / kStep); }

__device__ __forceinline__ bool weighted(int total) { return total >= kWeighted * kWarps * (int)gridDim.x; }

// The batch as every warp sees it: units of a sequence, sequences of a run, and in shared memory
// the steps before each run (times U: flat indices) and the lengths.  A unit has `more` (0 or 1)
// places beyond its steps; for want of a second prefix the units of an empty sequence have them too.
// The host keeps all of these within an int.
struct Batch {
    const Fp4DecodeArgs &a;
    const int *pre, *lens;
    int U, per, more;
    __device__ __forceinline__ int len(int b) const { return per == 1 ? lens[b] : clamped_len(a, b); }
    __device__ __forceinline__ int steps(int b) const { return steps_of(len(b)); }
    __device__ __forceinline__ int place(int run) const { return U * (pre[run] + more * min(run * per, a.B)); }
};

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kFull, x, o));
    return x;
}
// A step's place: sequence, unit within it (kv head * head blocks + block), step of the unit's nt.
struct Pos {
    int b, y, step, nt;
};

// n steps on (not past the last step of the batch).
__device__ __forceinline__ void advance(Pos &p, int n, const Batch &bt) {
    p.step += n;
    if (p.step < p.nt) return;
    unsigned flat = (unsigned)p.y * p.nt + p.step;
    while (flat >= (unsigned)bt.U * p.nt) {
        flat -= (unsigned)bt.U * p.nt;
        do {
            if (++p.b >= bt.a.B) {
                p = {bt.a.B - 1, 0, 0, 1};
                return;
            }
            p.nt = bt.steps(p.b);
        } while (p.nt == 0);
    }
    p.y = flat / p.nt;
    p.step = flat - p.y * p.nt;
}

// The step at place f or, where that is a unit's extra place, the next one (a whole warp calls it with
// the same f).  `index`: the step's flat index, the number of steps if there is none.
__device__ __forceinline__ Pos locate(int f, const Batch &bt, int lane, int &index) {
    // the first run that ends behind f, by its eighth and then its place there
    static_assert(kRuns == 256, "32 lanes of 8 runs");
    int run = (__ffs(__ballot_sync(kFull, bt.place(8 * lane + 8) > f)) - 1) * 8;
    run += __ffs(__ballot_sync(kFull, bt.place(run + (lane & 7) + 1) > f)) - 1;
    unsigned local = f - bt.place(run);
    int b = run * bt.per, before = bt.pre[run];
    if (bt.per > 1) {
        for (const int end = min(bt.a.B, b + bt.per); b < end; b += 32) {
            const int places = b + lane < end ? bt.steps(b + lane) + bt.more : 0;
            int incl = places;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int t = __shfl_up_sync(kFull, incl, o);
                if (lane >= o) incl += t;
            }
            const unsigned past = __ballot_sync(kFull, (unsigned)(bt.U * incl) > local);
            const int src = past ? __ffs(past) - 1 : 32;
            const int skipped = __shfl_sync(kFull, past ? incl - places : incl, src & 31);
            const int all = past ? skipped : __shfl_sync(kFull, incl, 31);
            local -= bt.U * all;
            before += all - bt.more * src;
            if (past) {
                b += src;
                break;
            }
        }
    }
    Pos p = {b, 0, 0, bt.steps(b)};
    if (p.nt == 0) {  // of an empty sequence
#pragma unroll 1
        do
            if (++p.b >= bt.a.B) {
                index = bt.U * bt.pre[kRuns];
                return {bt.a.B - 1, 0, 0, 1};
            }
        while ((p.nt = bt.steps(p.b)) == 0);
    } else {
        p.y = local / (p.nt + bt.more);
        p.step = max((int)(local - p.y * (p.nt + bt.more)) - bt.more, 0);
    }
    index = bt.U * before + p.y * p.nt + p.step;
    return p;
}

// The place of the first step of p's unit.
__device__ __forceinline__ int first_place(const Batch &bt, const Pos &p, int more) {
    const int run = bt.per == 1 ? p.b : p.b / bt.per;
    int before = bt.pre[run];
    if (bt.per > 1)
#pragma unroll 1
        for (int b = run * bt.per; b < p.b; ++b) before += bt.steps(b);
    return bt.U * (before + more * p.b) + p.y * (p.nt + more) + more;
}

// The batch's places in equal shares, the first `rem` of them one longer.
struct Shares {
    int q, rem;
    __device__ __forceinline__ int start(int w) const { return w * q + min(w, rem); }
    __device__ __forceinline__ int owner(int f) const {
        const int big = rem * (q + 1);
        return f < big ? f / (q + 1) : rem + (f - big) / q;
    }
};

// The query heads of unit y of sequence b: kv head, first row of q, heads.
struct Heads {
    int kvh, row0, n;
    __device__ __forceinline__ Heads(const Fp4DecodeArgs &a, int blocks, int hpc, int b, int y) {
        const int g = a.Hq / a.Hk;
        kvh = blocks == 1 ? y : y / blocks;
        const int h0 = (y - kvh * blocks) * hpc;
        n = min(hpc, g - h0);
        row0 = b * a.Hq + kvh * g + h0;
    }
};

// One warp's attention over part of a unit: lane (gq = lane / 4, cq = lane % 4).
template <int D>
struct State {
    using C = Cfg<D>;
    static constexpr int W = D / 32;  // 32-bit words of a lane's codes per token row / pair
    uint32_t qf[C::KS][2];            // q^T fragments: head gq, dims (D / 4) cq + 4 ks ..
    float kmul[2];                    // to log2 units, for heads 2 cq and + 1
    float o[C::KS][4];                // dims gq C + 2 dt (e = 0, 1) and + 1 (e = 2, 3); heads 2 cq + (e & 1)
    float m[2], l[2];
    float s[2][4];                    // a step's scores per tile: products, then exponents
    uint32_t vr[4][W], vs[4];         // its values and their scales: pairs of tile h in 2 h and 2 h + 1

    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int dt = 0; dt < C::KS; ++dt) o[dt][0] = o[dt][1] = o[dt][2] = o[dt][3] = 0.f;
        m[0] = m[1] = l[0] = l[1] = 0.f;
    }

    // q in two parts: the loads, and what becomes of them.  `rows`: the unit's n heads; the columns
    // past them are zero and never looked at.
    struct Query {
        uint32_t w[D / 8];
        float mul;
    };
    static __device__ __forceinline__ Query fetch_q(const Fp4DecodeArgs &a, const Heads &hd, int lane) {
        const int gq = lane >> 2, cq = lane & 3;
        const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(a.q) +
                                                           (size_t)(hd.row0 + (gq < hd.n ? gq : 0)) * D + cq * (D / 4));
        Query x;
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            *reinterpret_cast<uint4 *>(x.w + 4 * i) = gq < hd.n ? __ldg(src + i) : make_uint4(0u, 0u, 0u, 0u);
        x.mul = a.scale * kLog2e * (a.k_scale ? __ldg(a.k_scale + hd.kvh) : 1.f);
        return x;
    }

    __device__ __forceinline__ void set_q(const Query &x, int lane) {
        const int cq = lane & 3;
        const uint32_t(&w)[D / 8] = x.w;
        uint32_t big = 0;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) big = __vmaxu2(big, w[i] & 0x7fff7fffu);
        big = __vmaxu2(big, __shfl_xor_sync(kFull, big, 1));
        big = __vmaxu2(big, __shfl_xor_sync(kFull, big, 2));
        // the head's power of two: the largest |q| into [2^14, 2^15) (none for infinities and NaN)
        const int ex = max(big >> 16, big & 0xffffu) >> 7, e = ex == 255 ? 0 : min(141 - ex, 126);
        const float up = __int_as_float((127 + e) << 23), down = __int_as_float((127 - e) << 23);
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            qf[i / 2][i & 1] = pack_f16(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xffff0000u) * up);
        kmul[0] = x.mul * __shfl_sync(kFull, down, 8 * cq);
        kmul[1] = x.mul * __shfl_sync(kFull, down, 8 * cq + 4);
    }

    // The products q k of a step's two tiles; its values into registers.
    __device__ __forceinline__ void scores(const uint8_t *slot, int lane) {
        const int gq = lane >> 2, cq = lane & 3;
        const uint8_t *kp = slot + gq * (D / 2) + cq * (D / 8);
        const uint8_t *ksp = slot + 8 * D + gq * (D / 16) + (D == 128 ? 2 * cq : cq);
        const uint8_t *vp = slot + 2 * C::kTile + gq * (4 * C::C) + cq * C::C;
        const uint8_t *vsp = slot + 2 * C::kTile + 8 * D + cq * (D / 8) + (gq * C::C / 16) * 2;
        uint32_t kr[4][W], sc[4][2];  // rows of tile h in 2 h and 2 h + 1; their scales, twice each
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const int at = (h >> 1) * C::kTile;
            load_words(kr[h], kp + at + (h & 1) * (8 * D / 2));
            const uint8_t *two = ksp + at + (h & 1) * (8 * D / 16);
            const uint32_t x = e4m3x2_to_f16(D == 128 ? *reinterpret_cast<const uint16_t *>(two) : *two * 0x0101u);
            sc[h][0] = __byte_perm(x, x, 0x1010);
            sc[h][1] = __byte_perm(x, x, 0x3232);
        }
        // a chain of products per tile
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int blk = i / 2;  // 16 dims
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t ha[4], hb[4];
                e2m1x8_to_f16(kr[2 * h][i], ha);
                e2m1x8_to_f16(kr[2 * h + 1][i], hb);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t af[4] = {hmul2(ha[2 * k], sc[2 * h][blk]), hmul2(hb[2 * k], sc[2 * h + 1][blk]),
                                            hmul2(ha[2 * k + 1], sc[2 * h][blk]), hmul2(hb[2 * k + 1], sc[2 * h + 1][blk])};
                    if (i + k == 0) mma_first(s[h], af, qf[0][0], qf[0][1]);
                    else mma(s[h], af, qf[2 * i + k][0], qf[2 * i + k][1]);
                }
            }
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const int at = (h >> 1) * C::kTile;
            load_words(vr[h], vp + at + (h & 1) * (4 * D));
            vs[h] = *reinterpret_cast<const uint16_t *>(vsp + at + (h & 1) * (4 * D / 8));
        }
    }

    // Fold the step in, `valid` tokens of it; `fresh`: the first since reset().
    __device__ __forceinline__ void fold(int valid, bool fresh, int lane) {
        const int gq = lane >> 2, cq = lane & 3;
        // ---- online softmax in log2 units, scores less the reference; only the steps that move the
        // reference take the column maxima and a rescale
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[h][e] = fmaf(s[h][e], kmul[e & 1], -m[e & 1]);
        if (valid < kStep) {  // what follows the sequence may be anything: its scores and scales go
            __syncwarp();     // (keeps this a branch: 113 -> 109.5 us at batch 256, before a unit had an extra place)
#pragma unroll
            for (int h = 0; h < 4; ++h) {
                if (2 * cq + 8 * h >= valid) vs[h] = 0u;
                if (2 * cq + 8 * h + 1 >= valid) vs[h] &= 0xffu;
                if (gq + 8 * h >= valid) s[h >> 1][2 * (h & 1)] = s[h >> 1][2 * (h & 1) + 1] = -INFINITY;
            }
        }
        float top = -INFINITY;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, s[h][e]);
        if (__any_sync(kFull, top > kLazyRef || fresh)) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = fmaxf(fmaxf(s[0][e], s[0][e + 2]), fmaxf(s[1][e], s[1][e + 2]));
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
                // 0 where the head's reference stays; it may begin anywhere
                const float up = fresh ? mx - kRefBelow : fmaxf(mx - kRefBelow, 0.f);
                const float alpha = fresh ? 1.f : ex2_approx(-up);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    s[h][e] -= up;
                    s[h][e + 2] -= up;
                }
                m[e] += up;
                l[e] *= alpha;
#pragma unroll
                for (int dt = 0; dt < C::KS; ++dt) {
                    o[dt][e] *= alpha;
                    o[dt][e + 2] *= alpha;
                }
            }
        }
        uint32_t pb[2][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = ex2_approx(s[h][e]);
            l[0] += p[0] + p[2];
            l[1] += p[1] + p[3];
            pb[h][0] = transpose8x8(pack_f16(p[0], p[1]));
            pb[h][1] = transpose8x8(pack_f16(p[2], p[3]));
        }

        // ---- O^T += V^T P^T
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t va = e4m3x2_to_f16(vs[2 * h]), vb = e4m3x2_to_f16(vs[2 * h + 1]);
#pragma unroll
            for (int i = 0; i < W; ++i) {
                uint32_t ha[4], hb[4];
                e2m1x8_to_f16(vr[2 * h][i], ha);
                e2m1x8_to_f16(vr[2 * h + 1][i], hb);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const uint32_t af[4] = {hmul2(ha[2 * k], va), hmul2(ha[2 * k + 1], va), hmul2(hb[2 * k], vb),
                                            hmul2(hb[2 * k + 1], vb)};
                    mma(o[2 * i + k], af, pb[h][0], pb[h][1]);
                }
            }
        }
    }

    // Sum l over the lanes that share a head column.
    __device__ __forceinline__ void finish() {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(kFull, l[e], 4);
            l[e] += __shfl_xor_sync(kFull, l[e], 8);
            l[e] += __shfl_xor_sync(kFull, l[e], 16);
        }
    }

    __device__ __forceinline__ void dump(float *dst, int lane) const {
        const int gq = lane >> 2, cq = lane & 3;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int h = 2 * cq + e;
            float4 *row = reinterpret_cast<float4 *>(dst + h * C::RS + gq * C::C);
#pragma unroll
            for (int i = 0; i < C::C / 4; ++i)
                row[i] = make_float4(o[2 * i][e], o[2 * i][e + 2], o[2 * i + 1][e], o[2 * i + 1][e + 2]);
            if (gq == 0) {
                dst[kHeads * C::RS + h] = m[e];
                dst[kHeads * C::RS + kHeads + h] = l[e];
            }
        }
    }
};

// V consecutive dims of a row at index `idx`, times r.
template <bool F32, int V>
__device__ __forceinline__ void store_dims(void *out, size_t idx, const float (&x)[V], float r) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
        if (F32) reinterpret_cast<float2 *>(out)[(idx + i) / 2] = make_float2(x[i] * r, x[i + 1] * r);
        else reinterpret_cast<uint32_t *>(out)[(idx + i) / 2] = pack_bf16(x[i] * r, x[i + 1] * r);
    }
}

template <int D, bool F32>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    decode_fp4_kernel(const Fp4DecodeArgs a, const int hpc, const int blocks) {
    using CF = Cfg<D>;
    constexpr int S = CF::kStages, V = D / 32;
    extern __shared__ uint8_t smem_raw[];
    Smem<D> &sm = *reinterpret_cast<Smem<D> *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int U = a.Hk * blocks;
    Batch bt = {a, sm.pre, sm.len, U, a.B <= kRuns ? 1 : (a.B + kRuns - 1) / kRuns, 0};

    // launched with programmatic stream serialization: nothing below reads or writes before the
    // previous kernel of the stream is complete
    grid_dependency_wait();
    grid_dependents_launch();

    // ---- steps before each run of sequences
    int none = 0;  // a sequence without tokens?
    bool whole = bt.per == 1 && a.B * U <= (int)gridDim.x;  // few short units, a CTA each?
    {
        const int b0 = min(a.B, (int)threadIdx.x * bt.per), b1 = min(a.B, b0 + bt.per);
        int incl = 0, longest = 0;
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            const int L0 = __ldg(a.seq_lens + b), L = clamped(a, L0);
            if (L != L0 && blockIdx.x == 0) set_error(a.err, GQA_ERR_BAD_PAGE);
            if (bt.per == 1) sm.len[b] = L;
            incl += steps_of(L);
            longest = steps_of(L);
            none |= L == 0;
        }
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int t = __shfl_up_sync(kFull, incl, o);
            if (lane >= o) incl += t;
        }
        if (lane == 31) sm.wsum[warp] = incl;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) incl += w < warp ? sm.wsum[w] : 0;
        sm.pre[threadIdx.x + 1] = incl;
        if (threadIdx.x == 0) sm.pre[0] = 0;
        none = __syncthreads_or(none);
        if (whole) whole = !__syncthreads_or(longest > kWhole);
    }
    const int total = U * sm.pre[kRuns];
    bt.more = weighted(total);
    const int T = total + bt.more * U * a.B;

    if (none) {  // zeros and -inf
        const float zero[4] = {};
#pragma unroll 1
        for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
            if (bt.len(b) != 0) continue;
#pragma unroll 1
            for (int e = threadIdx.x; e < a.Hq * D / 4; e += kThreads) {
                store_dims<F32>(a.out, (size_t)b * a.Hq * D + 4 * e, zero, 0.f);
                if (a.lse && e % (D / 4) == 0) a.lse[(size_t)b * a.Hq + e / (D / 4)] = -INFINITY;
            }
        }
    }
    // ---- this warp's share: n steps from p on
    Shares sh = {0, 0};
    Pos p = {a.B - 1, 0, 0, 1};
    int n;
    if (whole) {
        // a CTA per unit
        if (blockIdx.x >= a.B * U) return;
        const int b = blockIdx.x / U, nt = bt.steps(b);
        if (nt == 0) return;
        const int from = nt * warp / kWarps;
        n = nt * (warp + 1) / kWarps - from;
        p = {b, (int)blockIdx.x - b * U, from, nt};
    } else {
        const int NC = max(1, min((int)gridDim.x, T / kWarps));  // CTAs with work
        if (T == 0 || blockIdx.x >= NC) return;
        // (below the whole grid NC is T / kWarps: a step each, and one more for some)
        sh.q = NC == (int)gridDim.x ? (int)((unsigned)T / (gridDim.x * kWarps)) : (T >= kWarps ? 1 : 0);
        sh.rem = T - sh.q * (NC * kWarps);
        const int s_w = sh.start(blockIdx.x * kWarps + warp), e_w = sh.start(blockIdx.x * kWarps + warp + 1);
        int index = 0;
        n = e_w - s_w;
        if (n > 0) p = locate(s_w, bt, lane, index);
        if (bt.more) {
            int end = total;
            if (e_w < T) locate(e_w, bt, lane, end);
            n = end - index;
        }
    }
    if (lane < 2) sm.cut[lane][warp].unit = -1;
    if (lane == 0) sm.empty[warp] = n == 0;
    __syncwarp();
    if (n > 0) {
        const uint64_t policy = policy_evict_first();
        const int tshift = a.P == 16 ? 0 : (a.P == 32 ? 1 : 2);  // tiles of a page: 1, 2 or 4
        // window of 32 steps: lane i holds the place and the pool tiles of the share's step 32 w + i
        // (-1: none)
        Pos wp = p;
        int2 win = make_int2(-1, -1);

        const uint32_t ring = smem_u32(sm.ring[warp][0][0]) + lane * 16;
        auto ask = [&](int i) {  // step i of the share; a group of copies for every i
            if (i < n) {
                if ((i & 31) == 0) {
                    advance(wp, i == 0 ? lane : 32, bt);
                    win = make_int2(-1, -1);
                    if (i + lane < n) {
                        const int32_t *row = a.page_table + (size_t)wp.b * a.pt_stride;
                        const int t0 = 2 * wp.step, c0 = t0 >> tshift, c1 = (t0 + 1) >> tshift;
                        const bool two = t0 + 1 < (bt.len(wp.b) + kFp4Tile - 1) / kFp4Tile;
                        const int p0 = __ldg(row + c0), p1 = c1 == c0 || !two ? p0 : __ldg(row + c1);
                        const int kvh = blocks == 1 ? wp.y : wp.y / blocks;
                        if (p0 >= 0 && p0 < a.num_pages) win.x = ((p0 * a.Hk + kvh) << tshift) + (t0 & ((1 << tshift) - 1));
                        if (two && p1 >= 0 && p1 < a.num_pages)
                            win.y = ((p1 * a.Hk + kvh) << tshift) + ((t0 + 1) & ((1 << tshift) - 1));
                        // a bad page reads as zeros
                        if (win.x < 0 || (two && win.y < 0)) set_error(a.err, GQA_ERR_BAD_PAGE);
                    }
                }
                const uint32_t slot = ring + (i & (S - 1)) * (4 * CF::kTile);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int t = __shfl_sync(kFull, h ? win.y : win.x, i & 31);
                    const size_t at = (size_t)max(t, 0) * CF::kTile + lane * 16;
                    const uint32_t bytes = t < 0 ? 0 : 16;
#pragma unroll
                    for (int c = 0; c < CF::kTile; c += 512) {
                        if (c + 512 > CF::kTile && lane * 16 >= CF::kTile - c) continue;
                        copy16(slot + h * CF::kTile + c, a.k_pages + at + c, bytes, policy);
                        copy16(slot + (2 + h) * CF::kTile + c, a.v_pages + at + c, bytes, policy);
                    }
                }
            }
            copies_commit();
        };
        // the first q sets out before the first keys, and is looked at between the first asks
        State<D> st;
        const auto q0 = State<D>::fetch_q(a, Heads(a, blocks, hpc, p.b, p.y), lane);
        ask(0);
        st.set_q(q0, lane);
#pragma unroll 1
        for (int i = 1; i < S; ++i) ask(i);
        Heads hd(a, blocks, hpc, 0, 0);
        bool fresh = true, began = p.step == 0;
        int valid = 0;
#pragma unroll 1
        for (int r = 0; r < n; ++r) {
            if (fresh) {
                hd = Heads(a, blocks, hpc, p.b, p.y);
                valid = bt.len(p.b) - p.step * kStep;
                st.reset();
                if (r > 0) st.set_q(State<D>::fetch_q(a, hd, lane), lane);
            }
            copies_wait<S - 1>();
            __syncwarp();
            st.scores(sm.ring[warp][r & (S - 1)][0], lane);
            __syncwarp();  // the slot is in registers
            ask(r + S);
            st.fold(valid, fresh, lane);
            fresh = false;
            valid -= kStep;
            const bool ended = ++p.step == p.nt;
            if (!ended && r < n - 1) continue;
            // ---- the end of a unit, or of the share
            st.finish();
            if (began && ended) {
                const float vf = a.v_scale ? __ldg(a.v_scale + hd.kvh) : 1.f;
                const int gq = lane >> 2, cq = lane & 3;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int h = 2 * cq + e;
                    if (h >= hd.n) continue;
                    float x[CF::C];
#pragma unroll
                    for (int d = 0; d < CF::C; ++d) x[d] = st.o[d / 2][e + 2 * (d & 1)];
                    store_dims<F32>(a.out, (size_t)(hd.row0 + h) * D + gq * CF::C, x, st.l[e] == 0.f ? 0.f : vf / st.l[e]);
                    if (gq == 0 && a.lse) a.lse[hd.row0 + h] = (st.m[e] + log2f(st.l[e])) * kLn2;
                }
            } else {
                // a share that ends inside the unit: the ring is free, no copy is in flight
                st.dump(began ? reinterpret_cast<float *>(sm.ring[warp]) : sm.head[warp], lane);
                if (lane == 0) sm.cut[began][warp] = {p.b * U + p.y, first_place(bt, p, bt.more), p.nt, hd.kvh, hd.row0, hd.n};
            }
            fresh = began = true;
            if (r == n - 1) break;
            p.step = 0;  // on to the next unit
            if (++p.y == U) {
                p.y = 0;
#pragma unroll 1
                do p.nt = bt.steps(++p.b);
                while (p.nt == 0);
            }
        }
    }
    __syncthreads();

    // ---- units cut between warps.  Task w + 1: the unit that warp w began and did not end; task 0:
    // the unit that an earlier CTA began.  Its states lie in warp order.  Lane t looks task t up; a
    // warp then merges one head of one task at a time, each lane D / 32 dims.
    const int c_start = sh.start(blockIdx.x * kWarps), c_end = sh.start((blockIdx.x + 1) * kWarps);
    const int slot_floats = piece_floats(hpc, D);
    Cut tc = {-1, 0, 0, 0, 0, 0};
    unsigned has = 0;  // the warps that have a state of it
    if (lane <= kWarps) {
        int w0 = max(lane - 1, 0);
        if (lane == 0)
            while (w0 < kWarps - 1 && sm.empty[w0]) ++w0;
        tc = sm.cut[lane > 0][w0];
#pragma unroll
        for (int k = 0; k < kWarps; ++k)
            if (k > w0 && sm.cut[0][k].unit == tc.unit) has |= 1u << k;
        has |= 1u << w0;
    }
    // does the unit go on in other CTAs?  From which to which?
    const bool cross = !whole && tc.unit >= 0 && (tc.first < c_start || tc.first + tc.steps > c_end);
    const int c0 = cross ? sh.owner(tc.first) / kWarps : 0, c1 = cross ? sh.owner(tc.first + tc.steps - 1) / kWarps : 0;
    const unsigned crossing = __ballot_sync(kFull, cross);
    auto put = [&](int row, int kvh, const float(&acc)[V], float M, float L) {
        const float vf = a.v_scale ? __ldg(a.v_scale + kvh) : 1.f;
        store_dims<F32>(a.out, (size_t)row * D + lane * V, acc, L == 0.f ? 0.f : vf / L);
        if (lane == 0 && a.lse) a.lse[row] = (M + log2f(L)) * kLn2;
    };
    int h = warp;  // the tasks' heads, end to end, are dealt to the warps in turn
#pragma unroll 1
    for (unsigned left = __ballot_sync(kFull, tc.unit >= 0); left; left &= left - 1) {
        const int t = __ffs(left) - 1, heads = __shfl_sync(kFull, tc.n, t);
        const int row0 = __shfl_sync(kFull, tc.row0, t), kvh = __shfl_sync(kFull, tc.kvh, t);
        const unsigned of = __shfl_sync(kFull, has, t);
#pragma unroll 1
        for (; h < heads; h += kWarps) {
            auto state = [&](int w) { return w == t - 1 ? reinterpret_cast<const float *>(sm.ring[w]) : sm.head[w]; };
            const bool there = of >> lane & 1;
            const float m = there ? state(lane & (kWarps - 1))[kHeads * CF::RS + h] : kNoRef;
            const float M = warp_max(m), f = there ? ex2_approx(m - M) : 0.f;
            float L = 0.f, acc[V] = {};
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float fw = __shfl_sync(kFull, f, w);
                if (!(of >> w & 1)) continue;
                const float *s = state(w);
                L += fw * s[kHeads * CF::RS + kHeads + h];
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] += fw * s[h * CF::RS + lane * V + i];
            }
            if (crossing >> t & 1) {
                // a CTA's pieces: of the unit begun earlier, and of the one begun in it
                float *piece = a.pieces + ((size_t)blockIdx.x * 2 + (t > 0)) * slot_floats;
                store_dims<true>(piece, (size_t)h * D + lane * V, acc, 1.f);
                if (lane == 0) {
                    piece[hpc * D + h] = M;
                    piece[hpc * D + hpc + h] = L;
                }
            } else {
                put(row0 + h, kvh, acc, M, L);
            }
        }
        h -= heads;
    }
    if (!crossing) return;

    // ---- units cut between CTAs (at most one begun before this one and one in it): the last to
    // arrive merges the pieces
    __syncthreads();
    if (warp == 0 && cross) {
        // (release: the CTA's pieces, by way of the barrier; acquire: those of the CTAs before)
        const Arrivals at(c0, c1);
        unsigned *count = a.arrivals + at.word, before;
        asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(before) : "l"(count), "r"(1u << at.shift) : "memory");
        const bool last = (before >> at.shift & at.mask) == (unsigned)(c1 - c0);
        if (last) atomicSub(count, (unsigned)(c1 - c0 + 1) << at.shift);  // zero again for the next launch
        sm.last[lane > 0] = last ? c1 - c0 + 1 : 0;
    }
    __syncthreads();
#pragma unroll 1
    for (unsigned left = crossing; left; left &= left - 1) {
        const int t = __ffs(left) - 1, np = sm.last[t > 0], from = __shfl_sync(kFull, c0, t);
        if (np == 0) continue;
        const int heads = __shfl_sync(kFull, tc.n, t), row0 = __shfl_sync(kFull, tc.row0, t);
        const int kvh = __shfl_sync(kFull, tc.kvh, t);
        // begun in the unit's first CTA (piece 1), carried on in the others (piece 0)
        auto piece = [&](int k) { return a.pieces + ((size_t)(from + k) * 2 + (k == 0)) * slot_floats; };
#pragma unroll 1
        for (h = warp; h < heads; h += kWarps) {
            float M = kNoRef, L = 0.f, acc[V] = {};
#pragma unroll 1
            for (int c = 0; c < np; c += 32) {
                const bool there = c + lane < np;
                const float *mine = piece(there ? c + lane : c) + hpc * D + h;
                const float m = there ? __ldcg(mine) : kNoRef, l = __ldcg(mine + hpc);
                const float up = fmaxf(M, warp_max(m)), f = there ? ex2_approx(m - up) : 0.f, keep = ex2_approx(M - up);
                M = up;
                L *= keep;
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] *= keep;
                const int end = min(32, np - c);
#pragma unroll 4
                for (int j = 0; j < end; ++j) {
                    const float fj = __shfl_sync(kFull, f, j);
                    L += fj * __shfl_sync(kFull, l, j);
                    const float *s = piece(c + j) + h * D + lane * V;
#pragma unroll
                    for (int i = 0; i < V; i += 2) {
                        const float2 x = __ldcg(reinterpret_cast<const float2 *>(s + i));
                        acc[i] += fj * x.x;
                        acc[i + 1] += fj * x.y;
                    }
                }
            }
            put(row0 + h, kvh, acc, M, L);
        }
    }
}

template <int D, bool F32>
cudaError_t launch_t(const Fp4DecodeArgs &a, cudaStream_t stream) {
    const int g = a.Hq / a.Hk;
    const int hpc = a.pack_gqa ? (g < kHeads ? g : kHeads) : 1;
    const size_t smem = sizeof(Smem<D>) + 128;
    auto kern = decode_fp4_kernel<D, F32>;
    // once per device: the call takes as long as a tenth of a small step
    static std::atomic<uint64_t> ready{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (!(ready.load(std::memory_order_acquire) & bit)) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        ready.fetch_or(bit, std::memory_order_release);
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.sms * kCtasPerSm);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, a, hpc, (g + hpc - 1) / hpc);
}

}  // namespace

// Two pieces per CTA of the largest grid.
size_t fp4_decode_piece_bytes(int Hq, int Hk, int D) {
    const int g = Hq / Hk, hpc = g < kHeads ? g : kHeads;
    return (size_t)kMaxCtas * 2 * piece_floats(hpc, D) * sizeof(float);
}

cudaError_t launch_decode_fp4(const Fp4DecodeArgs &a, cudaStream_t stream) {
    if (a.D == 128) return a.out_f32 ? launch_t<128, true>(a, stream) : launch_t<128, false>(a, stream);
    return a.out_f32 ? launch_t<64, true>(a, stream) : launch_t<64, false>(a, stream);
}

}  // namespace gqa
