// quant_kv.h -- host-side interfaces of the quantised-cache kernels (write_kv.cu, read_kv.cu,
// decode_fp4.cu).  Not part of the public ABI.
#pragma once

#include <cuda_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "gqa_internal.h"

namespace gqa {

// Writing tokens into the cache: the last Lq_b = cu_q[b+1] - cu_q[b] tokens of every sequence.
struct WriteArgs {
    const void *k_new, *v_new;      // bf16 rows of [Hk][D]
    long long k_stride, v_stride;   // elements from one row to the next
    const int32_t *cu_q;            // NULL: one row per sequence, none where seq_lens[b] = 0
    void *k_pages, *v_pages;
    float *k_scale, *v_scale;       // e4m3: [num_pages][Hk]; fp4: [Hk] or NULL
    const int32_t *page_table;
    int pt_stride;
    const int32_t *seq_lens;
    int B, Hk, D, P, num_pages;
    int kv_dtype;
    int total_q, max_q_len;
    int *err;
};
cudaError_t launch_write_kv(const WriteArgs &a, cudaStream_t stream);

// Reading tokens [starts[b], seq_lens[b]) back as bf16.
struct ReadArgs {
    const void *k_pages, *v_pages;
    const float *k_scale, *v_scale;
    const int32_t *page_table;
    int pt_stride;
    const int32_t *starts;          // NULL: 0
    const int32_t *seq_lens;
    const int64_t *cu_out;          // [B+1] rows, or pages when paged
    int B, Hk, D, P, num_pages;
    int kv_dtype;
    long long total;                // rows, or pages when paged
    int paged;
    void *k_out, *v_out;            // bf16
    int *err;
};
cudaError_t launch_read_kv(const ReadArgs &a, cudaStream_t stream);

// Decode over a 4-bit cache.
struct Fp4DecodeArgs {
    const void *q;
    const uint8_t *k_pages, *v_pages;
    const float *k_scale, *v_scale;  // [Hk] or NULL
    const int32_t *page_table;
    int pt_stride;
    const int32_t *seq_lens;
    int B, Hq, Hk, D, P, num_pages;
    float scale;
    int pack_gqa;
    void *out;
    int out_f32;
    float *lse;
    int *err;
    unsigned *arrivals;  // of a cut unit's pieces, in the workspace's header; zero between launches
    float *pieces;
    int sms;
};
size_t fp4_decode_piece_bytes(int Hq, int Hk, int D);  // a multiple of 256
cudaError_t launch_decode_fp4(const Fp4DecodeArgs &a, cudaStream_t stream);

}  // namespace gqa
