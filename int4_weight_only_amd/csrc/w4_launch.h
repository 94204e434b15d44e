// w4_launch.h -- host-side launchers of the gfx950 kernels (called by the C ABI after the
// arguments have been validated).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kv_device.h"

namespace w4 {

// Threads of one launch, at most.
constexpr uint32_t kMaxThreads = UINT32_MAX;

hipError_t launch_pack(const float *w, int64_t d_out, int64_t d_in, int64_t ldw, int64_t span,
                       int64_t n_groups, int64_t k_pad, int mode, uint8_t *qweight,
                       uint16_t *scales, uint16_t *zeros, hipStream_t stream);

hipError_t launch_act_quant(const uint16_t *x, int64_t M, int64_t K, int64_t ldx, int8_t *q,
                            int64_t ldq, float *s_x, int32_t *q_sum, hipStream_t stream);

// Decode W4A16 for 1 <= M <= 64 (no scratch memory).
hipError_t launch_gemv(const uint16_t *x, int64_t M, int64_t ldx, const uint8_t *qweight,
                       const uint16_t *scales, const uint16_t *zeros, const uint16_t *bias,
                       int64_t d_out, int64_t d_in, int64_t k_pad, int64_t span,
                       int64_t n_groups, void *y, int64_t ldy, bool out_f32, hipStream_t stream);

hipError_t launch_w4a8(const int8_t *q, const float *s_x, int64_t M, int64_t ldq,
                       const uint8_t *qweight, const uint16_t *s_w, const uint16_t *bias,
                       int64_t d_out, int64_t d_in, int64_t k_pad, void *y, int64_t ldy,
                       bool out_f32, int32_t *acc, hipStream_t stream);

// Decode W4A16 for 2 <= M <= 64 on matrices with few rows per compute unit (groups of 128 or 256
// columns or one per row), the reduction dimension split over S column slices
// (decode_split.hip). With S > 1 the slices' fp32 partial sums go through a caller-provided
// workspace of split_work_bytes() bytes and a second kernel adds them.
bool split_forced();  // the test build's hook (always false in the product library)
struct SplitPlan {
    int tw, S, slices, xk, gshift;
    bool ok;
};
SplitPlan plan_split(int64_t M, int64_t d_out, int64_t k_pad, int64_t span, int64_t n_groups);
size_t split_work_bytes(const SplitPlan &p, int64_t M, int64_t d_out);
bool gemv_split_supported(const SplitPlan &p, int64_t M, int64_t d_in, int64_t k_pad,
                          int64_t ldx);
hipError_t launch_gemv_split(const SplitPlan &p, const uint16_t *x, int64_t M, int64_t ldx,
                             const uint8_t *qweight, const uint16_t *scales,
                             const uint16_t *zeros, const uint16_t *bias, int64_t d_out,
                             int64_t d_in, int64_t k_pad, int64_t n_groups, void *work, void *y,
                             int64_t ldy, bool out_f32, hipStream_t stream);

// W4A8 with the activation quantization folded into the GEMV (bf16 x in; s_x out, nullable).
bool w4a8_linear_supported(int64_t M, int64_t k_pad);
hipError_t launch_w4a8_linear(const uint16_t *x, int64_t M, int64_t ldx, const uint8_t *qweight,
                              const uint16_t *s_w, const uint16_t *bias, int64_t d_out,
                              int64_t d_in, int64_t k_pad, void *y, int64_t ldy, bool out_f32,
                              float *s_x, int32_t *acc, hipStream_t stream);

// GPTQ (gptq.hip): Hessian, factorization of its damped inverse, column loop.
hipError_t launch_gptq_hessian(const uint16_t *x, int64_t N, int64_t d_in, int64_t ldx, float *h,
                               hipStream_t stream);
hipError_t launch_gptq_factor(float *h, int64_t d_in, float alpha, float *u, float *v,
                              uint8_t *dead, hipStream_t stream);
// The device address of this GPU's block-error array for w4_gptq_quantize_noalloc
// (kGqScratchRows rows of 32 floats).
constexpr int64_t kGqScratchRows = int64_t(1) << 16;
hipError_t gptq_scratch(float **ptr);
hipError_t launch_gptq_quantize(float *w, int64_t d_out, int64_t d_in, int64_t ldw,
                                const float *u, const uint8_t *dead, int64_t span, int mode,
                                uint8_t *qweight, uint16_t *scales, uint16_t *zeros,
                                int64_t n_groups, int64_t k_pad, float *ebuf, float *row_loss,
                                hipStream_t stream);

// Repack of bf16 weights on the 4-bit grid into the g32 symmetric format (qat_repack.hip).
bool qat_repack_supported(int64_t d_out, int64_t n_groups);
hipError_t launch_qat_repack(const uint16_t *w, int64_t d_out, int64_t d_in, int64_t ldw,
                             uint8_t *qweight, uint16_t *scales, uint8_t *m_out,
                             hipStream_t stream);

// W4A8 prefill GEMM on the int8 matrix cores (gemm_w4a8.hip), any M.
bool gemm_w4a8_supported(int64_t M, int64_t d_out, int64_t ldq, int64_t k_pad);
hipError_t launch_gemm_w4a8(const int8_t *q, const float *s_x, int64_t M, int64_t ldq,
                            const uint8_t *qweight, const uint16_t *s_w, const uint16_t *bias,
                            int64_t d_out, int64_t d_in, int64_t k_pad, void *y, int64_t ldy,
                            bool out_f32, int32_t *acc, hipStream_t stream);

hipError_t launch_gemm(const uint16_t *x, int64_t M, int64_t ldx, const uint8_t *qweight,
                       const uint16_t *scales, const uint16_t *zeros, const uint16_t *bias,
                       int64_t d_out, int64_t d_in, int64_t k_pad, int64_t span,
                       int64_t n_groups, void *y, int64_t ldy, bool out_f32, hipStream_t stream);

// Persistent streaming decode GEMVs (decode_stream.hip).
bool gemv_stream_supported(int64_t M, int64_t k_pad);
bool w4a8_stream_supported(int64_t M, int64_t k_pad, bool fused_quant);
hipError_t launch_gemv_stream(const uint16_t *x, int64_t M, int64_t ldx, const uint8_t *qweight,
                              const uint16_t *scales, const uint16_t *zeros, const uint16_t *bias,
                              int64_t d_out, int64_t d_in, int64_t k_pad, int chunk_group_shift,
                              int64_t n_groups, void *y, int64_t ldy, bool out_f32,
                              hipStream_t stream);
// act: int8 codes [M][ldq] with their scales in s_x, or (fused_quant) bf16 x [M][ldq], quantized
// per token inside the kernel with the act_quant rule, the scales written to s_x if given.
hipError_t launch_w4a8_stream(const void *act, bool fused_quant, float *s_x, int64_t M,
                              int64_t ldq, const uint8_t *qweight, const uint16_t *s_w,
                              const uint16_t *bias, int64_t d_out, int64_t d_in, int64_t k_pad,
                              void *y, int64_t ldy, bool out_f32, int32_t *acc,
                              hipStream_t stream);

// Few-token decode on the fp16 matrix cores (decode_mfma.hip): activations converted inside
// each block, one pass over the weights for all tokens of a 16-token tile; no workspace.
// W4A8 decode for 2..64 tokens on the int8 matrix cores (decode_w4a8_mfma.hip): the weights are
// read once per 16 tokens; same y and acc as the streaming kernel
bool w4a8_tok_supported(int64_t M, int64_t d_out, int64_t d_in, int64_t k_pad, int64_t ldq);
hipError_t launch_w4a8_tok(const int8_t *q, const float *s_x, int64_t M, int64_t ldq,
                           const uint8_t *qweight, const uint16_t *s_w, const uint16_t *bias,
                           int64_t d_out, int64_t d_in, int64_t k_pad, void *y, int64_t ldy,
                           bool out_f32, int32_t *acc, hipStream_t stream);
bool gemv_mfma_supported(int64_t M, int64_t d_out, int64_t d_in, int64_t k_pad, int64_t span,
                         int64_t n_groups, int64_t ldx, bool zp);
hipError_t launch_gemv_mfma(const uint16_t *x, int64_t M, int64_t ldx, const uint8_t *qweight,
                            const uint16_t *scales, const uint16_t *zeros, const uint16_t *bias,
                            int64_t d_out, int64_t d_in, int64_t k_pad, int64_t span,
                            int64_t n_groups, void *y, int64_t ldy, bool out_f32,
                            hipStream_t stream);

// One to four tokens on the int8 matrix cores (decode_i8.hip): activations as exact integer
// digits prepared inside each block, raw codes as the other operand; no workspace.
// glu: the fused gate/up GEMV with the SiLU(gate) * up epilogue (2 d_out weight rows, d_out
// outputs).
bool gemv_i8_supported(int64_t M, int64_t d_out, int64_t d_in, int64_t k_pad, int64_t span,
                       int64_t n_groups, int64_t ldx, bool glu = false);
bool gemv_i8_preferred(int64_t M, int64_t d_out, int64_t k_pad);
hipError_t launch_gemv_i8(const uint16_t *x, int64_t M, int64_t ldx, const uint8_t *qweight,
                          const uint16_t *scales, const uint16_t *zeros, const uint16_t *bias,
                          int64_t d_out, int64_t d_in, int64_t k_pad, int64_t span,
                          int64_t n_groups, void *y, int64_t ldy, bool out_f32, bool glu,
                          hipStream_t stream);

// Rotary positions with the cache append (rope.hip).
hipError_t launch_rope_append(const uint16_t *qkv, int64_t T, int64_t ldqkv, int n_heads,
                              const int32_t *q_start, const float *inv_freq, int rot_dim,
                              bool interleaved, float factor, const KvView &cache, uint16_t *q,
                              int64_t ldq, hipStream_t stream);

// Attention over the paged cache (attn_decode.hip, attn_prefill.hip).
struct AttnArgs {
    const uint16_t *q;
    int64_t T, ldq;
    int n_heads;
    const int32_t *q_start;  // NULL: one row per sequence
    float scale;
    int window, sinks;  // window 0: none
    void *y;
    int64_t ldy;
    bool out_f32;
    float *lse;
    void *work;
};
// Sizes that the kernels count in 31 bits and that one launch takes.
bool attn_decode_supported(int n_heads, const KvView &cache, int window, int sinks);
bool attn_prefill_supported(int64_t T, int n_heads, const KvView &cache, int window, int sinks);
size_t attn_decode_work_bytes(int n_heads, const KvView &cache, int window, int sinks);
hipError_t launch_attn_decode(const AttnArgs &a, const KvView &cache, hipStream_t stream);
size_t attn_prefill_work_bytes(int64_t T, int n_heads, const KvView &cache, int window, int sinks);
hipError_t launch_attn_prefill(const AttnArgs &a, const KvView &cache, hipStream_t stream);
// The same with every key of its sequence seen by each row.
hipError_t launch_attn_prefill_cross(const AttnArgs &a, const KvView &cache, hipStream_t stream);

// Attention of sequences that share prefixes, and cross attention (attn_units.hip). Without q_start
// a.T is the number of sequences.
size_t attn_shared_work_bytes(int64_t T, int n_heads, const KvView &cache);
bool attn_shared_supported(int64_t T, int n_heads, const KvView &cache, const Prefixes &prefixes);
hipError_t launch_attn_shared(const AttnArgs &a, const KvView &cache, const Prefixes &prefixes,
                              hipStream_t stream);
// (single: without q_start)
bool attn_cross_supported(int64_t T, int n_heads, const KvView &cache, bool single);
size_t attn_cross_work_bytes(int64_t T, int n_heads, const KvView &cache, bool single);
hipError_t launch_attn_cross(const AttnArgs &a, const KvView &cache, hipStream_t stream);

// Tables, lengths and slots of a step (tables.hip). slots, seqs and positions may be NULL; in_place:
// an output is the input of its kind.
struct TablesArgs {
    const int32_t *kv_len, *n_new, *spans;
    int32_t *page_table, *ring;
    const int32_t *ring_state;
    int32_t *q_start;
    int64_t *slots;
    int32_t *seqs, *positions, *kv_len_out, *spans_out, *ring_state_out;
    int64_t ld_table;
    int32_t n_seqs, table_cols, page_shift, ring_size, T;
};
hipError_t launch_batch_tables(const TablesArgs &a, bool in_place, hipStream_t stream);

// The residual norm (norm.hip); pointers checked, r and r_out of the type r_f32 says.
struct NormArgs {
    const uint16_t *x;
    const void *r;
    const uint16_t *w_post, *w_pre, *gate;
    void *r_out;
    uint16_t *y;
    int64_t ldx, ldr, ldg, ldr_out, ldy;
    int64_t T;
    int d;
    bool r_f32;
    float weight_offset, alpha, eps;
};
hipError_t launch_residual_norm(const NormArgs &a, hipStream_t stream);

// Records the text of a failed HIP call for w4_last_hip_error; returns W4_ERR_HIP.
int hip_fail(hipError_t err) noexcept;

// Number of compute units of the current device (cached per device). The entry points ask for it
// outside of any try block.
int device_cu_count() noexcept;

}  // namespace w4
