// kda_internal.hpp -- launcher interface between the C ABI (kda_api.cpp) and the
// kernel translation units.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime_api.h>
#include <hip/hip_vector_types.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

// The input front (kda_front in include/kda.h): gate_scale == nullptr means none.  With a
// front, the g argument holds raw gates z (g = -gate_scale[h] softplus(z)), beta raw values
// (beta = sigmoid), and q, k, v the inputs of the causal depthwise convolution.
struct FrontArgs {
    const float* gate_scale = nullptr;  // [H]
    const float* conv_q = nullptr;      // [H, dk, conv_width]
    const float* conv_k = nullptr;      // [H, dk, conv_width]
    const float* conv_v = nullptr;      // [H, dv, conv_width]
    void* conv_state = nullptr;         // [num_slots, H, conv_width - 1, 2 dk + dv], io dtype
    int conv_width = 1;
    int conv_silu = 0;
};

struct DecodeArgs {
    const void* q;
    const void* k;
    const void* v;
    const float* g;
    const float* beta;
    float* pool;
    const int32_t* slot_idx;
    void* o;
    float* records;  // nullptr: commit mode
    int N, T, H;
    float scale;
    int use_l2;
    FrontArgs front = {};
};

struct ReplayArgs {
    float* pool;
    const int32_t* slot_idx;
    const float* records;
    const int32_t* accepted;
    int N, T, H;
};

struct PrefillArgs {
    const void* q;
    const void* k;
    const void* v;
    const float* g;
    const float* beta;
    const int32_t* cu_seqlens;
    int num_seqs;
    int64_t total_tokens;
    float* pool;
    const int32_t* slot_idx;
    int h0_from_pool;
    int H;
    float scale;
    int use_l2;
    // output [T][H][dv]; nullptr (internal: the backward's forward pass, which keeps only the
    // chunk states) computes no O, and the intra-chunk records then skip QG and P
    void* o;
    void* workspace;
    // prefix snapshots (0 / nullptr / 0: none): the state after (j + 1) * snap_every tokens of
    // sequence i goes to slot snap_slots[i * max_snaps + j] (negative: skipped)
    int snap_every = 0;
    const int32_t* snap_slots = nullptr;
    int max_snaps = 0;
    // chunk states (nullptr: none): the fp32 [dk][dv] state entering chunk c of the batch
    // (global chunk index, head h) goes to chunk_states + (c * H + h) * chunk_state_stride
    float* chunk_states = nullptr;
    size_t chunk_state_stride = 0;  // floats
    FrontArgs front = {};
};

struct BackwardArgs {
    PrefillArgs fwd;   // the forward's inputs; its pool, slots, o and chunk states are set by
                       // backward_setup to parts of the backward workspace
    const float* h0;   // [num_seqs, H, dk, dv] or nullptr (zero)
    const void* dout;  // [T, H, dv] dtype
    const float* dht;  // [num_seqs, H, dk, dv] or nullptr (zero)
    void* dq;          // [T, H, dk] dtype
    void* dk;          // [T, H, dk] dtype
    void* dv;          // [T, H, dv] dtype
    float* dg;         // [T, H, dk]
    float* dbeta;      // [T, H]
    float* dh0;        // [num_seqs, H, dk, dv] or nullptr
};

// Softmax attention over packed prompts (kda_attn_prefill and its gradients).
struct AttnPrefillArgs {
    const void* q;  // token strides ldq, ldk, ldv in elements; heads contiguous in a token
    const void* k;
    const void* v;
    int64_t ldq, ldk, ldv;
    const int32_t* cu_q;
    const int32_t* cu_k;
    int num_seqs, total_q, total_k;
    int H, Hk;
    float scale_abs;  // |scale| (never 0: a zero scale comes as the smallest that keeps -inf * it)
    bool scale_neg;
    void* o;     // [total_q, H, dv]
    float* lse;  // [total_q, H] or nullptr
    void* workspace;
    int parts = 0;  // of shared tiles, that the workspace has room for (the launcher's)
};

struct AttnBackwardArgs {
    AttnPrefillArgs fwd;  // o and lse unused
    const void* o;        // [total_q, H, dv], the forward's
    const float* lse;     // [total_q, H], the forward's
    const void* dout;     // [total_q, H, dv]
    float scale;          // with its sign
    void* dq;             // [total_q, H, dk]
    void* dk;             // [total_k, Hk, dk]
    void* dv;             // [total_k, Hk, dv]
    void* workspace;
    // the launcher's: parts of shared tiles that the workspace has room for, dq's first
    int query_parts = 0, key_parts = 0;
};

struct AttnAppendArgs {
    const void* k;  // [total, Hk, dk], token strides ldk, ldv in elements
    const void* v;
    int64_t ldk, ldv;
    const int32_t* cu;
    const int32_t* start_len;
    int N, total, Hk;
    uint8_t* k_cache;  // [num_blocks, Hk, bt, dk]
    uint8_t* v_cache;  // [num_blocks, Hk, dv, bt]
    float* k_scale;    // [num_blocks, Hk]
    float* v_scale;
    int num_blocks, bt;
    const int32_t* table;  // [N, max_blocks]
    int max_blocks;
    bool clear;  // positions behind the new tokens become zero
};

struct AttnDecodeArgs {
    const void* q;  // [N, T, H, dk], token stride ldq in elements
    int64_t ldq;
    const uint8_t* k_cache;
    const uint8_t* v_cache;
    const float* k_scale;
    const float* v_scale;
    int num_blocks, bt, bt_log2;
    const int32_t* table;
    int max_blocks;
    const int32_t* context_len;
    int N, T, H, Hk;
    float scale;
    void* o;
    int row_groups;   // workgroups that share the rows of one (sequence, kv head)
    int pieces;       // about so many pieces of keys per kv head; 0: sequences are not cut
    float* part_o;    // [pieces made, T, H, dv]
    float2* part_ml;  // [pieces made, T, H] maximum and sum
};

// Each launcher returns hipSuccess or the launch error.
hipError_t launch_decode(const DecodeArgs& a, int bf16, int dk, int dv, hipStream_t stream);
hipError_t launch_replay(const ReplayArgs& a, int dk, int dv, hipStream_t stream);
hipError_t launch_state_stream(float* pool, const int32_t* slot_idx, int N, int H, int dk, int dv,
                               hipStream_t stream);
size_t prefill_workspace_bytes(int num_seqs, int64_t total_tokens, int H, int dk, int dv,
                               int bf16);
// False where the prefill LDS plan does not fit a CU (every dk, dv in {64, 128} fits).
bool prefill_supported(int bf16, int dk, int dv);
hipError_t launch_prefill(const PrefillArgs& a, int bf16, int dk, int dv, hipStream_t stream);
// The static prefill workspace of kda_chunk_prefill_noalloc (KDA_NOALLOC_SCRATCH_BYTES per
// GPU): its device address on the current device, looked up once per device; nullptr if the
// lookup fails.
void* prefill_noalloc_scratch();
size_t backward_workspace_bytes(int num_seqs, int64_t total_tokens, int H, int dk, int dv, int bf16);
void backward_setup(BackwardArgs& b, int dk, int dv, int bf16);
hipError_t launch_backward(const BackwardArgs& b, int bf16, int dk, int dv, hipStream_t stream);
size_t attn_prefill_workspace_bytes(int num_seqs, int64_t total_q, int64_t total_k, int H, int dv, int bf16);
hipError_t launch_attn_prefill(const AttnPrefillArgs& a, int bf16, int dk, int dv, hipStream_t stream);
size_t attn_backward_workspace_bytes(int num_seqs, int64_t total_q, int64_t total_k, int H, int Hk, int dk, int dv,
                                     int bf16);
hipError_t launch_attn_backward(const AttnBackwardArgs& b, int bf16, int dk, int dv, hipStream_t stream);
hipError_t launch_attn_append(const AttnAppendArgs& a, int bf16, int dk, int dv, hipStream_t stream);
int attn_decode_row_groups(int T, int H, int Hk);
int attn_decode_pieces(int N, int T, int H, int Hk, int bt, int max_blocks);
int64_t attn_decode_most_pieces(int N, int pieces);
hipError_t launch_attn_decode(const AttnDecodeArgs& a, int bf16, int dk, int dv, hipStream_t stream);

}  // namespace kda
