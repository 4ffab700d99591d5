// Internal (non-exported) declarations shared by the host side of libgdr:
// kernel argument blocks and launchers.  Not part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>
#include <type_traits>

namespace gdr {

// Token-loop kernel (dense recurrent, paged decode, verify).
struct RecurrentArgs {
    const void* q;
    const void* k;
    const void* v;
    const float* g;
    const void* beta;
    void* o;
    const int32_t* cu_seqlens;   // NULL: see one_token_per_seq
    int32_t one_token_per_seq;   // with cu_seqlens NULL: 1 -> sequence n is token n; 0 -> one sequence of T tokens
    int32_t prefetch;            // 1: load token t+1's inputs while token t computes (multi-token sequences)
    int64_t T;
    const void* src;             // state source [*, HV, V, K] (pool or initial state), NULL = zeros
    void* dst;                   // state destination (pool on commit, final state), NULL = none
    const int32_t* slots;        // state_indices (paged) or NULL (dense: slot = sequence)
    void* ibuf;                  // per-token states [*, cache_steps, HV, V, K] or NULL
    const int32_t* ibuf_idx;
    int32_t cache_steps;
    int32_t N, HK, HV, V;
    float scale;
    // gating front, read only by the gated instantiation: g and beta are formed per token from
    // the raw inputs a, b and the per-head A_log, dt_bias; q and k are l2-normalised when asked
    const void* ga;              // a [T, HV] io dtype
    const void* gb;              // b [T, HV] io dtype
    const float* A_log;          // [HV]
    const float* dt_bias;        // [HV]
    float l2_eps;
    int32_t qk_l2norm;
    float beta_mul;              // 1, or 2 when negative eigenvalues are allowed
};

// Copy n fp32 values src -> dst (zeros when src is NULL); nothing when src == dst.
hipError_t launch_state_copy(const float* src, float* dst, int64_t n, hipStream_t stream);

// dtype codes: 0 = fp32, 1 = bf16; ib_dtype -1 = no intermediate buffer.  gated needs !per_k.
// Requires a.T >= 1.
hipError_t launch_recurrent(const RecurrentArgs& a, int K, int io_dtype, int st_dtype, int ib_dtype,
                            bool per_k, bool gated, hipStream_t stream);

// Gating front as a pass of its own: normalised q, k and activated g, beta for every token.
struct GatingArgs {
    const void* q;
    const void* k;
    void* q_out;                 // may equal q (each row is read whole before it is written)
    void* k_out;
    const void* a;
    const void* b;
    const float* A_log;
    const float* dt_bias;
    float* g_out;                // [T, HV] fp32
    void* beta_out;              // [T, HV] io dtype
    int64_t T;
    int32_t HK, HV;
    float l2_eps;
    int32_t qk_l2norm;
    float beta_mul;
};

hipError_t launch_gating(const GatingArgs& a, int K, int io_dtype, hipStream_t stream);

// Chunked path (64-token chunks).
struct ChunkArgs {
    const void* q;
    const void* k;
    const void* v;               // NULL reads as zeros
    const float* g;
    const void* beta;
    const int32_t* cu_seqlens;   // NULL only when N == 1
    const float* h0;             // [N, HV, V, K] or NULL (zeros)
    void* o;                     // NULL: outputs not written
    float* ht;                   // [N, HV, V, K] or NULL; may equal h0 (each thread reads its part first)
    // non-NULL selects the paired run of the segmented route (bf16, K = V, either gate): besides
    // ht, map [N, HV, K, K] receives the end state from the identity with v = 0; q and o are unused
    float* map;
    int64_t T;
    int32_t N, HK, HV, K, V;
    float scale;
};

hipError_t launch_chunk(const ChunkArgs& a, int io_dtype, bool per_k, hipStream_t stream);

// Fused KDA decode front (gdr_kda.hip): convolution + SiLU, gate projection, q/k l2 norm, beta,
// per-key-channel recurrence against the paged state, optional gated RMSNorm epilogue.
struct KdaArgs {
    const void* q;               // [T, HV, K] io dtype, raw (before the convolution)
    const void* k;               // [T, HV, K]
    const void* v;               // [T, HV, V]
    const int32_t* cu_seqlens;   // [N + 1] or NULL (one token per sequence)
    void* pool;                  // [slots, HV, V, K] state dtype
    const int32_t* slots;        // [N]; negative = padded sequence
    int32_t commit;              // write the state and the convolution windows back
    void* o;                     // [T, HV, V] io dtype
    int32_t conv_width;          // 1..4
    const void* conv_weight;     // [C, W] io dtype, C = 2 HV K + HV V (q | k | v)
    const void* conv_bias;       // [C] or NULL
    void* conv_state;            // [slots, C, W - 1] io dtype
    const void* gate_in;         // [T, R] io dtype
    const void* gate_weight;     // [HV K, R] io dtype
    int32_t gate_rank;           // R, a multiple of 8
    const float* A_log;          // [HV]
    const float* dt_bias;        // [HV K]
    const void* b;               // [T, HV] io dtype
    float l2_eps;
    const void* norm_weight;     // [V] io dtype, or NULL: no epilogue
    const void* norm_gate;       // [T, HV, V] io dtype
    float norm_eps;
    float scale;
    int32_t N, HV;
};

hipError_t launch_kda(const KdaArgs& a, int K, int V, int io_dtype, int st_dtype, hipStream_t stream);

// Context parallelism for a few long sequences (gdr_cp.hip): every sequence is cut into segments of
// seg_tokens tokens (a multiple of 64; a sequence's last segment may be shorter) that run as the
// sequences of three chunk-kernel launches.
constexpr int kCpWorkgroups = 256;   // target chunk-kernel workgroups per run: one per CU of the part
constexpr int kCpMinChunks = 8;      // at least this many chunks per segment
constexpr int kCpMinSegments = 4;    // segments per sequence; below this the three runs cost more than they save

struct CpPlan {
    int P;                           // segments the workspace holds (an upper bound on the real count); 1 = no CP
    int N;                           // sequences
    int64_t seg_tokens;
    size_t cu_seg, seg_first, B, M, S, total;   // workspace offsets (256-byte aligned) and size
};

CpPlan cp_plan(int64_t T, int32_t N, int32_t HV, int32_t K, int32_t V, int io_bytes);
// identity: also set every segment map to the identity (the start state of the separate map run)
hipError_t launch_cp_setup(const CpPlan& pl, char* ws, const int32_t* cu, int64_t T, int32_t HV, int32_t K,
                           bool identity, hipStream_t stream);
hipError_t launch_cp_scan(const CpPlan& pl, char* ws, const float* h0, int32_t HV, int32_t K, int32_t V,
                          hipStream_t stream);
hipError_t launch_cp_final(const CpPlan& pl, const char* ws, float* out, int32_t HV, int32_t K, int32_t V,
                           hipStream_t stream);

// Gated linear recurrence (gdr_linear.hip).
constexpr int kLinearBlock = 64;     // tokens per row of block_states (GDR_LINEAR_BLOCK)

struct LinearArgs {
    const void* x;               // [T, D] io dtype
    const void* gate;            // [T, D] fp32 log-decay, or io dtype before the sigmoid
    const int32_t* cu;           // [N + 1]; NULL: one sequence (scan), one token per sequence (decode)
    const float* h0;             // [N, D] or NULL (zeros)
    void* y;                     // [T, D] io dtype
    float* ht;                   // [N, D] or NULL
    float* block_states;         // [ceil(T / kLinearBlock), D]: the state entering each block, or NULL
    uint32_t* ticket;            // workspace, set by the launcher: tiles handed out so far
    uint64_t* runs;              // workspace: a word per (tile, channel)
    // backward
    const void* dy;              // [T, D] io dtype
    const float* dht;            // [N, D] or NULL (zeros)
    void* dx;                    // [T, D] io dtype
    void* dgate;                 // [T, D] the gate's dtype
    float* dh0;                  // [N, D] or NULL
    // decode
    void* pool;                  // [num_slots, D] state dtype
    const int32_t* slots;        // [N]; negative = padded sequence
    int32_t num_slots, commit, max_q_len;
    int64_t T, D;
    int32_t N;
    int32_t nch;                 // set by the launcher: workgroups across the channels, tiles along the tokens
    int64_t tiles;
};

size_t linear_workspace(int64_t T, int64_t D);
// kind 0: log-decay, 1: sigmoid.  Requires a.T >= 1 and a workspace of linear_workspace bytes.
hipError_t launch_linear_scan(const LinearArgs& a, char* ws, int kind, int io_dtype, bool backward, hipStream_t stream);
hipError_t launch_linear_decode(const LinearArgs& a, int kind, int io_dtype, int st_dtype, hipStream_t stream);
// dst = src (zeros without src), count floats: the states of a batch of empty sequences.
hipError_t launch_linear_copy(const float* src, float* dst, int64_t count, hipStream_t stream);

// Beam search (gdr_beam.hip).
constexpr int kBeamMaxBeams = 32, kBeamMaxOut = 64, kBeamMaxVocab = 1 << 20;

struct BeamArgs {
    const void* logits;          // [batch, beams, >= vocab] io dtype, rows `stride` elements apart
    int64_t stride;
    const float* scores;         // [batch, beams]
    const uint8_t* finished;     // [batch, beams] or NULL
    float* out_scores;           // [batch, out]
    int32_t* out_parents;
    int32_t* out_tokens;
    int32_t batch, beams, vocab, out, eos;
    // workspace, per (row, split)
    double* sums;
    float* tops;
    uint64_t* entries;           // [row, split, out]
    int32_t splits, chunk;       // set by the plan
    int32_t merge_list;          // set by the launcher: candidates the merge may hold
};

struct BeamPlan {
    int per_thread;              // logits per thread of a row kernel's workgroup
    int splits, chunk;
    size_t sums, tops, entries, total;   // workspace offsets (256-byte aligned) and size
};

BeamPlan beam_plan(int32_t batch, int32_t beams, int32_t vocab, int32_t out);
hipError_t launch_beam_select(const BeamArgs& a, const BeamPlan& pl, char* ws, int io_dtype, hipStream_t stream);

struct ReorderArgs {
    char* pool;                  // [layers, num_slots, slot_bytes]
    int64_t slot_bytes, layer_bytes;
    int32_t layers, num_slots, batch, beams;
    const int32_t* slots;        // [batch, beams]
    const int32_t* parents;      // [batch, beams]
    int32_t* slots_out;          // [batch, beams]
};

hipError_t launch_beam_reorder(const ReorderArgs& a, hipStream_t stream);

// Rotary positions and the paged cache's new rows (gdr_rope.hip).  Strides in elements from one token's row to the
// next; q_out, k_out dense.
struct RopeArgs {
    const void *q, *k, *v;       // [T, HQ | HK, D] io dtype; q may be NULL, v without pages
    int64_t q_stride, k_stride, v_stride;
    const int32_t* cu;           // [N + 1]; NULL: one sequence, or one token per sequence (one_token)
    bool one_token;
    const int32_t* context;      // [N]: tokens in the cache before these, negative = padded; NULL: 0
    const float* freq;           // [axes, rotary / 2]
    const int32_t* positions;    // [axes, T] or NULL
    int32_t axes, rotary, interleaved;
    void *k_pages, *v_pages;     // [num_pages, HK, 1 << page_shift, D] or NULL
    const int32_t* table;        // [N, max_pages]
    int32_t num_pages, max_pages, page_shift;
    void *q_out, *k_out;         // k_out may be NULL
    int64_t first;               // token of a launch
    int64_t T;
    int32_t N, HQ, HK;
};

hipError_t launch_rope_append(const RopeArgs& a, int D, int io_dtype, hipStream_t stream);

// Attention over packed prompts (gdr_attn.hip).  Strides in elements from one token's row to the next.
struct AttnPrefillArgs {
    const void *q, *k, *v;       // [T, HQ | HK, D] io dtype
    int64_t q_stride, k_stride, v_stride;
    const int32_t* cu;           // [N + 1], or NULL: one sequence
    void* o;                     // [T, HQ, D]
    float* lse;                  // [T, HQ] or NULL
    int64_t T;
    int32_t N, HQ, HK;
    float c;                     // |scale| log2(e), above 0
    bool negate;                 // scale < 0: the scores' sign is taken into q
    int32_t tiles;               // set by the launcher
};

int64_t attn_prefill_tiles(int64_t T);
hipError_t launch_attn_prefill(AttnPrefillArgs a, int D, int io_dtype, hipStream_t stream);

// Attention against a paged cache (gdr_attn_paged.hip).
struct AttnOpen {                // the block of rows that a workgroup has begun and left unfinished
    int32_t token0, row0, rows, kvh;
    int32_t parts;               // 0: none
};

struct AttnPagedArgs {
    const void* q;               // [T, HQ, D] io dtype
    int64_t q_stride;            // elements from one token's row to the next
    const int32_t* cu;           // [N + 1]; NULL: one token per sequence
    const int32_t* context;      // [N]: tokens before these, negative = padded
    const void *k_pages, *v_pages;   // [num_pages, HK, 1 << page_shift, D] io dtype
    const int32_t* table;        // [N, max_pages]
    int32_t num_pages, max_pages, page_shift;
    int32_t groups;              // 0: nothing is shared
    const int32_t* group_offsets;    // [groups + 1]
    const int32_t* prefix_lens;  // [groups]
    void* o;                     // [T, HQ, D]
    float* lse;                  // [T, HQ] or NULL
    int64_t T;
    int32_t N, HQ, HK;
    float c;                     // as AttnPrefillArgs
    bool negate;
    // set by the launcher
    int32_t per;                 // query heads per key head
    int32_t workers, per_head;            // workgroups, those of a key head
    int32_t rows, prefix_rows;            // rows of a block of one sequence's, of one group's
    int64_t capacity;            // tokens a row of the table can hold
    // workspace
    int32_t *start, *prefix_start;   // [N + 1], [groups + 1]: tiles before each unit on the line of a key head
    int32_t *item, *prefix_item;     // row blocks before each unit
    int32_t *pre, *group;        // [N]: keys read with the group's prefix, the group or -1
    int32_t* prefix;             // [groups]: keys of the prefix
    int32_t* first;              // [groups + 1]: the groups' first sequences
    AttnOpen* open;              // [workers]
    char *slots, *prefix_slots;  // parts: [rows, D] fp32, maxima, sums
};

struct AttnPagedPlan {
    int32_t workers, per_head, rows, prefix_rows;
    size_t start, item, pre, group, prefix_start, prefix_item, prefix, first, open, slots, prefix_slots, total;
};

AttnPagedPlan attn_paged_plan(int64_t T, int32_t N, int32_t HQ, int32_t HK, int D, int32_t max_q_len, int32_t groups);
hipError_t launch_attn_paged(AttnPagedArgs a, const AttnPagedPlan& p, char* ws, int D, int io_dtype, hipStream_t stream);

}  // namespace gdr
