// Host-side interface between the C ABI (gdn_api.cu) and the kernel
// translation units.  Not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "../../include/gdn_decode.h"

struct gdn_pool {
    float *data;
    int num_slots;
    gdn_dims dims;
    bool owned;
    int work_index; // this pool's pair of work counters in the library's table
    unsigned int *qk_count; // in-place counters [num_slots][qk_stride], or NULL
    int qk_stride;          // counters a slot: hk rounded up to a multiple of 4
    bool owns_qk_count;     // allocated with the pool (create), else caller memory
};

struct conv_pool {
    void *data;
    int num_slots;
    int channels;
    int width;
    int dtype;
    bool owned;
};

struct kv_page_pool {
    void *k, *v; // each [layers][num_pages][hkv][page_size][d]
    int num_pages, page_size, layers, hkv, d, dtype;
    bool owned;
    // tensor maps of k and v for paged_attention, made by its first call
    std::mutex map_mutex;
    bool mapped;
    CUtensorMap kmap, vmap;
    kv_page_pool(void *k_, void *v_, int pages, int size, int layers_, int hkv_, int d_, int dtype_, bool owned_)
        : k(k_), v(v_), num_pages(pages), page_size(size), layers(layers_), hkv(hkv_), d(d_), dtype(dtype_),
          owned(owned_), mapped(false)
    {
    }
};

namespace gdn {

// The C ABI's error state, for its other translation units: set the calling
// thread's message and return the code; clear it (GDN_OK); report a failed
// runtime call; find the current device's error word.
int api_fail(int code, const char *fmt, ...);
int api_ok();
int api_cuda_fail(cudaError_t e, const char *what);
int api_error_word(int **out);

// Everything one launch of the state kernels needs.  Pointers are device
// pointers; layouts as in gdn_decode.h.
struct StepArgs {
    // gdn_decode_step inputs (unused by the fused layer)
    const void *q, *k, *v;
    // shared
    const void *a, *b;
    const float *A_log, *dt_bias;
    float *pool;
    int num_slots;
    const int32_t *read_slot, *write_slot;
    int in_place;
    void *out;
    int rows, hk, hv, dk, dv;
    int *err;
    unsigned int *work; // the pool's two work counters (claim, producers done), zero between launches
    int commit;         // twin only: swap read_slot and write_slot once every producer has read them
    const int32_t *n_live; // device count or NULL: rows at or past *n_live are left alone (outputs zero)
    unsigned int *qk_count; // fused layer, in place: the pool's counters [slot][qk_stride], or NULL
    int qk_stride;
    // fused layer only
    const void *x;
    void *conv;        // conv pool data
    const void *w;     // [C][W]
    const void *bias;  // [C] or null
    int silu;
    int width;
    int channels;
};

struct ConvArgs {
    const void *x;
    int x_stride;
    void *conv;
    int num_slots;
    const int32_t *read_slot, *write_slot;
    const void *w, *bias;
    int silu;
    void *out;
    int rows, channels, width;
    int *err;
};

// Many tokens a sequence (prefill, verification).  Sequence r holds tokens
// [cu_seqlens[r], cu_seqlens[r+1]) of the packed token-major inputs.
struct PrefillArgs {
    const void *q, *k, *v, *a, *b;
    const float *A_log, *dt_bias;
    float *pool;
    int num_slots;
    const int32_t *cu_seqlens, *read_slot;
    const int32_t *write_slot; // NULL: in place
    const int32_t *token_slot; // non-NULL: the state after each token goes to token_slot[t]
    void *out;
    int nseq, total_tokens, hk, hv, dk, dv;
    int *err;
    void *work;                // gdn_prefill_chunked, bf16: the chunk prep workspace
};

struct ConvPrefillArgs {
    const void *x; // [T][C]
    void *conv;
    int num_slots;
    const int32_t *cu_seqlens, *read_slot, *write_slot, *token_slot;
    const void *w, *bias;
    int silu;
    void *out;
    int nseq, total_tokens, channels, width;
    int *err;
};

// Linear attention with a decay for each head: one token a row, or (with
// cu_seqlens) packed sequences.
struct LinearArgs {
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride; // elements a token
    const float *log_decay;
    long long decay_stride;                 // elements a token: hv, or 0 (a decay a head)
    float *pool;
    int num_slots;
    const int32_t *cu_seqlens, *read_slot;
    const int32_t *write_slot;              // NULL: in place
    float scale;
    void *out;
    int rows, total_tokens, hk, hv, dk, dv; // rows: of the batch, or sequences
    int most;                               // tokens of the longest sequence that the serial kernel takes
    int span;                               // the chunked kernels': tokens a segment, whole chunks (linear_divide)
    bool cut;                               // whether sequences of the mean length have several segments
    int *err;
    void *work;                             // the chunked kernels'
};

// One layer of a page pool, for a kernel.
struct PageView {
    void *k, *v; // the layer's [num_pages][hkv][page_size][d]
    int num_pages, page_size, page_shift, hkv, d, layer;
};

// New tokens of cache rows: row r's are [cu_seqlens[r], cu_seqlens[r+1]).
struct CacheRows {
    const int32_t *table;
    const int32_t *seq_len, *cu_seqlens;
    int max_pages, rows, total_tokens;
};

struct PrologueArgs {
    const void *q, *k, *v;
    long long q_stride, k_stride, v_stride; // elements a token
    PageView pages;
    CacheRows c;
    const float *rope;
    int rope_positions, rot, interleaved;
    const float *q_norm, *k_norm;
    float eps;
    void *q_out;
    int hq;
    int *err;
};

struct AttentionArgs {
    const void *q;
    long long q_stride;
    PageView pages;
    CacheRows c;
    float scale;
    void *out;
    int hq;
    void *work;
    int *err;
};

// Groups of rows that share their first pages (paged_attention_shared).
struct SharedPrefix {
    const int32_t *bounds, *prefix; // [groups + 1], [rows][2]
    int groups;
};

struct PageTables {
    int32_t *table;
    int table_rows, max_pages;
    int32_t *seq_len, *refs;
    int num_pages, page_size;
    int *err;
};

// Launchers return cudaSuccess or the launch error.  Shapes were validated by
// the caller.
cudaError_t launch_gdn_step(const StepArgs &a, int dtype, cudaStream_t s);
cudaError_t launch_gdn_layer(const StepArgs &a, int dtype, cudaStream_t s);
cudaError_t launch_conv(const ConvArgs &a, int dtype, cudaStream_t s);
cudaError_t launch_gdn_prefill(const PrefillArgs &a, int dtype, cudaStream_t s);
cudaError_t launch_conv_prefill(const ConvPrefillArgs &a, int dtype, cudaStream_t s);
// The chunked (tensor-core) form of launch_gdn_prefill: in place or twin, no token slots.
// bf16 activations run the tcgen05 kernel (gdn_chunked_tc.cu), fp32 the mma.sync one.
cudaError_t launch_gdn_prefill_chunked(const PrefillArgs &a, int dtype, cudaStream_t s);
cudaError_t launch_gdn_prefill_chunked_tc(const PrefillArgs &a, cudaStream_t s);
// Bytes of the workspace the bf16 chunked prefill needs (0 for no sequence).
size_t prefill_chunked_workspace_bytes(int nseq, int total_tokens, int hv);

// Linear attention: one token a row, and packed sequences token after token
// (those of up to a.most tokens).
cudaError_t launch_linear_decode(const LinearArgs &a, int dtype, cudaStream_t s);
cudaError_t launch_linear_serial(const LinearArgs &a, int dtype, cudaStream_t s);
// Packed sequences: the short ones by the serial kernel, the others in chunks, bf16 with dk and dv 64 or 128 on the
// tensor cores (launch_linear_chunked), the rest to fp32's precision.
// linear_divide comes before the others and sets a.span and a.cut from the counts and sizes (of one sequence and token at least).
void linear_divide(LinearArgs &a, int dtype);
size_t linear_prefill_workspace_bytes(const LinearArgs &a);
cudaError_t launch_linear_prefill(LinearArgs a, int dtype, cudaStream_t s);
int linear_chunked_segment(const LinearArgs &a, bool &cut);
cudaError_t launch_linear_chunked(const LinearArgs &a, cudaStream_t s);

// Attention layers over a page pool.
cudaError_t launch_rope_table(const double *inv_freq, int rot, int positions, double mscale, float *table,
                              cudaStream_t s);
cudaError_t launch_attn_prologue(const PrologueArgs &a, int dtype, cudaStream_t s);
// paged_attention and, with f, paged_attention_shared: bf16 (attn_tc.cu) and fp32 (attn_f32.cu)
size_t attention_tc_workspace_bytes(int d, int hq, int hkv, int total_tokens, bool shared);
size_t attention_f32_workspace_bytes(int d, int hq, int hkv, int total_tokens, bool shared);
cudaError_t launch_paged_attention_tc(const AttentionArgs &a, const SharedPrefix *f, kv_page_pool &pool, cudaStream_t s);
cudaError_t launch_paged_attention_f32(const AttentionArgs &a, const SharedPrefix *f, cudaStream_t s);
cudaError_t launch_pages_shared(const CacheRows &c, const int32_t *bounds, int groups, int page_size, int32_t *prefix,
                                int *err, cudaStream_t s);
cudaError_t launch_pages_reserve(const PageTables &t, const int32_t *list_rows, const int32_t *tokens, int n,
                                 int32_t *status, cudaStream_t s);
cudaError_t launch_pages_fork(const PageTables &t, const int32_t *src_rows, const int32_t *dst_rows, int n,
                              int32_t *move_src, int32_t *move_dst, int32_t *move_count, int32_t *status,
                              cudaStream_t s);
cudaError_t launch_pages_free(const PageTables &t, const int32_t *list_rows, int n, cudaStream_t s);
cudaError_t launch_pages_compact(const PageTables &t, int32_t *table_out, int32_t *refs_out, int32_t *remap,
                                 int32_t *move_src, int32_t *move_dst, int32_t *move_count, int32_t *scratch,
                                 cudaStream_t s);
cudaError_t launch_pages_copy(const kv_page_pool &pool, const int32_t *src, const int32_t *dst, int n,
                              const int32_t *count, int *err, cudaStream_t s);

// True when the state kernels are built for (dk, dv).
bool step_shape_supported(int dk, int dv);
// True when the chunked prefill is built for (dk, dv).
bool chunked_shape_supported(int dk, int dv);
// True when the fused layer can run this shape.
bool layer_shape_supported(int dk, int dv, int group, bool in_place);

} // namespace gdn
