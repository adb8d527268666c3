// gdn_internal.h -- launcher interface between the C-ABI layer (gdn_api.cu)
// and the kernel files.  Host-only types; nothing here is exported.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

namespace gdn {

// A kernel's dynamic shared-memory limit belongs to its instance on one device,
// so it is raised once per device: bit d of `done` records device d (devices
// 0..63).  Two threads racing through the first call both raise it, which is
// harmless.
template <typename... KArgs>
cudaError_t raise_smem_limit(void (*kernel)(KArgs...), int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_acq_rel);
    return e;
}

// The same for kernels of which several CTAs are to share an SM: all of its memory beside the L1 cache goes to them (left to
// itself the driver provides for one CTA).
template <typename... KArgs>
cudaError_t raise_smem_limit_shared(void (*kernel)(KArgs...), int bytes, std::atomic<uint64_t>& done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (done.load(std::memory_order_acquire) & (1ull << (dev & 63))) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    return e == cudaSuccess ? raise_smem_limit(kernel, bytes, done) : e;
}

// SMs of the current device, queried once per device (1 if the query fails).
int sm_count();

// Launch with programmatic stream serialization: the kernel may become resident
// while the previous kernel of the stream finishes; it calls griddep_wait()
// before touching memory, so the stream order of memory effects is unchanged.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                       Args&&... args) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}

// The same for a grid of clusters of `size` CTAs along x.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, int size, cudaStream_t st,
                               Args&&... args) {
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)size;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}

// Geometry + options after validation (all derived fields filled in).
struct Geom {
    int Hk, Hv, D, K, G, C_ch, chunk;
    int act_bf16;  // 1: bf16 activations, 0: fp32
    float q_scale, l2_eps, norm_eps;
    uint32_t flags;
};

struct LayerParams {
    const void* conv_w;
    const void* conv_b;
    const float* A_log;
    const float* dt_bias;
    const void* norm_w;
};

// decode (r = 1, snap_idx = NULL: in place) and verify (snap_idx [B][r])
struct RowsJob {
    const void *x, *z, *a, *b;
    void* conv_pool;
    float* state_pool;
    const int32_t* slot_idx;
    const int32_t* snap_idx;
    void* y;
    int B, r, n_slots;
    // 0: decode (state in place) or verify with snapshots; 1: verify that
    // writes y only; 2: commit by recompute -- the first accepted[b] rows
    // applied in place, no y
    int mode = 0;
    const int32_t* accepted = nullptr;
};
cudaError_t launch_rows(const Geom& g, const LayerParams& prm, const RowsJob& job, cudaStream_t st);

// conv + SiLU over all channels, then roll each sequence's conv state
struct ConvJob {
    const void* x;
    void* conv_pool;
    const int32_t* slot_idx;
    void* u_out;
    int n_seq, n_tok, n_slots;
};
cudaError_t launch_conv_update(const Geom& g, const LayerParams& prm, const ConvJob& job,
                               cudaStream_t st);

struct CommitJob {
    void* conv_pool;
    float* state_pool;
    const int32_t *slot_idx, *snap_idx, *accepted;
    int B, r, n_slots;
};
cudaError_t launch_commit(const Geom& g, const CommitJob& job, cudaStream_t st);

// prefill: single sequence (cu_seqlens == NULL) or packed varlen
struct PrefillJob {
    const void *x, *z, *a, *b;
    void* y;
    int64_t n_tokens;
    int n_seq;
    const int32_t* cu_seqlens;  // NULL: one sequence [0, n_tokens)
    // varlen: pools + slots
    const int32_t* slot_idx;
    const uint8_t* has_init;
    float* state_pool;
    void* conv_pool;
    int n_slots;
    // single sequence: direct pointers
    const float* s0;
    float* s_final;
    const void* conv0;
    void* conv_final;
    void* workspace;
    size_t ws_bytes;
    // varlen snapshots every ckpt_every tokens (0: none) into pool slots
    // ckpt_slots[ckpt_offset[s] + k]
    int32_t ckpt_every;
    const int32_t* ckpt_offset;
    const int32_t* ckpt_slots;
};
size_t prefill_workspace_bytes(const Geom& g, int64_t n_tokens, int n_seq);
// the tcgen05 path for d = 128, chunk 64, bf16 activations (gdn_chunk16.cu):
// the state chain only; the caller launches the conv-state tail after it
bool chunk16_applies(const Geom& g);
size_t chunk16_workspace_bytes(const Geom& g, int64_t n_tokens, int n_seq);
cudaError_t chunk16_launch(const Geom& g, const LayerParams& prm, const PrefillJob& job, cudaStream_t st);
cudaError_t launch_prefill(const Geom& g, const LayerParams& prm, const PrefillJob& job,
                           cudaStream_t st);

// out[t][n] = sum_k act[t][k] w[n][k] (bf16, fp32 accumulation); weight rows
// [seg.n0, seg.n1) land in columns [0, n1 - n0) of seg.out (row stride seg.ld)
struct ProjOut {
    void* out;
    int64_t ld;
    int32_t n0, n1;
};
struct ProjJob {
    const void* w;    // bf16 [n_out][k]
    const void* act;  // bf16 [n_tok][k]
    int32_t n_out, k;
    int64_t n_tok;
    int nseg;
    ProjOut seg[4];
    void* ws;  // fp32 partial sums when K is split (proj_plan().ws_bytes)
    size_t ws_bytes;
};
struct ProjPlan {
    int bt;           // tokens per tile
    int64_t n_tiles;  // (128-row weight block, token block) tiles
    int ks;           // CTAs per tile splitting K (1: none)
    size_t ws_bytes;  // workspace for the split's partial sums
};
ProjPlan proj_plan(int32_t n_out, int32_t k, int64_t n_tok);
cudaError_t launch_proj(const ProjJob& job, cudaStream_t st);

// decode attention over a paged KV cache (bf16), GQA with G = Hq / Hkv in
// {1, 2, 4, 8, 12, 16}; D in {128, 256}
struct AttnJob {
    const void *q, *k_new, *v_new;
    void *k_pool, *v_pool;
    const int32_t* block_table;
    const int32_t* seq_lens;
    void* o;
    void* ws;
    int B, Hq, Hkv, D, page, max_pages, n_pages, max_seq_len;
    float scale;
};
struct AttnPlan {
    int n_split, span;
};
AttnPlan attn_plan(int B, int Hq, int Hkv, int max_seq_len);
size_t attn_workspace_bytes(int B, int Hq, int Hkv, int D, int max_seq_len);
cudaError_t launch_attn_decode(const AttnJob& job, cudaStream_t st);

// prefill attention: new tokens cu_seqlens[s] .. cu_seqlens[s+1] of sequence s at
// positions ctx_lens[s] + i, appended to the pages, then causal attention
struct AttnPfJob {
    const void *q, *k_new, *v_new;
    void *k_pool, *v_pool;
    const int32_t* block_table;
    const int32_t* cu_seqlens;
    const int32_t* ctx_lens;
    void* o;
    int n_seq, Hq, Hkv, D, page, max_pages, n_pages;
    int64_t n_tokens;
    float scale;
};
cudaError_t launch_attn_prefill(const AttnPfJob& job, cudaStream_t st);

// ---- trees of drafted tokens ----
// nodes cu_nodes[b] .. cu_nodes[b+1] of sequence b; parents[i]: the node within the
// sequence that node i follows, or the end of the cached sequence where it is outside [0, i)

// attention of every node over the cached tokens, its ancestors and itself
struct AttnTreeJob {
    const void *q, *k_new, *v_new, *k_pool, *v_pool;
    const int32_t* block_table;
    const int32_t* cu_nodes;
    const int32_t* parents;
    const int32_t* ctx_lens;
    void* o;
    void* ws;
    int B, Hq, Hkv, D, page, max_pages, n_pages, n_nodes, max_nodes, max_ctx;
    float scale;
};
size_t attn_tree_workspace_bytes(int B, int Hq, int Hkv, int D, int max_nodes, int max_ctx);
cudaError_t launch_attn_tree(const AttnTreeJob& job, cudaStream_t st);

// the layer's output at every node; the pools are not written
struct TreeJob {
    const void *x, *z, *a, *b;
    const void* conv_pool;
    const float* state_pool;
    const int32_t* slot_idx;
    const int32_t* cu_nodes;
    const int32_t* parents;
    void* y;
    int B, n_nodes, max_nodes, n_slots;
};
cudaError_t launch_tree_verify(const Geom& g, const LayerParams& prm, const TreeJob& job, cudaStream_t st);

// rows src_rows[cu_rows[b]] .. of x, a, b (src_rows NULL: those rows themselves) applied to
// slot_idx[b] in place, in order
struct TreeCommitJob {
    const void *x, *a, *b;
    void* conv_pool;
    float* state_pool;
    const int32_t* slot_idx;
    const int32_t* cu_rows;
    const int32_t* src_rows;
    int B, n_rows, n_src, max_rows, n_slots;
};
cudaError_t launch_tree_commit(const Geom& g, const LayerParams& prm, const TreeCommitJob& job, cudaStream_t st);

// pages and row maps from request lengths
struct TablesJob {
    const int32_t *ctx_lens, *new_lens, *free_pages, *head;
    const int32_t *path, *cu_nodes;  // NULL: no source rows
    int32_t *block_table, *cu_rows, *src_rows, *head_out;
    int64_t* slot_map;
    int B, page, n_pages, max_pages, n_free, n_rows, path_len;
};
cudaError_t launch_page_tables(const TablesJob& job, cudaStream_t st);

// K and V rows src_rows[i] (NULL: i) into cache rows slot_map[i]
struct AppendJob {
    const void *k_new, *v_new;
    const int64_t* slot_map;
    const int32_t* src_rows;
    void *k_pool, *v_pool;
    int64_t n_rows, n_src;
    int Hkv, D, page, n_pages;
};
cudaError_t launch_append(const AppendJob& job, cudaStream_t st);

// ---- around the attention and the projections ----
// rotary positions of rows of q and k (out == in: in place); pieces and step_h are the launcher's
struct RopeJob {
    const void *q, *k;
    void *q_out, *k_out;
    int64_t ldq, ldk, ldqo, ldko;  // elements between tokens
    const int32_t* positions;
    int64_t n_tok;
    int hq, hkv, D, rot, half, bf16;
    int pieces, step_h;
    float mscale;
    unsigned long long turns[128];  // turns per position of pair i, in units of 2^-64
};
void rope_turns(int rot, double theta, double factor, int orig_len, double beta_fast, double beta_slow, uint64_t* turns);
cudaError_t launch_rope(RopeJob job, cudaStream_t st);

constexpr int64_t kProjTokens = (int64_t)1 << 22;  // the most tokens of a call of the fused projections

// out[t][n] of few tokens: x_t . w_n, plus (rank > 0) v_t . b_n of the token's adapter; or, with w2,
// silu(x_t . w_n) (x_t . w2_n)
struct FewJob {
    const void *x, *w, *w2;
    void* out;
    int64_t n_tok, ld;
    int32_t n_out, k;
    int early;  // the kernel ahead in the stream is of the same call and its launches follow the rule of `k_few`
    const float* v;              // [n_tok][rank]
    const int32_t* tok_adapter;  // [n_tok], -1: none
    const int32_t *cu_rows, *adapter_idx;  // what tok_adapter was made from
    const void* b;               // [n_adapters][n_out][rank]
    int32_t rank, n_adapters, n_seg;
    int32_t* zero;  // as in WideJob
    int32_t n_zero;
};
cudaError_t launch_few(const FewJob& job, cudaStream_t st);
struct FewPlan {
    int n, ks;      // tokens of a tile, CTAs that share a tile's K
    int64_t us100;  // what the call should take, in hundredths of a microsecond
};
FewPlan few_plan(int64_t n_tok, int32_t n_out, int32_t k, bool gated, int32_t rank);

// Tiles of a launch_wide: `whole` in whole waves over the GPU, the `rest` in `split` parts along K, joined through a
// workspace by whichever part of a tile comes last.
struct WidePlan {
    int64_t whole, rest;
    int32_t split, counters;
    size_t counter_bytes, ws_bytes;
    int64_t us100;  // as in FewPlan
};
// the same of many tokens; out 16-byte aligned, ld a multiple of 8
struct WideJob {
    const void *x, *w, *w2;
    void* out;
    int64_t n_tok, ld;
    int32_t n_out, k;
    const void* v;               // bf16 [n_tok][low_row(rank)]
    const int32_t* tok_adapter;  // [n_tok], -1: none
    const void* b;               // [n_adapters][n_out][rank]
    int32_t rank, n_adapters;
    WidePlan plan;
    void* split_ws;  // plan.ws_bytes, of which the first `counters` int32 are zero
    int32_t* zero;   // counters to set to zero, for a launch_wide behind this one
    int32_t n_zero;
};
cudaError_t launch_wide(const WideJob& job, cudaStream_t st);
// adapters: different ones in a block of 256 tokens, about
WidePlan wide_plan(int64_t n_tok, int32_t n_out, int32_t k, bool gated, int32_t rank, int64_t adapters);
// the most ws_bytes of such plans (not gated) of up to n_tok tokens
size_t wide_ws_most(int64_t n_tok, int32_t n_out, int32_t k);

// Low-rank activations for launch_wide: v = hi + lo in bf16, a row of low_row(rank) elements being [hi | lo] in parts
// of 16 ceil(rank / 16) (rank <= 32) or 64 ceil(rank / 64) elements, each padded with zeros to a multiple of 16.
constexpr int low_row(int rank) { return rank <= 32 ? 64 : 2 * ((rank + 63) / 64 * 64); }

constexpr int kShortRequest = 16;  // tokens from which on the tensor cores make a request's v for launch_wide

// each token's adapter, and v = scale A x, for launch_few (wide 0: fp32 [n_tok][rank]) or launch_wide (wide 1)
struct LowJob {
    const void *x, *a;
    const float* scale;  // NULL: 1
    const int32_t *cu_rows, *adapter_idx;
    void* v;
    int32_t* tok_adapter;  // [n_tok], -1: none
    int64_t n_tok;
    int32_t n_seg, n_adapters, rank, k, wide;
    int32_t* zero;  // as in WideJob
    int32_t n_zero;
};
cudaError_t launch_lora_low(const LowJob& job, cudaStream_t st);

// GDN_DEBUG: device-side check that the na + nb indices of idx_a then idx_b lie in
// [0, n_slots) and are distinct.  A violation ORs kDevBadSlot into the device status
// word.  With wait, the stream is synchronised and the first bad position (or -1)
// and the first repeated pair (or -1, -1) are returned, with the value found at
// the first of them.
cudaError_t check_slots(const int32_t* idx_a, int na, const int32_t* idx_b, int nb, int n_slots, cudaStream_t st,
                        bool wait, long long* bad_range, long long* dup_i, long long* dup_j, int32_t* value);

// read and clear the device status word of each kernel file (synchronous)
cudaError_t take_device_status_decode(unsigned* out);
cudaError_t take_device_status_prefill(unsigned* out);
cudaError_t take_device_status_chunk16(unsigned* out);
cudaError_t take_device_status_proj(unsigned* out);
cudaError_t take_device_status_tree(unsigned* out);
cudaError_t take_device_status_attn_tree(unsigned* out);
cudaError_t take_device_status_few(unsigned* out);
cudaError_t take_device_status_wide(unsigned* out);
cudaError_t take_device_status_lora(unsigned* out);

}  // namespace gdn
