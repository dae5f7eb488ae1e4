// Internal launchers of the paged 8-bit key/value cache and of the
// block-scaled FP8 product (host side, not part of the C ABI).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace q8 {

// The paged cache and one batch of sequences over it (include/q8.h,
// q8_kv_append): device pointers, sizes checked on the host.
struct KvView {
  uint8_t* k;              // [num_pages, kv_heads, page, dim] e4m3 codes
  uint8_t* v;              // [num_pages, kv_heads, dim, page] e4m3 codes
  uint8_t* ke;             // [num_pages, kv_heads] exponent bytes
  uint8_t* ve;
  const int32_t* q_start;  // [seqs + 1]
  const int32_t* kv_len;   // [seqs]
  const int32_t* table;    // [seqs, max_pages]
  int num_pages, kv_heads, seqs, max_pages, page, tokens;
};

struct AppendArgs {
  KvView kv;
  const void *q, *k, *v;           // [tokens, heads, dim] with token strides (elements); q may be null
  int64_t q_stride, k_stride, v_stride;
  void* q_out;                     // [tokens, heads, dim] dense
  int heads;
  const float *cos, *sin;          // [positions, rot / 2]
  int positions, rot, interleaved;
  int reach;                       // grid extent over the pages one sequence's new tokens touch (the launcher's)
  int max_q;
  // with norms (launch_kv_append_norm): weights [dim] of type w_dt, null where a side has none; each
  // token's position for the rotation, null for its slot's
  const void *qw, *kw;
  const int32_t* pos;
  float eps;
  int w_dt;
};
hipError_t launch_kv_append(const AppendArgs& a, int dt, int dim, hipStream_t st);
hipError_t launch_kv_append_norm(const AppendArgs& a, int dt, int dim, hipStream_t st);

struct AttnArgs {
  KvView kv;
  const void* q;                   // [tokens, heads, dim]
  int64_t q_stride;
  void* out;                       // [tokens, heads, dim] dense
  float* lse;                      // [tokens, heads] or null
  int heads, causal, window;
  int max_q;
  int64_t max_kv;
  float scale_log2;                // softmax scale times log2(e)
  float *part, *part_ml;           // [splits, tokens * heads, dim], [splits, tokens * heads, 2] (trees: 3)
  const uint64_t* mask;            // drafted trees: [tokens, words]
  int words;
  const int32_t* pos;              // [tokens] or null
};
// Splits of the key axis for this shape (1: no workspace, one launch).
int attn_splits(int heads, int kv_heads, int dim, int seqs, int64_t max_q, int64_t max_kv, int window);
hipError_t launch_attention(const AttnArgs& a, int dt, int dim, hipStream_t st);
int tree_splits(int heads, int kv_heads, int dim, int seqs, int64_t max_q, int64_t max_kv, int window);
hipError_t launch_attention_tree(const AttnArgs& a, int dt, int dim, hipStream_t st);

// One layer's cache, as a KvView has it.
struct CacheLayer {
  uint8_t *k, *v, *ke, *ve;
};
constexpr int kLayers = 64;        // of one launch (their pointers are kernel arguments)

// Kept drafts to the front of their slots (kv_pages.hip); kv: the batch, its cache pointers unused.
struct CompactArgs {
  KvView kv;
  const int32_t* keep;             // [seqs, width]
  const int32_t* n_keep;           // [seqs]
  int32_t* len_out;                // [seqs]; null: not written
  int width;
  CacheLayer layer[kLayers];
};
hipError_t launch_kv_compact(const CompactArgs& a, int dim, int layers, hipStream_t st);

struct ForkArgs {
  const int32_t *table, *kv_len, *refs, *parent;     // [seqs, max_pages], [seqs], [num_pages], [outs]
  int32_t *table_out, *len_out, *refs_out, *missing;
  // workspace: first row of each sequence [seqs], new pages of a row and those before it [outs], the pages
  // taken [num_pages], (source, target) of each row's copy [outs]
  int32_t *first, *fresh, *taken, *copies;
  int64_t room, page_bytes;        // of a page's keys
  int seqs, outs, max_pages, num_pages, page, kv_heads;
  CacheLayer layer[kLayers];
};
hipError_t launch_kv_fork(const ForkArgs& a, hipStream_t st);                          // the tables
hipError_t launch_copy_pages(const ForkArgs& a, int layers, hipStream_t st);           // then the pages

// Block-scaled FP8 (fp8_block.hip): activations [M, K] in groups of 128 along
// K with x_scale [ceil(K / 128), M], weights in 128 x 128 blocks with w_scale
// [ceil(N / 128), ceil(K / 128)].
constexpr int kScaleBlock = 128;
hipError_t launch_quant_weight_block(const void* w, int dt, int64_t N, int64_t K, uint8_t* wq, float* w_scale,
                                     hipStream_t st);
hipError_t launch_quant_act_block(const void* x, int dt, int64_t M, int64_t K, uint8_t* xq, float* x_scale,
                                  hipStream_t st);
hipError_t launch_gemm_fp8_block(const uint8_t* xq, const float* x_scale, int64_t M, int64_t K, const uint8_t* wq,
                                 const float* w_scale, int64_t N, const float* bias, void* y, int ydt, hipStream_t st);
// Decode-shaped, with the activation quantization in the same launch, for the few tokens where
// fp8_block_is_fused.
bool fp8_block_is_fused(int64_t M);
hipError_t launch_gemv_fp8_block(const void* x, int xdt, int64_t M, int64_t K, const uint8_t* wq, const float* w_scale,
                                 int64_t N, const float* bias, void* y, int ydt, hipStream_t st);

}  // namespace q8
