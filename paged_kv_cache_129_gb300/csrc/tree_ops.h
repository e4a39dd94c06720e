// Launchers of the kernels of a speculative step with a drafted tree over a paged 16 / 32-bit cache.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "kv_ops.h"
#include "step_ops.h"

namespace pa {

constexpr int kMaxTreeNodes = 1024;  // of one request
constexpr int kMaxTreeWords = kMaxTreeNodes / 64;

struct TreeMaskArgs {
    int32_t* positions;  // [num_tokens]
    int64_t* tree_mask;  // [num_tokens, mask_words]
    const int32_t* parents;
    const int32_t* context_lens;
    const int32_t* q_offsets;
    int num_seqs, num_tokens, mask_words;
    unsigned* err;
};

struct AcceptArgs {
    int32_t* accepted;      // [num_seqs, max_accepted]
    int32_t* num_accepted;  // [num_seqs]
    void* next_tokens;      // [num_seqs], of token_bytes
    const int32_t* parents;
    const void* tokens;
    const void* choices;
    const int32_t* q_offsets;
    int num_seqs, num_tokens, max_accepted, token_bytes;
    unsigned* err;
};

// Caches of the layers, passed by value as a kernel argument.
struct CachePtrs {
    char* key[kMaxLayers];
    char* value[kMaxLayers];
};

struct CompactArgs {
    const int64_t* slot_mapping;  // [num_tokens]
    const int32_t* q_offsets;
    const int32_t* accepted;      // [num_seqs, max_accepted]
    const int32_t* num_accepted;  // [num_seqs]
    const int32_t* block_tables;
    const int32_t* context_lens;
    int32_t* free_blocks;
    const int32_t* num_free;
    int32_t* context_lens_out;  // may be context_lens
    int32_t* num_free_out;      // may be num_free
    int num_layers, num_seqs, num_tokens, max_accepted, num_kv_heads, row_bytes, block_size, max_blocks, num_blocks;
    int vector;  // rows and caches are multiples of 16 bytes
    int elem_bytes;
    int num_sms;
    unsigned* err;
};

struct NormRopeArgs {
    RopeArgs r;
    void* key_cache;
    void* value_cache;
    const int32_t* positions;
    const int64_t* slot_mapping;
    const void* q_weight;  // [head_dim], or nullptr: ones
    const void* k_weight;
    int weight_dtype;
    float weight_offset, eps;
    int num_sms;
};

struct TreeAttendArgs {
    void* out;
    const void* query;
    const void* key_cache;
    const void* value_cache;
    const int64_t* tree_mask;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* q_offsets;
    int num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, block_size, max_blocks, num_blocks, mask_words, dtype;
    int group;  // query heads of a kv head
    float scale;
    void* workspace;
    int num_sms;
    unsigned* err;
};

cudaError_t tree_masks_launch(const TreeMaskArgs& a, cudaStream_t stream);
cudaError_t accept_tree_launch(const AcceptArgs& a, cudaStream_t stream);
cudaError_t compact_tree_launch(const CompactArgs& a, const CachePtrs& caches, cudaStream_t stream);
cudaError_t norm_rope_write_kv_launch(const NormRopeArgs& a, cudaStream_t stream);
// Scratch of one attend_tree call.
size_t attend_tree_workspace_bytes(int num_sms, int head_dim);
// kmap, vmap: group_map()s of K and V.
cudaError_t attend_tree_launch(const TreeAttendArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t stream);

// A 16-bit cache as groups of eight rows, in panels of 64 elements: what one copy brings of a block (of a kv head) is a box of
// block_size / 8 groups, each panel with the 128-byte swizzle.  PA_OK or a failure with its message.
int group_map(CUtensorMap* map, const void* base, long long groups, int block_size, int head_dim);

}  // namespace pa
