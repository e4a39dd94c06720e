// Launchers of the kernels of a serving step: block tables and slot maps from request lengths,
// rotary positions with the paged write, causal attention of ragged runs over FP8 caches.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

namespace pa {

constexpr int kMaxStepSeqs = 8192;  // requests of one call
constexpr int kMaxStepRows = 0x7fff0000;  // tokens or blocks of one call: int counters go past them by a grid's step

struct AdvanceArgs {
    int32_t* block_tables;        // [num_seqs, max_blocks], new entries written
    const int32_t* context_lens;  // [num_seqs]
    const int32_t* new_lens;      // [num_seqs]; < 0: the request gives its blocks back
    int32_t* free_blocks;         // [num_blocks], a stack of *num_free ids
    const int32_t* num_free;
    int32_t* context_lens_out;  // may be context_lens
    int32_t* num_free_out;      // may be num_free
    int32_t* q_offsets;         // [num_seqs + 1]
    int32_t* positions;         // [num_tokens]
    int64_t* slot_mapping;      // [num_tokens]
    int num_seqs, max_blocks, num_blocks, block_size, num_tokens;
    unsigned* err;
};

// Rotary rows and their destinations.  Strides are in elements, between tokens; heads of a token are contiguous.
struct RopeArgs {
    void* query_out;  // [num_tokens, num_heads, head_dim], contiguous
    const void* query;
    const void* key;
    const void* value;
    long long q_stride, k_stride, v_stride;
    const double* inv_freq;  // [rotary_dim / 2]
    int rotary_dim, interleaved;
    float factor;
    int num_tokens, num_heads, num_kv_heads, head_dim, block_size, num_blocks, dtype;
    unsigned* err;
};

struct RopeWriteArgs {
    RopeArgs r;
    void* key_cache;
    void* value_cache;
    const int32_t* positions;
    const int64_t* slot_mapping;
    int num_sms;
};

struct RopeAppendArgs {
    RopeArgs r;
    uint8_t* key_cache;
    uint8_t* value_cache;  // nullptr: K and V records in key_cache
    float* k_scale;
    float* v_scale;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* q_offsets;
    int num_seqs, max_blocks;
    int num_sms;
};

struct AttendArgs {
    void* out;
    const void* query;
    const uint8_t* key_cache;
    const uint8_t* value_cache;  // nullptr: K and V records in key_cache
    const float* k_scale;
    const float* v_scale;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* q_offsets;
    int num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, block_size, max_blocks, num_blocks, dtype;
    float scale;
    void* workspace;
    int num_sms;
    unsigned* err;
};

cudaError_t advance_tables_launch(const AdvanceArgs& a, cudaStream_t stream);
cudaError_t rope_write_kv_launch(const RopeWriteArgs& a, cudaStream_t stream);
cudaError_t rope_append_fp8_launch(const RopeAppendArgs& a, cudaStream_t stream);
// Scratch of one attend_fp8 call.
size_t attend_fp8_workspace_bytes(int num_sms, int num_seqs, int num_tokens, int num_heads, int num_kv_heads, int head_dim,
                                  int block_size, int max_blocks);
// kmap, vmap: record_map()s of K and V.
cudaError_t attend_fp8_launch(const AttendArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t stream);

// A cache as rows of record_bytes (K or V of one block and kv head), for gathers of rows in parts of at most 2 KB.  PA_OK or a failure
// with its message.
int record_map(CUtensorMap* map, const void* base, long long records, int record_bytes);

}  // namespace pa
