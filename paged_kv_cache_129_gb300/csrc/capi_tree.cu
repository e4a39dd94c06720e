// C-ABI entry points of a speculative step with a drafted tree: argument checks in front of the kernels of tree_ops.h.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "capi_checks.h"
#include "pa.h"
#include "pa_internal.h"
#include "tree_ops.h"

using namespace pa;

namespace {

struct Span {
    const void* p;
    long long bytes;
    int align;
};

// NULL or misaligned buffers, outputs that overlap one another or an input (other than `in_place[i]` of output i); PA_OK or a failure.
int spans(const char* fn, std::initializer_list<Span> outs, std::initializer_list<Span> ins, std::initializer_list<const void*> in_place = {}) {
    for (const auto* list : {&outs, &ins})
        for (const Span& s : *list) {
            if (s.bytes > 0 && !s.p) return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", fn);
            if (!aligned(s.p, (uintptr_t)s.align)) return fail(PA_ERR_INVALID_ARG, "%s: misaligned buffer", fn);
        }
    int i = 0;
    for (const Span& o : outs) {
        const void* same = i < (int)in_place.size() ? in_place.begin()[i] : nullptr;
        for (const Span& in : ins)
            if (!(same && in.p == same && o.p == same) && overlap(o.p, o.bytes, in.p, in.bytes))
                return fail(PA_ERR_INVALID_ARG, "%s: an output overlaps an input", fn);
        for (int j = 0; j < i; ++j)
            if (overlap(o.p, o.bytes, outs.begin()[j].p, outs.begin()[j].bytes))
                return fail(PA_ERR_INVALID_ARG, "%s: outputs overlap one another", fn);
        ++i;
    }
    return PA_OK;
}

int rows_ok(const char* fn, int num_seqs, int num_tokens) {
    if (num_seqs < 0 || num_seqs > kMaxStepSeqs) return fail(PA_ERR_INVALID_ARG, "%s: num_seqs=%d outside [0, %d]", fn, num_seqs, kMaxStepSeqs);
    if (num_tokens < 0 || num_tokens > kMaxStepRows)
        return fail(PA_ERR_INVALID_ARG, "%s: num_tokens=%d outside [0, %d]", fn, num_tokens, kMaxStepRows);
    return PA_OK;
}

// Whether two of the caches of the layers, of `bytes` each, share a byte.
bool caches_overlap(const CachePtrs& caches, int num_layers, unsigned long long bytes) {
    uintptr_t at[2 * kMaxLayers];
    uintptr_t* end = at;
    for (const auto* list : {&caches.key, &caches.value})
        for (int l = 0; l < num_layers; ++l) *end++ = reinterpret_cast<uintptr_t>((*list)[l]);
    if (!std::is_sorted(at, end)) std::sort(at, end);
    for (const uintptr_t* p = at + 1; p < end; ++p)
        if (*p - p[-1] < bytes) return true;
    return false;
}

bool attend_sizes_ok(int num_heads, int num_kv_heads, int head_dim) {
    return num_heads > 0 && num_kv_heads > 0 && num_heads % num_kv_heads == 0 && (head_dim == 64 || head_dim == 128);
}

}  // namespace

extern "C" {

static_assert(PA_MAX_TREE_NODES == kMaxTreeNodes, "the header's limit is the kernels'");

int pa_tree_masks(int32_t* positions, int64_t* tree_mask, const int32_t* parents, const int32_t* context_lens,
                  const int32_t* q_offsets, int num_seqs, int num_tokens, int mask_words, void* stream) {
    CallRange range("pa_tree_masks");
    clear_error();
    int st = rows_ok("pa_tree_masks", num_seqs, num_tokens);
    if (st != PA_OK) return st;
    if (mask_words < 1 || mask_words > kMaxTreeWords)
        return fail(PA_ERR_INVALID_ARG, "pa_tree_masks: mask_words=%d outside [1, %d]", mask_words, kMaxTreeWords);
    if (num_tokens == 0) return PA_OK;
    st = spans("pa_tree_masks", {{positions, 4ll * num_tokens, 4}, {tree_mask, 8ll * num_tokens * mask_words, 8}},
               {{parents, 4ll * num_tokens, 4}, {context_lens, 4ll * num_seqs, 4}, {q_offsets, 4ll * (num_seqs + 1), 4}});
    if (st != PA_OK) return st;
    TreeMaskArgs a{positions, tree_mask, parents, context_lens, q_offsets, num_seqs, num_tokens, mask_words, nullptr};
    int sms = 0;
    st = device_state(&a.err, &sms);
    if (st != PA_OK) return st;
    const cudaError_t e = tree_masks_launch(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : launch_failed(e, "pa_tree_masks");
}

int pa_accept_tree(int32_t* accepted, int32_t* num_accepted, void* next_tokens, const int32_t* parents, const void* tokens,
                   const void* choices, const int32_t* q_offsets, int num_seqs, int num_tokens, int max_accepted, int token_bytes,
                   void* stream) {
    CallRange range("pa_accept_tree");
    clear_error();
    int st = rows_ok("pa_accept_tree", num_seqs, num_tokens);
    if (st != PA_OK) return st;
    if (max_accepted < 1 || max_accepted > kMaxTreeNodes)
        return fail(PA_ERR_INVALID_ARG, "pa_accept_tree: max_accepted=%d outside [1, %d]", max_accepted, kMaxTreeNodes);
    if (token_bytes != 4 && token_bytes != 8) return fail(PA_ERR_INVALID_ARG, "pa_accept_tree: token_bytes=%d must be 4 or 8", token_bytes);
    if (num_seqs == 0) return PA_OK;
    const long long tb = token_bytes;
    st = spans("pa_accept_tree", {{accepted, 4ll * num_seqs * max_accepted, 4}, {num_accepted, 4ll * num_seqs, 4}, {next_tokens, tb * num_seqs, token_bytes}},
               {{parents, 4ll * num_tokens, 4}, {tokens, tb * num_tokens, token_bytes}, {choices, tb * num_tokens, token_bytes},
                {q_offsets, 4ll * (num_seqs + 1), 4}});
    if (st != PA_OK) return st;
    AcceptArgs a{accepted, num_accepted, next_tokens, parents, tokens, choices, q_offsets, num_seqs, num_tokens, max_accepted, token_bytes, nullptr};
    int sms = 0;
    st = device_state(&a.err, &sms);
    if (st != PA_OK) return st;
    const cudaError_t e = accept_tree_launch(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : launch_failed(e, "pa_accept_tree");
}

int pa_compact_tree(void* const* key_caches, void* const* value_caches, int num_layers, const int64_t* slot_mapping,
                    const int32_t* q_offsets, const int32_t* accepted, const int32_t* num_accepted, const int32_t* block_tables,
                    const int32_t* context_lens, int32_t* free_blocks, const int32_t* num_free, int32_t* context_lens_out,
                    int32_t* num_free_out, int num_seqs, int num_tokens, int max_accepted, int num_kv_heads, int head_dim,
                    int block_size, int max_blocks_per_seq, int num_blocks, int dtype, void* stream) {
    CallRange range("pa_compact_tree");
    clear_error();
    if (dtype != PA_F32 && dtype != PA_F16 && dtype != PA_BF16)
        return fail(PA_ERR_INVALID_ARG, "pa_compact_tree: dtype %d (an FP8 cache has scales by block: its codes cannot move alone)", dtype);
    if (num_layers < 1 || num_layers > PA_MAX_LAYERS)
        return fail(PA_ERR_INVALID_ARG, "pa_compact_tree: num_layers=%d outside [1, %d]", num_layers, PA_MAX_LAYERS);
    int st = rows_ok("pa_compact_tree", num_seqs, num_tokens);
    if (st != PA_OK) return st;
    if (max_accepted < 1 || max_accepted > kMaxTreeNodes)
        return fail(PA_ERR_INVALID_ARG, "pa_compact_tree: max_accepted=%d outside [1, %d]", max_accepted, kMaxTreeNodes);
    if (num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 || num_blocks > kMaxStepRows)
        return fail(PA_ERR_INVALID_ARG, "pa_compact_tree: bad sizes");
    const int eb = bytes_of(dtype);
    if (!fits_int((long long)max_blocks_per_seq * block_size) || !fits_int((long long)num_kv_heads * head_dim * eb * num_layers * 2))
        return fail(PA_ERR_INVALID_ARG, "pa_compact_tree: max_blocks_per_seq * block_size and a token's bytes in all layers must be < 2^31");
    if (!key_caches || !value_caches) return fail(PA_ERR_INVALID_ARG, "pa_compact_tree: NULL pointer array");
    const long long b = num_seqs;
    st = spans("pa_compact_tree", {{context_lens_out, 4 * b, 4}, {num_free_out, 4, 4}, {free_blocks, 4ll * num_blocks, 4}},
               {{slot_mapping, 8ll * num_tokens, 8}, {q_offsets, 4 * (b + 1), 4}, {accepted, 4 * b * max_accepted, 4}, {num_accepted, 4 * b, 4},
                {block_tables, 4 * b * max_blocks_per_seq, 4}, {context_lens, 4 * b, 4}, {num_free, 4, 4}},
               {context_lens, num_free});
    if (st != PA_OK) return st;
    CachePtrs caches{};
    const int row_bytes = head_dim * eb;
    bool vector = row_bytes % 16 == 0;
    for (int l = 0; l < num_layers; ++l) {
        if (!key_caches[l] || !value_caches[l]) return fail(PA_ERR_INVALID_ARG, "pa_compact_tree: NULL pointer for layer %d", l);
        if (!aligned(key_caches[l], eb) || !aligned(value_caches[l], eb))
            return fail(PA_ERR_INVALID_ARG, "pa_compact_tree: layer %d caches not aligned to the element size", l);
        vector = vector && aligned(key_caches[l], 16) && aligned(value_caches[l], 16);
        caches.key[l] = static_cast<char*>(key_caches[l]);
        caches.value[l] = static_cast<char*>(value_caches[l]);
    }
    if (caches_overlap(caches, num_layers, (unsigned long long)num_blocks * block_size * num_kv_heads * row_bytes))
        return fail(PA_ERR_INVALID_ARG, "pa_compact_tree: caches overlap (each is listed once: a cache compacted twice loses rows)");
    CompactArgs a{slot_mapping, q_offsets, accepted, num_accepted, block_tables, context_lens, free_blocks, num_free, context_lens_out,
                  num_free_out, num_layers, num_seqs, num_tokens, max_accepted, num_kv_heads, row_bytes, block_size, max_blocks_per_seq,
                  num_blocks, vector ? 1 : 0, eb, 0, nullptr};
    st = device_state(&a.err, &a.num_sms);
    if (st != PA_OK) return st;
    const cudaError_t e = compact_tree_launch(a, caches, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : launch_failed(e, "pa_compact_tree");
}

int pa_attend_tree(void* out, const void* query, const void* key_cache, const void* value_cache, const int64_t* tree_mask,
                   const int32_t* block_tables, const int32_t* context_lens, const int32_t* q_offsets, int num_seqs, int num_tokens,
                   int num_heads, int num_kv_heads, int head_dim, int block_size, int max_blocks_per_seq, int num_blocks,
                   int mask_words, float scale, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    CallRange range("pa_attend_tree");
    clear_error();
    if (dtype != PA_F16 && dtype != PA_BF16) return fail(PA_ERR_UNSUPPORTED, "pa_attend_tree: queries and caches are f16 or bf16");
    if (num_seqs < 0 || num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0)
        return fail(PA_ERR_INVALID_ARG, "pa_attend_tree: bad sizes");
    if (num_heads % num_kv_heads != 0)
        return fail(PA_ERR_INVALID_ARG, "pa_attend_tree: num_heads=%d must be a multiple of num_kv_heads=%d", num_heads, num_kv_heads);
    if (!attend_sizes_ok(num_heads, num_kv_heads, head_dim) || (block_size != 16 && block_size != 32))
        return fail(PA_ERR_UNSUPPORTED, "pa_attend_tree: compiled for head_dim 64 and 128, block_size 16 and 32 (head_dim=%d block_size=%d)",
                    head_dim, block_size);
    if (mask_words < 1 || mask_words > kMaxTreeWords)
        return fail(PA_ERR_INVALID_ARG, "pa_attend_tree: mask_words=%d outside [1, %d]", mask_words, kMaxTreeWords);
    if (!fits_int((long long)max_blocks_per_seq * block_size + 1024) || !fits_int((long long)num_blocks * num_kv_heads * block_size) ||
        !fits_int((long long)num_tokens * num_heads))
        return fail(PA_ERR_INVALID_ARG, "pa_attend_tree: max_blocks_per_seq * block_size + 1024, num_blocks * num_kv_heads * block_size "
                                        "and num_tokens * num_heads must be < 2^31");
    if (num_seqs > kMaxStepSeqs) return fail(PA_ERR_UNSUPPORTED, "pa_attend_tree: num_seqs=%d > %d", num_seqs, kMaxStepSeqs);
    if (!std::isfinite(scale)) return fail(PA_ERR_INVALID_ARG, "pa_attend_tree: scale is not finite");
    if (num_tokens == 0 || num_seqs == 0) return PA_OK;
    const long long q_bytes = 2ll * num_tokens * num_heads * head_dim, pool = 2ll * num_blocks * num_kv_heads * block_size * head_dim;
    int st = spans("pa_attend_tree", {{out, q_bytes, 16}},
                   {{query, q_bytes, 16}, {key_cache, pool, 16}, {value_cache, pool, 16}, {tree_mask, 8ll * num_tokens * mask_words, 8},
                    {block_tables, 4ll * num_seqs * max_blocks_per_seq, 4}, {context_lens, 4ll * num_seqs, 4},
                    {q_offsets, 4ll * (num_seqs + 1), 4}});
    if (st != PA_OK) return st;
    TreeAttendArgs a{out, query, key_cache, value_cache, tree_mask, block_tables, context_lens, q_offsets, num_seqs, num_tokens, num_heads,
                     num_kv_heads, head_dim, block_size, max_blocks_per_seq, num_blocks, mask_words, dtype, num_heads / num_kv_heads, scale,
                     workspace, 0, nullptr};
    st = device_state(&a.err, &a.num_sms);
    if (st != PA_OK) return st;
    const size_t need = attend_tree_workspace_bytes(a.num_sms, head_dim);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return fail(PA_ERR_INVALID_ARG, "pa_attend_tree: needs a 256-byte aligned workspace of %zu bytes (%zu given)", need,
                    workspace ? workspace_bytes : (size_t)0);
    const long long groups = (long long)num_blocks * num_kv_heads * (block_size / 8);
    CUtensorMap kmap, vmap;
    st = group_map(&kmap, key_cache, groups, block_size, head_dim);
    if (st == PA_OK) st = group_map(&vmap, value_cache, groups, block_size, head_dim);
    if (st != PA_OK) return st;
    const cudaError_t e = attend_tree_launch(a, kmap, vmap, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : launch_failed(e, "pa_attend_tree");
}

size_t pa_attend_tree_workspace_size(int num_tokens, int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                                     int max_blocks_per_seq, int dtype) {
    clear_error();
    if ((dtype != PA_F16 && dtype != PA_BF16) || num_tokens < 0 || num_seqs < 0 || !attend_sizes_ok(num_heads, num_kv_heads, head_dim) ||
        block_size <= 0 || max_blocks_per_seq <= 0)
        return 0;
    unsigned* err = nullptr;
    int sms = 0;
    if (device_state(&err, &sms) != PA_OK) return 0;
    return attend_tree_workspace_bytes(sms, head_dim);
}

}  // extern "C"
