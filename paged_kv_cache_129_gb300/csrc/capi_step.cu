// C-ABI entry points of a serving step: argument checks in front of the kernels of step_ops.h.
#include <cmath>
#include <cstdint>

#include <nvtx3/nvToolsExt.h>

#include "pa.h"
#include "pa_internal.h"
#include "step_ops.h"

using namespace pa;

namespace {

struct CallRange {
    explicit CallRange(const char* name) { nvtxRangePushA(name); }
    ~CallRange() { nvtxRangePop(); }
    CallRange(const CallRange&) = delete;
    CallRange& operator=(const CallRange&) = delete;
};

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool fits_int(long long x) { return x < (1ll << 31); }
int bytes_of(int dtype) { return dtype == PA_F32 ? 4 : 2; }

// Whether [p, p + n) and [q, q + m) share a byte.
bool overlap(const void* p, long long n, const void* q, long long m) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return n > 0 && m > 0 && a < b + (uintptr_t)m && b < a + (uintptr_t)n;
}

int launch_failed(cudaError_t e, const char* what) {
    return fail(PA_ERR_CUDA, "%s launch: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

// Checks shared by the two rotary entry points; fills what they share.
int rope_args(const char* fn, RopeArgs* r, void* query_out, const void* query, const void* key, const void* value,
              int64_t q_stride, int64_t k_stride, int64_t v_stride, const double* inv_freq, int rotary_dim, int layout,
              float factor, int num_tokens, int num_heads, int num_kv_heads, int head_dim, int block_size, int num_blocks,
              int dtype) {
    if (dtype != PA_F32 && dtype != PA_F16 && dtype != PA_BF16) return fail(PA_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, dtype);
    if (num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0)
        return fail(PA_ERR_INVALID_ARG, "%s: bad sizes", fn);
    if (num_tokens > kMaxStepRows) return fail(PA_ERR_INVALID_ARG, "%s: num_tokens=%d > %d", fn, num_tokens, kMaxStepRows);
    if (layout != PA_ROPE_HALF && layout != PA_ROPE_INTERLEAVED)
        return fail(PA_ERR_INVALID_ARG, "%s: unknown layout %d", fn, layout);
    if (!std::isfinite(factor)) return fail(PA_ERR_INVALID_ARG, "%s: factor is not finite", fn);
    if (rotary_dim < 0 || rotary_dim > head_dim || rotary_dim % 2 != 0 || head_dim % 2 != 0)
        return fail(PA_ERR_INVALID_ARG, "%s: rotary_dim=%d must be even and at most head_dim=%d (even)", fn, rotary_dim, head_dim);
    if (num_tokens == 0) return PA_OK;
    if (!query_out || !query || !key || !value || (rotary_dim > 0 && !inv_freq))
        return fail(PA_ERR_INVALID_ARG, "%s: NULL pointer", fn);
    const long long row_q = (long long)num_heads * head_dim, row_kv = (long long)num_kv_heads * head_dim;
    if (!fits_int(row_q) || !fits_int(row_kv)) return fail(PA_ERR_INVALID_ARG, "%s: a token's row is too long", fn);
    if (q_stride < row_q || k_stride < row_kv || v_stride < row_kv)
        return fail(PA_ERR_INVALID_ARG, "%s: a token stride is smaller than the token's heads", fn);
    if (query_out == query && q_stride != row_q)
        return fail(PA_ERR_INVALID_ARG, "%s: in place, the query rows must be contiguous", fn);
    const int eb = bytes_of(dtype);
    if (!aligned(query_out, eb) || !aligned(query, eb) || !aligned(key, eb) || !aligned(value, eb) || !aligned(inv_freq, 8))
        return fail(PA_ERR_INVALID_ARG, "%s: buffers must be aligned to the element size", fn);
    const long long n = num_tokens;
    if ((query_out != query && overlap(query_out, n * row_q * eb, query, ((n - 1) * q_stride + row_q) * eb)) ||
        overlap(query_out, n * row_q * eb, key, ((n - 1) * k_stride + row_kv) * eb) ||
        overlap(query_out, n * row_q * eb, value, ((n - 1) * v_stride + row_kv) * eb))
        return fail(PA_ERR_INVALID_ARG, "%s: query_out overlaps the inputs (it may be a contiguous query itself)", fn);
    r->query_out = query_out;
    r->query = query;
    r->key = key;
    r->value = value;
    r->q_stride = q_stride;
    r->k_stride = k_stride;
    r->v_stride = v_stride;
    r->inv_freq = inv_freq;
    r->rotary_dim = rotary_dim;
    r->interleaved = layout == PA_ROPE_INTERLEAVED ? 1 : 0;
    r->factor = factor;
    r->num_tokens = num_tokens;
    r->num_heads = num_heads;
    r->num_kv_heads = num_kv_heads;
    r->head_dim = head_dim;
    r->block_size = block_size;
    r->num_blocks = num_blocks;
    r->dtype = dtype;
    return PA_OK;
}

}  // namespace

extern "C" {

static_assert(PA_MAX_STEP_SEQS == kMaxStepSeqs && PA_MAX_STEP_ROWS == kMaxStepRows, "the header's limits are the kernels'");

int pa_advance_tables(int32_t* block_tables, const int32_t* context_lens, const int32_t* new_lens, int32_t* free_blocks,
                      const int32_t* num_free, int32_t* context_lens_out, int32_t* num_free_out, int32_t* q_offsets,
                      int32_t* positions, int64_t* slot_mapping, int num_seqs, int max_blocks_per_seq, int num_blocks,
                      int block_size, int num_tokens, void* stream) {
    CallRange range("pa_advance_tables");
    clear_error();
    if (num_seqs < 0 || num_seqs > kMaxStepSeqs)
        return fail(PA_ERR_INVALID_ARG, "pa_advance_tables: num_seqs=%d outside [0, %d]", num_seqs, kMaxStepSeqs);
    if (max_blocks_per_seq <= 0 || num_blocks <= 0 || block_size <= 0 || num_tokens < 0)
        return fail(PA_ERR_INVALID_ARG, "pa_advance_tables: bad sizes");
    if (num_tokens > kMaxStepRows || num_blocks > kMaxStepRows)
        return fail(PA_ERR_INVALID_ARG, "pa_advance_tables: num_tokens=%d or num_blocks=%d > %d", num_tokens, num_blocks, kMaxStepRows);
    if (!fits_int((long long)max_blocks_per_seq * block_size))
        return fail(PA_ERR_INVALID_ARG, "pa_advance_tables: max_blocks_per_seq * block_size must be < 2^31");
    if (!num_free || !num_free_out || !q_offsets || !free_blocks || (num_tokens > 0 && (!positions || !slot_mapping)) ||
        (num_seqs > 0 && (!block_tables || !context_lens || !new_lens || !context_lens_out)))
        return fail(PA_ERR_INVALID_ARG, "pa_advance_tables: NULL pointer");
    if (!aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(new_lens, 4) || !aligned(free_blocks, 4) ||
        !aligned(num_free, 4) || !aligned(context_lens_out, 4) || !aligned(num_free_out, 4) || !aligned(q_offsets, 4) ||
        !aligned(positions, 4) || !aligned(slot_mapping, 8))
        return fail(PA_ERR_INVALID_ARG, "pa_advance_tables: misaligned buffer");
    const struct {
        const void* p;
        long long n;
    } outs[] = {{context_lens_out, 4ll * num_seqs}, {num_free_out, 4}, {q_offsets, 4ll * (num_seqs + 1)},
                {positions, 4ll * num_tokens}, {slot_mapping, 8ll * num_tokens}},
      ins[] = {{block_tables, 4ll * num_seqs * max_blocks_per_seq}, {new_lens, 4ll * num_seqs}, {free_blocks, 4ll * num_blocks},
               {context_lens, 4ll * num_seqs}, {num_free, 4}};
    for (int i = 0; i < 5; ++i) {
        for (int j = 0; j < 5; ++j) {
            const bool in_place = ((i == 0 && j == 3) || (i == 1 && j == 4)) && outs[i].p == ins[j].p;
            if (!in_place && overlap(outs[i].p, outs[i].n, ins[j].p, ins[j].n))
                return fail(PA_ERR_INVALID_ARG, "pa_advance_tables: an output overlaps an input (lengths and count may be in place)");
        }
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
                return fail(PA_ERR_INVALID_ARG, "pa_advance_tables: outputs overlap one another");
    }
    AdvanceArgs a{block_tables, context_lens, new_lens, free_blocks, num_free, context_lens_out, num_free_out, q_offsets,
                  positions, slot_mapping, num_seqs, max_blocks_per_seq, num_blocks, block_size, num_tokens, nullptr};
    int sms = 0;
    const int st = device_state(&a.err, &sms);
    if (st != PA_OK) return st;
    const cudaError_t e = advance_tables_launch(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : launch_failed(e, "pa_advance_tables");
}

int pa_rope_write_kv(void* query_out, const void* query, const void* key, const void* value, void* key_cache,
                     void* value_cache, const double* inv_freq, const int32_t* positions, const int64_t* slot_mapping,
                     int64_t q_stride, int64_t k_stride, int64_t v_stride, int num_tokens, int num_heads, int num_kv_heads,
                     int head_dim, int rotary_dim, int layout, float factor, int block_size, int num_blocks, int dtype,
                     void* stream) {
    CallRange range("pa_rope_write_kv");
    clear_error();
    RopeWriteArgs a{};
    int st = rope_args("pa_rope_write_kv", &a.r, query_out, query, key, value, q_stride, k_stride, v_stride, inv_freq,
                       rotary_dim, layout, factor, num_tokens, num_heads, num_kv_heads, head_dim, block_size, num_blocks, dtype);
    if (st != PA_OK) return st;
    if (head_dim > 512) return fail(PA_ERR_UNSUPPORTED, "pa_rope_write_kv: head_dim=%d > 512", head_dim);
    if (num_tokens == 0) return PA_OK;
    if (!key_cache || !value_cache || !positions || !slot_mapping)
        return fail(PA_ERR_INVALID_ARG, "pa_rope_write_kv: NULL pointer");
    const int eb = bytes_of(dtype);
    if (!aligned(key_cache, eb) || !aligned(value_cache, eb) || !aligned(positions, 4) || !aligned(slot_mapping, 8))
        return fail(PA_ERR_INVALID_ARG, "pa_rope_write_kv: misaligned buffer");
    a.key_cache = key_cache;
    a.value_cache = value_cache;
    a.positions = positions;
    a.slot_mapping = slot_mapping;
    st = device_state(&a.r.err, &a.num_sms);
    if (st != PA_OK) return st;
    const cudaError_t e = rope_write_kv_launch(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : launch_failed(e, "pa_rope_write_kv");
}

int pa_rope_append_fp8(void* query_out, const void* query, const void* key, const void* value, void* key_cache,
                       void* value_cache, float* k_scale, float* v_scale, const double* inv_freq,
                       const int32_t* block_tables, const int32_t* context_lens, const int32_t* q_offsets,
                       int64_t q_stride, int64_t k_stride, int64_t v_stride, int num_seqs, int num_tokens, int num_heads,
                       int num_kv_heads, int head_dim, int rotary_dim, int layout, float factor, int block_size,
                       int max_blocks_per_seq, int num_blocks, int dtype, void* stream) {
    CallRange range("pa_rope_append_fp8");
    clear_error();
    RopeAppendArgs a{};
    int st = rope_args("pa_rope_append_fp8", &a.r, query_out, query, key, value, q_stride, k_stride, v_stride, inv_freq,
                       rotary_dim, layout, factor, num_tokens, num_heads, num_kv_heads, head_dim, block_size, num_blocks, dtype);
    if (st != PA_OK) return st;
    if (num_seqs < 0 || max_blocks_per_seq <= 0 || !fits_int((long long)max_blocks_per_seq * block_size))
        return fail(PA_ERR_INVALID_ARG, "pa_rope_append_fp8: num_seqs=%d max_blocks_per_seq=%d", num_seqs, max_blocks_per_seq);
    if ((head_dim != 64 && head_dim != 128) || (block_size != 16 && block_size != 32) || rotary_dim % 4 != 0)
        return fail(PA_ERR_UNSUPPORTED,
                    "pa_rope_append_fp8: compiled for head_dim 64 and 128, block_size 16 and 32, rotary_dim a multiple of 4 "
                    "(head_dim=%d block_size=%d rotary_dim=%d)",
                    head_dim, block_size, rotary_dim);
    if (num_tokens == 0 || num_seqs == 0) return PA_OK;
    if (!fits_int((long long)num_tokens * num_kv_heads * 2))
        return fail(PA_ERR_UNSUPPORTED, "pa_rope_append_fp8: num_tokens * num_kv_heads must be < 2^30");
    if (!key_cache || !k_scale || !v_scale || !block_tables || !context_lens || !q_offsets)
        return fail(PA_ERR_INVALID_ARG, "pa_rope_append_fp8: NULL pointer");
    if (!aligned(key_cache, 16) || !aligned(value_cache, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4) ||
        !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(q_offsets, 4))
        return fail(PA_ERR_INVALID_ARG, "pa_rope_append_fp8: misaligned buffer (caches: 16 bytes)");
    a.key_cache = static_cast<uint8_t*>(key_cache);
    a.value_cache = static_cast<uint8_t*>(value_cache);
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.q_offsets = q_offsets;
    a.num_seqs = num_seqs;
    a.max_blocks = max_blocks_per_seq;
    st = device_state(&a.r.err, &a.num_sms);
    if (st != PA_OK) return st;
    const cudaError_t e = rope_append_fp8_launch(a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : launch_failed(e, "pa_rope_append_fp8");
}

int pa_attend_fp8(void* out, const void* query, const void* key_cache, const void* value_cache, const float* k_scale,
                  const float* v_scale, const int32_t* block_tables, const int32_t* context_lens, const int32_t* q_offsets,
                  int num_seqs, int num_tokens, int num_heads, int num_kv_heads, int head_dim, int block_size,
                  int max_blocks_per_seq, int num_blocks, float scale, int dtype, void* workspace, size_t workspace_bytes,
                  void* stream) {
    CallRange range("pa_attend_fp8");
    clear_error();
    if (dtype != PA_F16 && dtype != PA_BF16) return fail(PA_ERR_UNSUPPORTED, "pa_attend_fp8: queries are f16 or bf16");
    if (num_seqs < 0 || num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0)
        return fail(PA_ERR_INVALID_ARG, "pa_attend_fp8: bad sizes");
    if (num_heads % num_kv_heads != 0)
        return fail(PA_ERR_INVALID_ARG, "pa_attend_fp8: num_heads=%d must be a multiple of num_kv_heads=%d", num_heads, num_kv_heads);
    if ((head_dim != 64 && head_dim != 128) || (block_size != 16 && block_size != 32))
        return fail(PA_ERR_UNSUPPORTED, "pa_attend_fp8: compiled for head_dim 64 and 128, block_size 16 and 32 (head_dim=%d block_size=%d)",
                    head_dim, block_size);
    if (!fits_int((long long)max_blocks_per_seq * block_size + 1024) || !fits_int((long long)num_blocks * num_kv_heads * block_size) ||
        !fits_int((long long)num_tokens * num_heads))
        return fail(PA_ERR_INVALID_ARG, "pa_attend_fp8: max_blocks_per_seq * block_size + 1024, num_blocks * num_kv_heads * block_size "
                                        "and num_tokens * num_heads must be < 2^31");
    if (num_seqs > kMaxStepSeqs) return fail(PA_ERR_UNSUPPORTED, "pa_attend_fp8: num_seqs=%d > %d", num_seqs, kMaxStepSeqs);
    if (!std::isfinite(scale)) return fail(PA_ERR_INVALID_ARG, "pa_attend_fp8: scale is not finite");
    if (num_tokens == 0 || num_seqs == 0) return PA_OK;
    if (!out || !query || !key_cache || !k_scale || !v_scale || !block_tables || !context_lens || !q_offsets)
        return fail(PA_ERR_INVALID_ARG, "pa_attend_fp8: NULL pointer");
    if (!aligned(out, 16) || !aligned(query, 16) || !aligned(key_cache, 16) || !aligned(value_cache, 16) || !aligned(k_scale, 4) ||
        !aligned(v_scale, 4) || !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(q_offsets, 4))
        return fail(PA_ERR_INVALID_ARG, "pa_attend_fp8: misaligned buffer (query, out and caches: 16 bytes)");
    const long long q_bytes = 2ll * num_tokens * num_heads * head_dim;
    if (overlap(out, q_bytes, query, q_bytes)) return fail(PA_ERR_INVALID_ARG, "pa_attend_fp8: out overlaps query");
    AttendArgs a{out, query, static_cast<const uint8_t*>(key_cache), static_cast<const uint8_t*>(value_cache), k_scale, v_scale,
                 block_tables, context_lens, q_offsets, num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, block_size,
                 max_blocks_per_seq, num_blocks, dtype, scale, workspace, 0, nullptr};
    const int st = device_state(&a.err, &a.num_sms);
    if (st != PA_OK) return st;
    const size_t need = attend_fp8_workspace_bytes(a.num_sms, num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, block_size,
                                                   max_blocks_per_seq);
    if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256)))
        return fail(PA_ERR_INVALID_ARG, "pa_attend_fp8: needs a 256-byte aligned workspace of %zu bytes (%zu given)", need,
                    workspace ? workspace_bytes : (size_t)0);
    // rows of K and V of a (block, head); in the layout of records K and V alternate
    const long long records = (long long)num_blocks * num_kv_heads * (value_cache ? 1 : 2);
    CUtensorMap kmap, vmap;
    int ms = record_map(&kmap, key_cache, records, block_size * head_dim);
    if (ms == PA_OK && value_cache) ms = record_map(&vmap, value_cache, records, block_size * head_dim);
    if (ms != PA_OK) return ms;
    const cudaError_t e = attend_fp8_launch(a, kmap, value_cache ? vmap : kmap, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? PA_OK : launch_failed(e, "pa_attend_fp8");
}

size_t pa_attend_fp8_workspace_size(int num_tokens, int num_seqs, int num_heads, int num_kv_heads, int head_dim, int block_size,
                                    int max_blocks_per_seq, int dtype) {
    clear_error();
    if ((dtype != PA_F16 && dtype != PA_BF16) || (head_dim != 64 && head_dim != 128) || num_tokens < 0 || num_seqs < 0 ||
        num_kv_heads <= 0 || num_heads <= 0 || num_heads % num_kv_heads != 0 || block_size <= 0 || max_blocks_per_seq <= 0)
        return 0;
    unsigned* err = nullptr;
    int sms = 0;
    if (device_state(&err, &sms) != PA_OK) return 0;
    return attend_fp8_workspace_bytes(sms, num_seqs, num_tokens, num_heads, num_kv_heads, head_dim, block_size, max_blocks_per_seq);
}

}  // extern "C"
