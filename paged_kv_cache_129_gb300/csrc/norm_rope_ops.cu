// Norms of query and key heads, rotary positions and the paged write, in one pass.
//
// For every query and key head x of d elements, with weights w:
//     y_i = x_i / sqrt(sum x^2 / d + eps) * (w_i + offset),  then the pairs of y are turned as in rope_ops.cu;
// values pass as they are.  Squares, their sum, the norm, the products and the turn are float32; one rounding, to the stored type.
#include <algorithm>
#include <cstdint>

#include "pa_common.cuh"
#include "rope_math.cuh"
#include "tree_ops.h"

namespace pa {

namespace {

constexpr int kNormThreads = 256, kNormWarps = kNormThreads / 32;
constexpr int kNormTokens = 4;  // tokens of a CTA, at most

__device__ __forceinline__ float weight_at(const void* w, int dtype, int i) {
    return dtype == 0   ? static_cast<const float*>(w)[i]
           : dtype == 1 ? to_float(static_cast<const __half*>(w)[i])
                        : to_float(static_cast<const __nv_bfloat16*>(w)[i]);
}

// A row is ns = d / 2V slots of two chunks of V elements (as in rope_ops.cu); LPR lanes, a power of two, share it, S slots each.
template <typename T, int VB, int S>
__global__ void __launch_bounds__(kNormThreads) norm_rope_write_kv_kernel(const NormRopeArgs a, int tokens_per_cta, int LPR) {
    constexpr int V = Chunk<T, VB>::V;
    extern __shared__ float2 cs[];  // [tokens][rotary_dim / 2]; then the pairs' steps; then query and key weights, [d] each
    __shared__ long long dest[kNormTokens];
    griddep_wait();
    griddep_launch_dependents();
    const RopeArgs& r = a.r;
    const int half = r.rotary_dim / 2, d = r.head_dim, tid = threadIdx.x, lane = tid & 31;
    uint64_t* steps = reinterpret_cast<uint64_t*>(cs + tokens_per_cta * half);
    float* weights = reinterpret_cast<float*>(steps + half);
    const int tok0 = blockIdx.x * tokens_per_cta, ntok = min(tokens_per_cta, r.num_tokens - tok0);
    for (int i = tid; i < half; i += kNormThreads) steps[i] = turn_step(r.inv_freq[i]);
    for (int i = tid; i < d; i += kNormThreads) {
        weights[i] = (a.q_weight ? weight_at(a.q_weight, a.weight_dtype, i) : 1.f) + (a.q_weight ? a.weight_offset : 0.f);
        weights[d + i] = (a.k_weight ? weight_at(a.k_weight, a.weight_dtype, i) : 1.f) + (a.k_weight ? a.weight_offset : 0.f);
    }
    if (tid < ntok) {
        const long long slot = a.slot_mapping[tok0 + tid];
        long long to = -1;  // in rows of the cache, without the head
        if (slot >= (long long)r.num_blocks * r.block_size) {
            atomicOr(r.err, kErrBadSlot);
        } else if (slot >= 0) {
            const long long blk = slot / r.block_size;
            to = blk * r.num_kv_heads * r.block_size + (slot - blk * r.block_size);
        }
        dest[tid] = to;
    }
    __syncthreads();
    for (int i = tid; i < ntok * half; i += kNormThreads) {
        const int t = i / half;
        cs[i] = turn(steps[i - t * half], a.positions[tok0 + t], r.factor);
    }
    __syncthreads();
    const int ns = d / (2 * V), RPW = 32 / LPR, sub = lane / LPR, in_row = lane % LPR;
    const int per_token = r.num_heads + 2 * r.num_kv_heads, rows = ntok * per_token;
    for (int base = (tid >> 5) * RPW; base < rows; base += kNormWarps * RPW) {
        const int row = base + sub;
        const bool live = row < rows;
        const int t = live ? row / per_token : 0;
        int h = live ? row - t * per_token : 0;
        const bool is_query = h < r.num_heads;
        if (!is_query) h -= r.num_heads;
        const bool is_value = !is_query && h >= r.num_kv_heads;
        if (is_value) h -= r.num_kv_heads;
        const T* src = is_query   ? static_cast<const T*>(r.query) + (tok0 + t) * r.q_stride
                       : is_value ? static_cast<const T*>(r.value) + (tok0 + t) * r.v_stride
                                  : static_cast<const T*>(r.key) + (tok0 + t) * r.k_stride;
        src += (long long)h * d;
        Chunk<T, VB> x0[S], x1[S];
        int e0[S], e1[S];
        float sum = 0.f;
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int sl = in_row + s * LPR;
            const bool turns = sl < half / V, split = turns && !r.interleaved;
            e0[s] = split ? V * sl : 2 * V * sl;
            e1[s] = split ? V * sl + half : 2 * V * sl + V;
            if (!live || sl >= ns) continue;
            x0[s].load(src + e0[s]);
            x1[s].load(src + e1[s]);
            float y0[V], y1[V];
            widen_slot<T, VB>(x0[s], x1[s], y0, y1);
#pragma unroll
            for (int i = 0; i < V; ++i) sum = fmaf(y0[i], y0[i], fmaf(y1[i], y1[i], sum));
        }
        for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float norm = 1.f / sqrtf(sum / (float)d + a.eps);
        if (!live || (!is_query && dest[t] < 0)) continue;
        T* dst = is_query ? static_cast<T*>(r.query_out) + ((long long)(tok0 + t) * r.num_heads + h) * d
                          : static_cast<T*>(is_value ? a.value_cache : a.key_cache) + (dest[t] + (long long)h * r.block_size) * d;
        const float* w = weights + (is_query ? 0 : d);
#pragma unroll
        for (int s = 0; s < S; ++s) {
            const int sl = in_row + s * LPR;
            if (sl >= ns) continue;
            if (!is_value) {
                float y0[V], y1[V];
                widen_slot<T, VB>(x0[s], x1[s], y0, y1);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    y0[i] *= norm * w[e0[s] + i];
                    y1[i] *= norm * w[e1[s] + i];
                }
                if (sl < half / V) turn_slot<V>(y0, y1, cs + t * half + sl * V, r.interleaved != 0);
                pack_slot<T, VB>(y0, y1, x0[s], x1[s]);
            }
            x0[s].store(dst + e0[s]);
            x1[s].store(dst + e1[s]);
        }
    }
}

bool multiple(const void* p, long long bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0; }

template <typename T, int VB, int S>
cudaError_t norm_typed(const NormRopeArgs& a, cudaStream_t stream) {
    const int ns = a.r.head_dim / (2 * (VB / (int)sizeof(T)));
    int lpr = 1;
    while (lpr < ns && lpr < 32) lpr *= 2;
    if ((ns + lpr - 1) / lpr > S) return cudaErrorInvalidValue;
    const int per = a.r.num_tokens >= kNormTokens * a.num_sms ? kNormTokens : 1;
    const unsigned grid = (unsigned)((a.r.num_tokens + per - 1) / per);
    const size_t smem = (size_t)(per + 1) * (a.r.rotary_dim / 2) * sizeof(float2) + (size_t)2 * a.r.head_dim * sizeof(float);
    return launch_pdl(norm_rope_write_kv_kernel<T, VB, S>, dim3(grid), dim3(kNormThreads), smem, stream, a, per, lpr);
}

// Whether a row splits into chunks of 16 bytes: aligned bases and strides, slots of two chunks that do not straddle the end of the pairs.
bool splits(const NormRopeArgs& a, int eb) {
    const RopeArgs& r = a.r;
    const int v = 16 / eb;
    if (r.head_dim % (2 * v) || (r.rotary_dim / 2) % v) return false;
    for (const void* p : {(const void*)r.query_out, r.query, r.key, r.value, (const void*)a.key_cache, (const void*)a.value_cache})
        if (!multiple(p, 16)) return false;
    return (r.q_stride * eb) % 16 == 0 && (r.k_stride * eb) % 16 == 0 && (r.v_stride * eb) % 16 == 0;
}

}  // namespace

cudaError_t norm_rope_write_kv_launch(const NormRopeArgs& a, cudaStream_t stream) {
    switch (a.r.dtype) {  // (head_dim <= 512: at most 64 slots of 8 floats, 32 of 16 halves, 256 of 2)
        case 0: return splits(a, 4) ? norm_typed<float, 16, 2>(a, stream) : norm_typed<float, 4, 8>(a, stream);
        case 1: return splits(a, 2) ? norm_typed<__half, 16, 1>(a, stream) : norm_typed<__half, 2, 8>(a, stream);
        default: return splits(a, 2) ? norm_typed<__nv_bfloat16, 16, 1>(a, stream) : norm_typed<__nv_bfloat16, 2, 8>(a, stream);
    }
}

}  // namespace pa
