// Norms of query and key heads, rotary positions and the paged write, in one pass.
//
// For every query and key head x of d elements, with weights w:
//     y_i = x_i / sqrt(sum x^2 / d + eps) * (w_i + offset),  then the pairs of y are turned as in rope_ops.cu;
// values pass as they are.  Squares, their sum, the norm, the products and the turn are float32; one rounding, to the stored type.
// 8192 tokens of 28 + 2 * 4 heads of 128 (bf16) take 33.3 us, 4.5 TB/s, issue slots 54 % busy (rope_write_kv, without norms, 30); 1001 tokens of
// 16 + 2 * 8 heads of 64 (float32) 8.6 us on the GPU.
#include <algorithm>
#include <cstdint>

#include "pa_common.cuh"
#include "rope_math.cuh"
#include "tree_ops.h"

namespace pa {

namespace {

// Measured when chosen, 8192 tokens of 28 + 2 * 4 heads of 128 (bf16): three CTAs per SM 33.3 us (80 registers), four 35.8 (64, and spills);
// two slots a lane 35.8, one 39.2 (what a row costs besides its elements, addresses, sums and norm, is half of the instructions).
constexpr int kNormThreads = 256, kNormCtasPerSm = 3;
constexpr int kNormSlots = 2;  // slots of a lane, where a row has as many

__device__ __forceinline__ float weight_at(const void* w, int dtype, int i) {
    return dtype == 0   ? static_cast<const float*>(w)[i]
           : dtype == 1 ? to_float(static_cast<const __half*>(w)[i])
                        : to_float(static_cast<const __nv_bfloat16*>(w)[i]);
}

// Turns of a pair with its weights: (x, y) -> (x a + y b, x c + y d), a = cos w_x, b = -sin w_y, c = sin w_x, d = cos w_y.  Of a slot of V pairs
// two go together, as four packed operands (two 16-byte units); those of neighbouring slots lie next to each other, so that the lanes
// of a row read without bank conflicts.
template <int V>
__device__ __forceinline__ void put_turn(float* table, int pair, int slots, float4 t) {
    if constexpr (V == 1) {
        reinterpret_cast<float4*>(table)[pair] = t;
    } else {
        const int slot = pair / V, i = pair % V;
        float* at = table + (((i / 2) * 2) * slots + slot) * 4 + i % 2;
        at[0] = t.x;
        at[2] = t.y;
        at += slots * 4;
        at[0] = t.z;
        at[2] = t.w;
    }
}

// The pairs of one slot, normed, weighted and turned.
template <typename T, int VB, bool INTERLEAVED>
__device__ __forceinline__ void turn_pairs(Chunk<T, VB>& x0, Chunk<T, VB>& x1, const float* table, int slot, int slots, float norm) {
    constexpr int V = Chunk<T, VB>::V;
    const float4* t = reinterpret_cast<const float4*>(table);
    if constexpr (V == 1) {
        const float4 w = t[slot];
        const float x = x0.one() * norm, y = x1.one() * norm;
        x0.put_one(fmaf(x, w.x, y * w.y));
        x1.put_one(fmaf(x, w.z, y * w.w));
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {  // pairs 2i and 2i + 1
            const float4 p = t[2 * i * slots + slot], q = t[(2 * i + 1) * slots + slot];
            const float2 n = make_float2(norm, norm);
            if (INTERLEAVED) {  // a pair is neighbours: four elements of one chunk
                Chunk<T, VB>& c = 2 * i < V / 2 ? x0 : x1;
                const int at = 2 * i % (V / 2);
                const float2 u = mul2(c.pair(at), n), v = mul2(c.pair(at + 1), n);
                c.put(at, make_float2(fmaf(u.x, p.x, u.y * p.z), fmaf(u.x, q.x, u.y * q.z)));
                c.put(at + 1, make_float2(fmaf(v.x, p.y, v.y * p.w), fmaf(v.x, q.y, v.y * q.w)));
            } else {
                const float2 x = mul2(x0.pair(i), n), y = mul2(x1.pair(i), n);
                x0.put(i, fma2(x, make_float2(p.x, p.y), mul2(y, make_float2(p.z, p.w))));
                x1.put(i, fma2(x, make_float2(q.x, q.y), mul2(y, make_float2(q.z, q.w))));
            }
        }
    }
}

// Elements that do not turn: the pairs' own weights are the table's a and d.
template <typename T, int VB>
__device__ __forceinline__ void scale_pairs(Chunk<T, VB>& x0, Chunk<T, VB>& x1, const float* table, int slot, int slots, float norm) {
    constexpr int V = Chunk<T, VB>::V;
    const float4* t = reinterpret_cast<const float4*>(table);
    if constexpr (V == 1) {
        const float4 w = t[slot];
        x0.put_one(x0.one() * norm * w.x);
        x1.put_one(x1.one() * norm * w.w);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float4 p = t[2 * i * slots + slot], q = t[(2 * i + 1) * slots + slot];
            const float2 n = make_float2(norm, norm);
            x0.put(i, mul2(mul2(x0.pair(i), n), make_float2(p.x, p.y)));
            x1.put(i, mul2(mul2(x1.pair(i), n), make_float2(q.z, q.w)));
        }
    }
}

// A row (a query, key or value head of a token) is slots = d / 2V slots of two chunks of V elements, as in rope_ops.cu; LPR lanes, a power
// of two, share it, S slots each.  A warp takes a token at a time: its turns, with the weights, are made once and not once per head, in shared
// memory of the warp's own, so that no warp waits for another; the steps of the pairs, in float64, and the weights are the CTA's.  A lane has two
// rows in flight, the next ones while it works on these.  Rows are moved once: HBM bounds it for prompts, latency for steps.
template <typename T, int VB, int S, bool INTERLEAVED>
__global__ void __launch_bounds__(kNormThreads, kNormCtasPerSm) norm_rope_write_kv_kernel(const NormRopeArgs a, int LPR) {
    constexpr int V = Chunk<T, VB>::V;
    extern __shared__ float4 tables[];  // [warps][queries, keys][d / 2], see put_turn; then the pairs' steps; then weights [2][d]
    griddep_wait();
    griddep_launch_dependents();
    const RopeArgs& r = a.r;
    const int half = r.rotary_dim / 2, d = r.head_dim, pairs = d / 2, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int Hq = r.num_heads, Hk = r.num_kv_heads, rows = Hq + 2 * Hk;
    float4* table = tables + warp * 2 * pairs;
    uint64_t* steps = reinterpret_cast<uint64_t*>(tables + warps * 2 * pairs);
    float* weights = reinterpret_cast<float*>(steps + half);
    const int slots = d / (2 * V), RPW = 32 / LPR, sub = lane / LPR, in_row = lane % LPR;
    const float per_element = 1.f / (float)d;
    // where the lane's chunks are in a row
    int e0[S], e1[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        const int sl = in_row + s * LPR;
        const bool split = sl < half / V && !INTERLEAVED;
        e0[s] = split ? V * sl : 2 * V * sl;
        e1[s] = split ? V * sl + half : 2 * V * sl + V;
    }
    bool first = true;
    const long long stride = (long long)gridDim.x * warps;
    for (long long tok = (long long)blockIdx.x * warps + warp; first || tok < r.num_tokens; tok += stride) {
        const bool there = tok < r.num_tokens;
        Chunk<T, VB> x0[2][S], x1[2][S];
        auto load = [&](int u, int h) {  // row h: queries, keys, values
            if (h >= rows || !there) return;
            const bool is_query = h < Hq, is_value = h >= Hq + Hk;
            const T* src = static_cast<const T*>(is_query ? r.query : is_value ? r.value : r.key);
            src += tok * (is_query ? r.q_stride : is_value ? r.v_stride : r.k_stride);
            src += (h - (is_query ? 0 : is_value ? Hq + Hk : Hq)) * d;
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (in_row + s * LPR < slots) {
                    x0[u][s].load(src + e0[s]);
                    x1[u][s].load(src + e1[s]);
                }
        };
        load(0, sub);  // (the first rows are on their way while the turns are made)
        load(1, sub + RPW);
        const int pos = there ? a.positions[tok] : 0;
        const long long slot = there ? a.slot_mapping[tok] : -1;
        if (first) {
            for (int i = tid; i < half; i += blockDim.x) steps[i] = turn_step(r.inv_freq[i]);
            for (int i = tid; i < 2 * d; i += blockDim.x) {
                const void* w = i < d ? a.q_weight : a.k_weight;
                weights[i] = w ? weight_at(w, a.weight_dtype, i < d ? i : i - d) + a.weight_offset : 1.f;
            }
            __syncthreads();
            first = false;
            if (!there) return;
        }
        long long to = -1;  // in rows of the cache, without the head
        if (slot >= (long long)r.num_blocks * r.block_size) {
            if (lane == 0) atomicOr(r.err, kErrBadSlot);
        } else if (slot >= 0) {
            const long long blk = slot / r.block_size;
            to = blk * Hk * r.block_size + (slot - blk * r.block_size);
        }
        for (int pair = lane; pair < pairs; pair += 32) {
            const bool turns = pair < half;
            const float2 cs = turns ? turn(steps[pair], pos, r.factor) : make_float2(1.f, 0.f);
            // the pair's elements
            const int still = 2 * V * (pair / V) + pair % V;
            const int ex = !turns ? still : INTERLEAVED ? 2 * pair : pair, ey = !turns ? still + V : INTERLEAVED ? 2 * pair + 1 : pair + half;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float wx = weights[k * d + ex], wy = weights[k * d + ey];
                put_turn<V>(reinterpret_cast<float*>(table + k * pairs), pair, slots, make_float4(cs.x * wx, -cs.y * wy, cs.y * wx, cs.x * wy));
            }
        }
        __syncwarp();
        auto work = [&](int u, int h) {
            const bool live = h < rows;
            float2 sums = make_float2(0.f, 0.f);
#pragma unroll
            for (int s = 0; s < S; ++s) {
                if (!live || in_row + s * LPR >= slots) continue;
                if constexpr (V == 1) {
                    sums.x = fmaf(x0[u][s].one(), x0[u][s].one(), sums.x);
                    sums.y = fmaf(x1[u][s].one(), x1[u][s].one(), sums.y);
                } else {
#pragma unroll
                    for (int i = 0; i < V / 2; ++i) {
                        const float2 y = x0[u][s].pair(i), z = x1[u][s].pair(i);
                        sums = fma2(y, y, fma2(z, z, sums));
                    }
                }
            }
            float sum = sums.x + sums.y;
            for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (!live) return;
            const bool is_query = h < Hq, is_value = h >= Hq + Hk;
            T* dst;
            if (is_query) {
                dst = static_cast<T*>(r.query_out) + (tok * Hq + h) * d;
            } else {
                if (to < 0) return;
                dst = static_cast<T*>(is_value ? a.value_cache : a.key_cache) + (to + (long long)(h - (is_value ? Hq + Hk : Hq)) * r.block_size) * d;
            }
            if (!is_value) {
                const float norm = __frsqrt_rn(fmaf(sum, per_element, a.eps));
                const float* turns = reinterpret_cast<const float*>(table + (is_query ? 0 : pairs));
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    const int sl = in_row + s * LPR;
                    if (sl >= slots) continue;
                    if (sl < half / V)
                        turn_pairs<T, VB, INTERLEAVED>(x0[u][s], x1[u][s], turns, sl, slots, norm);
                    else
                        scale_pairs<T, VB>(x0[u][s], x1[u][s], turns, sl, slots, norm);
                }
            }
#pragma unroll
            for (int s = 0; s < S; ++s)
                if (in_row + s * LPR < slots) {
                    x0[u][s].store(dst + e0[s]);
                    x1[u][s].store(dst + e1[s]);
                }
        };
        for (int h = 0; h < rows; h += 2 * RPW) {
            work(0, h + sub);
            load(0, h + 2 * RPW + sub);
            if (h + RPW < rows) work(1, h + RPW + sub);
            load(1, h + 3 * RPW + sub);
        }
        __syncwarp();
    }
}

bool multiple(const void* p, long long bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0; }

template <typename T, int VB, int S>
cudaError_t norm_typed(const NormRopeArgs& a, cudaStream_t stream) {
    const int slots = a.r.head_dim / (2 * (VB / (int)sizeof(T)));
    int lpr = 1;
    while (lpr * kNormSlots < slots && lpr < 32) lpr *= 2;
    if ((slots + lpr - 1) / lpr > S) return cudaErrorInvalidValue;
    const int threads = a.r.head_dim <= 256 ? kNormThreads : kNormThreads / 2;  // (so that the turns take 32 KB at most)
    const long long ctas = ((long long)a.r.num_tokens + threads / 32 - 1) / (threads / 32);
    const unsigned grid = (unsigned)std::min(ctas, (long long)kNormCtasPerSm * a.num_sms);
    const size_t smem = (size_t)(threads / 32) * a.r.head_dim * sizeof(float4) + (size_t)(a.r.rotary_dim / 2) * sizeof(uint64_t) +
                        (size_t)2 * a.r.head_dim * sizeof(float);
    auto* kernel = a.r.interleaved ? norm_rope_write_kv_kernel<T, VB, S, true> : norm_rope_write_kv_kernel<T, VB, S, false>;
    return launch_pdl(kernel, dim3(grid), dim3(threads), smem, stream, a, lpr);
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
        case 1: return splits(a, 2) ? norm_typed<__half, 16, 2>(a, stream) : norm_typed<__half, 2, 8>(a, stream);
        default: return splits(a, 2) ? norm_typed<__nv_bfloat16, 16, 2>(a, stream) : norm_typed<__nv_bfloat16, 2, 8>(a, stream);
    }
}

}  // namespace pa
