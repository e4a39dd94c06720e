// Rotary positions of queries and keys, fused with the paged write of keys and values.
//
// Pair i < r / 2 of a head (elements i and i + r / 2, or 2i and 2i + 1), at position p, is turned by the angle
// p * inv_freq[i]:  (a, b) -> factor * (a cos - b sin, a sin + b cos); elements past r pass through.  Products
// are formed in float32 and rounded once to the stored type.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include <cuda_fp8.h>

#include "pa_common.cuh"
#include "rope_math.cuh"
#include "step_ops.h"

namespace pa {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 4;  // tokens of a CTA, at most
constexpr int kRopeBatch = 2;   // rows that a thread has in flight (8192 tokens: two 29.6 us, four 31.5)

// Turns the V pairs of one slot of a head row, held in two chunks.  Half layout: chunk 0 holds the pairs' first
// elements, chunk 1 their second; interleaved: the two chunks are 2V neighbours.
template <typename T, int VB, bool INTERLEAVED>
__device__ __forceinline__ void rotate(Chunk<T, VB>& x0, Chunk<T, VB>& x1, const float2* cs) {
    constexpr int V = Chunk<T, VB>::V;
    if constexpr (V == 1) {
        const float p = x0.one(), q = x1.one();
        x0.put_one(p * cs[0].x - q * cs[0].y);
        x1.put_one(p * cs[0].y + q * cs[0].x);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 a = x0.pair(i), b = x1.pair(i);
            if (INTERLEAVED) {
                const float2 t = cs[i], u = cs[V / 2 + i];
                x0.put(i, make_float2(a.x * t.x - a.y * t.y, a.x * t.y + a.y * t.x));
                x1.put(i, make_float2(b.x * u.x - b.y * u.y, b.x * u.y + b.y * u.x));
            } else {
                const float2 t = cs[2 * i], u = cs[2 * i + 1];
                x0.put(i, make_float2(a.x * t.x - b.x * t.y, a.y * u.x - b.y * u.y));
                x1.put(i, make_float2(a.x * t.y + b.x * t.x, a.y * u.y + b.y * u.x));
            }
        }
    }
}

// Rows of a token: its query heads, key heads, value heads.  A row is ns = head_dim / 2V slots of two chunks; a
// thread keeps one slot, so its place in a row and its pairs are fixed, and walks over the rows of the CTA's
// tokens.  The (cos, sin) of a token are computed once per CTA, not once per head, and the steps of the pairs, in float64, once for
// its tokens.  Rows are moved once, so HBM bounds it for prompts and latency for steps: 8192 tokens of 28 + 2 * 4 heads of 128 (bf16)
// take 30 us, 5.0 TB/s (31 with a step per token and pair); 64 tokens 5 us, 2.8 among others in a graph.
template <typename T, int VB, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_write_kv_kernel(const RopeWriteArgs a, int tokens_per_cta) {
    constexpr int V = Chunk<T, VB>::V;
    extern __shared__ float2 cs[];  // [tokens][rotary_dim / 2], then the pairs' steps
    __shared__ long long dest[kRopeTokens];
    griddep_wait();
    griddep_launch_dependents();
    const RopeArgs& r = a.r;
    const int half = r.rotary_dim / 2, tid = threadIdx.x;
    uint64_t* steps = reinterpret_cast<uint64_t*>(cs + tokens_per_cta * half);
    const int tok0 = blockIdx.x * tokens_per_cta, ntok = min(tokens_per_cta, r.num_tokens - tok0), pairs = ntok * half;
    // (loads that do not wait for one another, before the steps; destinations by threads that have no steps, where there are some)
    const int pos0 = tid < pairs ? a.positions[tok0 + tid / half] : 0;
    const int own = kRopeThreads - 1 - tid;
    const long long slot = own < ntok ? a.slot_mapping[tok0 + own] : -1;
    for (int i = tid; i < half; i += kRopeThreads) steps[i] = turn_step(r.inv_freq[i]);
    if (own < ntok) {
        long long d = -1;  // in rows of the cache, without the head
        if (slot >= (long long)r.num_blocks * r.block_size) {
            atomicOr(r.err, kErrBadSlot);
        } else if (slot >= 0) {
            const long long blk = slot / r.block_size;
            d = blk * r.num_kv_heads * r.block_size + (slot - blk * r.block_size);
        }
        dest[own] = d;
    }
    __syncthreads();
    for (int i = tid; i < pairs; i += kRopeThreads) {
        const int t = i / half;
        cs[i] = turn(steps[i - t * half], i == tid ? pos0 : a.positions[tok0 + t], r.factor);
    }
    __syncthreads();
    const int ns = r.head_dim / (2 * V), groups = kRopeThreads / ns;
    const int group = tid / ns, sl = tid - group * ns;
    if (group >= groups) return;
    // where the slot's two chunks are, and whether they turn
    const bool turns = sl < half / V;
    const int e0 = !turns || INTERLEAVED ? 2 * V * sl : V * sl;
    const int e1 = !turns || INTERLEAVED ? e0 + V : e0 + half;
    const int per_token = r.num_heads + 2 * r.num_kv_heads, rows = ntok * per_token;
    for (int row0 = group; row0 < rows; row0 += groups * kRopeBatch) {
        Chunk<T, VB> x0[kRopeBatch], x1[kRopeBatch];
#pragma unroll
        for (int u = 0; u < kRopeBatch; ++u) {
            const int row = row0 + u * groups;
            if (row >= rows) break;
            const int t = row / per_token;
            int h = row - t * per_token;
            const T* src;
            if (h < r.num_heads) {
                src = static_cast<const T*>(r.query) + (tok0 + t) * r.q_stride;
            } else if ((h -= r.num_heads) < r.num_kv_heads) {
                src = static_cast<const T*>(r.key) + (tok0 + t) * r.k_stride;
            } else {
                h -= r.num_kv_heads;
                src = static_cast<const T*>(r.value) + (tok0 + t) * r.v_stride;
            }
            x0[u].load(src + h * r.head_dim + e0);
            x1[u].load(src + h * r.head_dim + e1);
        }
#pragma unroll
        for (int u = 0; u < kRopeBatch; ++u) {
            const int row = row0 + u * groups;
            if (row >= rows) break;
            const int t = row / per_token;
            int h = row - t * per_token;
            const bool is_query = h < r.num_heads;
            if (!is_query) h -= r.num_heads;
            const bool is_value = !is_query && h >= r.num_kv_heads;
            if (is_value) h -= r.num_kv_heads;
            if (turns && !is_value) rotate<T, VB, INTERLEAVED>(x0[u], x1[u], cs + t * half + sl * V);
            T* dst;
            if (is_query) {
                dst = static_cast<T*>(r.query_out) + ((long long)(tok0 + t) * r.num_heads + h) * r.head_dim;
            } else {
                if (dest[t] < 0) continue;
                dst = static_cast<T*>(is_value ? a.value_cache : a.key_cache) +
                      (dest[t] + (long long)h * r.block_size) * r.head_dim;
            }
            x0[u].store(dst + e0);
            x1[u].store(dst + e1);
        }
    }
}

// ---- FP8 append --------------------------------------------------------------------------------

// Largest b in [0, n) with off[b] <= x, or -1; 32 probes at a time by the whole warp.
__device__ __forceinline__ int warp_find(const int32_t* off, int n, int x, int lane) {
    int lo = -1, hi = n;  // off[lo] <= x < off[hi], with off[-1] = -inf, off[n] = inf
    while (hi - lo > 1) {
        const int step = (hi - lo - 1 + 31) / 32;
        const int i = lo + (lane + 1) * step;
        const int below = __popc(__ballot_sync(0xffffffffu, i < hi && off[i] <= x));
        lo += below * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

constexpr int kAppendThreads = 256, kAppendWarps = kAppendThreads / 32;
constexpr float kScaleFloor = 7.888609052210118e-31f;  // 2^-100: the scale of a block of zeros

// e4m3 of four quotients y / scale, inv = 1 / scale rounded.  y * inv is within 2 steps of float32 of the quotient, and codes change
// at values whose lower 19 bits of mantissa are zero (four bits are kept, one decides; fewer below 2^-6): next to
// those alone the division is made.  (16 divisions a slot took more registers than there are for two CTAs per SM.)
__device__ __forceinline__ uint32_t codes_of(float y0, float y1, float y2, float y3, float scale, float inv) {
    float q[4] = {y0 * inv, y1 * inv, y2 * inv, y3 * inv};
    unsigned near = ~0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) near = min(near, (__float_as_uint(q[i]) + 4) & 0x7ffffu);
    if (near < 9) {
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {  // (one division in the code, not sixteen)
            const float x = y0 / scale;
            y0 = y1, y1 = y2, y2 = y3;
            q[0] = q[1], q[1] = q[2], q[2] = q[3], q[3] = x;
        }
    }
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, __NV_E4M3) |
           ((uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(q[2], q[3]), __NV_SATFINITE, __NV_E4M3) << 16);
}

// (cos, sin) of a token's pairs in shared memory, for slots of V pairs: two pairs to 16 bytes, those of neighbouring slots
// next to each other, so that the lanes of a row read without bank conflicts.
template <int V>
__device__ __forceinline__ int turn_place(int pair, int slots) {
    return V == 1 ? pair : (((pair % V) / 2) * slots + pair / V) * 2 + pair % 2;
}
template <int V>
__device__ __forceinline__ void load_turns(float2 (&cs)[V], const float2* of_token, int slot, int slots) {
    if constexpr (V == 1) {
        cs[0] = of_token[slot];
    } else {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            const float4 w = *reinterpret_cast<const float4*>(of_token + (j * slots + slot) * 2);
            cs[2 * j] = make_float2(w.x, w.y);
            cs[2 * j + 1] = make_float2(w.z, w.w);
        }
    }
}

// The V pairs of one slot in float32: first[] and second[], rotated where TURNS is set.  Interleaved slots hold V pairs too.
template <typename T, int VB>
__device__ __forceinline__ void turned(const Chunk<T, VB>& x0, const Chunk<T, VB>& x1, const float2* cs, bool turns, bool interleaved,
                                       float* y0, float* y1) {
    constexpr int V = Chunk<T, VB>::V;
    if constexpr (V == 1) {
        y0[0] = x0.one();
        y1[0] = x1.one();
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 a = x0.pair(i), b = x1.pair(i);
            y0[2 * i] = a.x, y0[2 * i + 1] = a.y;
            y1[2 * i] = b.x, y1[2 * i + 1] = b.y;
        }
    }
    if (!turns) return;
    if (V > 1 && interleaved) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float* y = 2 * i < V ? y0 : y1;
            const int e = (2 * i) % V;
            const float p = y[e], q = y[e + (V > 1 ? 1 : 0)];
            y[e] = p * cs[i].x - q * cs[i].y;
            y[e + (V > 1 ? 1 : 0)] = p * cs[i].y + q * cs[i].x;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float p = y0[i], q = y1[i];
            y0[i] = p * cs[i].x - q * cs[i].y;
            y1[i] = p * cs[i].y + q * cs[i].x;
        }
    }
}

template <int V>
__device__ __forceinline__ void store_codes(uint8_t* p, const float* y, float scale, float inv) {
    if constexpr (V == 1) {
        *p = (uint8_t)codes_of(y[0], y[0], y[0], y[0], scale, inv);
    } else {
        uint32_t w[V / 4];
#pragma unroll
        for (int i = 0; i < V / 4; ++i) w[i] = codes_of(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3], scale, inv);
        if constexpr (V == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t*>(p) = w[0];
    }
}

__device__ __forceinline__ uint32_t requantised(uint32_t c, float held, float scale, float inv) {
    const float2 lo = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xffffu), __NV_E4M3)));
    const float2 hi = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> 16), __NV_E4M3)));
    return codes_of(lo.x * held, lo.y * held, hi.x * held, hi.y * held, scale, inv);
}

// The codes that a block holds already, in a larger scale.  One warp.
__device__ __noinline__ void requantise(uint4* at, int units, float held, float scale, float inv, int lane) {
    for (int i = lane; i < units; i += 128) {
        uint4 c[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (i + 32 * u < units) c[u] = at[i + 32 * u];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (i + 32 * u < units)
                at[i + 32 * u] = make_uint4(requantised(c[u].x, held, scale, inv), requantised(c[u].y, held, scale, inv),
                                            requantised(c[u].z, held, scale, inv), requantised(c[u].w, held, scale, inv));
    }
}

// The new rows of one block of one request.
struct AppendPiece {
    int tok, rows, off;  // first row, rows, offset of the first in its block
    int blk;
};

// One unit: a piece, one kv head, K or V, by a warp.  Rows are slots of two chunks as in rope_write_kv, RPS rows side by
// side.  Two passes, since the scale comes before the codes; the second reads the rows again, from L1 or L2, and rotates them
// again: holding a block between the passes takes 32 to 64 registers more than there are (prompt chunks 70 us instead of 55).
template <typename T, int D, int BS, int VB>
__device__ __forceinline__ void append_unit(const RopeAppendArgs& a, const AppendPiece& piece, int h, bool is_value,
                                            const float2* cs_of_first, int lane) {
    constexpr int V = Chunk<T, VB>::V, NS = D / (2 * V), LPR = NS < 32 ? NS : 32, SPL = NS / LPR, RPS = 32 / LPR;
    constexpr int STEPS = BS / RPS;
    const RopeArgs& r = a.r;
    const int sub = lane / LPR, half = r.rotary_dim / 2, n = piece.rows, off = piece.off;
    const T* src = is_value ? static_cast<const T*>(r.value) + h * D + (long long)piece.tok * r.v_stride
                            : static_cast<const T*>(r.key) + h * D + (long long)piece.tok * r.k_stride;
    const long long stride = is_value ? r.v_stride : r.k_stride;
    const size_t si = (size_t)piece.blk * r.num_kv_heads + h;
    float* scale_at = (is_value ? a.v_scale : a.k_scale) + si;
    const float held = off > 0 ? *scale_at : 0.f;  // a block that starts here has no scale yet
    float most = 0.f, scale = 0.f, inv = 0.f;
    const bool both = a.value_cache == nullptr;
    uint8_t* base = both ? a.key_cache + (si * 2 + (is_value ? 1 : 0)) * BS * D
                         : (is_value ? a.value_cache : a.key_cache) + si * BS * D;
    // one slot of one row: pass 0 its largest magnitude, pass 1 its codes
    auto slot_of = [&](auto pass, const Chunk<T, VB>& x0, const Chunk<T, VB>& x1, int row, int sl, int e0, int e1, bool turns) {
        float2 cs[V];
        float y0[V], y1[V];
        if (turns) load_turns<V>(cs, cs_of_first + row * half, sl, half / V);
        turned<T, VB>(x0, x1, cs, turns, r.interleaved, y0, y1);
        if constexpr (decltype(pass)::value == 0) {
#pragma unroll
            for (int i = 0; i < V; ++i) {  // infinities saturate, NaN stays: neither sets a scale
                const float m0 = fabsf(y0[i]), m1 = fabsf(y1[i]);
                if (m0 <= 3.402823466e38f) most = fmaxf(most, m0);
                if (m1 <= 3.402823466e38f) most = fmaxf(most, m1);
            }
        } else {
            uint8_t* p = base + (off + row) * D;
            store_codes<V>(p + e0, y0, scale, inv);
            store_codes<V>(p + e1, y1, scale, inv);
        }
    };
    auto all = [&](auto pass) {
#pragma unroll 1
        for (int j = 0; j < STEPS * SPL; ++j) {
            const int row = j / SPL * RPS + sub, sl = j % SPL * LPR + lane % LPR;
            if (row >= n) continue;
            const bool turns = !is_value && sl < half / V, pairs = !turns || r.interleaved;  // neighbouring chunks
            const int e0 = pairs ? 2 * V * sl : V * sl, e1 = pairs ? e0 + V : e0 + half;
            Chunk<T, VB> x0, x1;
            x0.load(src + row * stride + e0);
            x1.load(src + row * stride + e1);
            slot_of(pass, x0, x1, row, sl, e0, e1, turns);
        }
    };
    all(std::integral_constant<int, 0>());
    // (magnitudes are not negative: their order is that of their bits)
    most = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(most)));
    scale = fmaxf(fmaxf(held, most / 448.f), kScaleFloor);
    inv = 1.f / scale;
    if (scale > held && off > 0) requantise(reinterpret_cast<uint4*>(base), off * (D / 16), held, scale, inv, lane);
    all(std::integral_constant<int, 1>());
    __syncwarp();
    if (lane == 0 && scale != held) *scale_at = scale;
}

// CTA (window, part): the query rows of a window of `window` tokens, and the blocks whose first row of this call lies in it.
// Their positions are found and their angles computed once, in shared memory; warps then take units and groups of query
// heads in turn, every parts-th CTA's worth of them.  Dependent steps bound it (rows, then the scale, then the codes), at two CTAs
// per SM: 8300 prompt tokens of 28 + 2 * 4 heads of 128 (bf16) take 46 us (3.1 TB/s), 2240 of 3 * 32 heads 54 us (1.7), a decode step
// of 64 tokens 7.4 us.  At 128 registers the 16-byte instances of 16-bit types spill 24 - 28 bytes; 80 registers for three CTAs spilled
// far more (prompts 64 us); the rows' prefetch into L2 while positions are
// found gained nothing.
template <typename T, int D, int BS, int VB>
__global__ void __launch_bounds__(kAppendThreads, 2) rope_append_fp8_kernel(const RopeAppendArgs a, int window, int parts) {
    constexpr int V = Chunk<T, VB>::V, NS = D / (2 * V), LPR = NS < 32 ? NS : 32, SPL = NS / LPR, RPS = 32 / LPR;
    constexpr int kBatch = 2, kGroup = kBatch * RPS;  // query heads of a warp's turn
    extern __shared__ __align__(16) float2 cs[];      // [window + BS - 1][rotary_dim / 2], see turn_place()
    __shared__ AppendPiece pieces[BS];
    __shared__ uint64_t steps[D / 2];
    __shared__ int position[2 * BS];
    __shared__ int num_pieces, num_positions;
    __shared__ unsigned rotated;  // tokens of the window that belong to a request
    griddep_wait();
    griddep_launch_dependents();
    const RopeArgs& r = a.r;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = a.num_seqs, half = r.rotary_dim / 2;
    const int part = blockIdx.x % parts;
    const int t0 = (int)(blockIdx.x / parts) * window;
    if (warp == 0) {
        const int t = t0 + lane, tokens = min(window, r.num_tokens - t0);
        int lo = warp_find(a.q_offsets, B + 1, t0, lane);
        int hi = (tokens > 1 ? warp_find(a.q_offsets, B + 1, t0 + tokens - 1, lane) : lo) + 1;
        while (hi - lo > 1) {  // largest b in [lo, hi) whose rows begin at or before t
            const int mid = lo + (hi - lo) / 2;
            if (a.q_offsets[mid] <= t) lo = mid;
            else hi = mid;
        }
        bool in = lane < tokens && lo >= 0 && lo < B, own = false;
        int pos = 0, n = 0, off = 0, blk = 0, first = 0, next = 0;
        if (in) {  // (where offsets do not ascend, the search may end anywhere: CTA 0 reports them)
            first = a.q_offsets[lo];
            next = a.q_offsets[lo + 1];
            in = first >= 0 && first <= t && t < next && next <= r.num_tokens;
        }
        if (in) {
            const int L = a.context_lens[lo];
            const long long start = (long long)L - ((long long)next - first);  // position of its first row
            pos = (int)(start + (t - first));
            if (start < 0 || L > (long long)a.max_blocks * BS) {
                if (t == first && part == 0) atomicOr(r.err, kErrBadContext);
            } else {
                off = pos % BS;
                n = min(BS - off, next - t);
                own = n > 0 && (t == first || off == 0);
                if (own) blk = a.block_tables[(size_t)lo * a.max_blocks + pos / BS];
                if (own && (blk < 0 || blk >= r.num_blocks)) {
                    if (part == 0) atomicOr(r.err, kErrBadTable);
                    own = false;
                }
            }
            position[lane] = pos;
        }
        const unsigned owners = __ballot_sync(0xffffffffu, own), some = __ballot_sync(0xffffffffu, in);
        if (own) pieces[__popc(owners & ((1u << lane) - 1))] = AppendPiece{t, n, off, blk};
        // the last piece may reach past the window
        const int last = owners ? 31 - __clz(owners) : 0;
        const int end = owners ? last + __shfl_sync(0xffffffffu, n, last) : 0, last_pos = __shfl_sync(0xffffffffu, pos, last);
        if (tokens + lane < end) position[tokens + lane] = last_pos + (tokens + lane - last);
        if (lane == 0) {
            num_pieces = __popc(owners);
            num_positions = max(some ? 32 - __clz(some) : 0, end);
            rotated = some;
        }
    } else {
        for (int i = tid - 32; i < half; i += kAppendThreads - 32) steps[i] = turn_step(r.inv_freq[i]);
        if (blockIdx.x == 0) {
            bool bad = false;
            for (int b = tid - 32; b < B; b += kAppendThreads - 32) bad |= !is_run(a.q_offsets[b], a.q_offsets[b + 1], r.num_tokens);
            if (bad) atomicOr(r.err, kErrBadContext);
        }
    }
    __syncthreads();
    for (int i = tid; i < num_positions * half; i += kAppendThreads) {
        const int t = i / half, pair = i - t * half;
        const float2 x = turn(steps[pair], position[t], r.factor);
        cs[t * half + turn_place<V>(pair, half / V)] = x;
    }
    __syncthreads();
    const int units = num_pieces * r.num_kv_heads * 2, groups = (r.num_heads + kGroup - 1) / kGroup;
    const int tokens = min(window, r.num_tokens - t0), items = units + tokens * groups;
    for (int item = part * kAppendWarps + warp; item < items; item += parts * kAppendWarps) {
        if (item < units) {
            const int of_piece = item / (r.num_kv_heads * 2), u = item - of_piece * (r.num_kv_heads * 2);
            const AppendPiece piece = pieces[of_piece];
            append_unit<T, D, BS, VB>(a, piece, u >> 1, u & 1, cs + (piece.tok - t0) * half, lane);
            continue;
        }
        const int i = (item - units) / groups, head0 = (item - units - i * groups) * kGroup;
        if (!(rotated >> i & 1)) continue;
        const T* src = static_cast<const T*>(r.query) + (long long)(t0 + i) * r.q_stride;
        T* dst = static_cast<T*>(r.query_out) + (long long)(t0 + i) * r.num_heads * D;
#pragma unroll
        for (int s = 0; s < SPL; ++s) {
            const int sl = s * LPR + lane % LPR;
            const bool turns = sl < half / V, pairs = !turns || r.interleaved;  // neighbouring chunks
            const int e0 = pairs ? 2 * V * sl : V * sl, e1 = pairs ? e0 + V : e0 + half;
            float2 c[V];
            if (turns) load_turns<V>(c, cs + i * half, sl, half / V);
            Chunk<T, VB> x0[kBatch], x1[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int h = head0 + k * RPS + lane / LPR;
                if (h < r.num_heads) {
                    x0[k].load(src + h * D + e0);
                    x1[k].load(src + h * D + e1);
                }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int h = head0 + k * RPS + lane / LPR;
                if (h >= r.num_heads) continue;
                if (turns && r.interleaved) rotate<T, VB, true>(x0[k], x1[k], c);
                else if (turns) rotate<T, VB, false>(x0[k], x1[k], c);
                x0[k].store(dst + h * D + e0);
                x1[k].store(dst + h * D + e1);
            }
        }
    }
}

bool multiple(const void* p, long long bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0; }

template <typename T, int VB>
cudaError_t rope_write_typed(const RopeWriteArgs& a, cudaStream_t stream) {
    // Four tokens share a CTA when that still gives every SM one; fewer tokens take a CTA each.  (In a graph, four against one: 8192
    // tokens, bf16, 29.6 and 38.6 us; 1001 tokens, f32, 2.8 and 4.7; 64 tokens 4.8 and 2.8.)
    const int per = a.r.num_tokens >= kRopeTokens * a.num_sms ? kRopeTokens : 1;
    const unsigned grid = (unsigned)((a.r.num_tokens + per - 1) / per);
    const size_t smem = (size_t)(per + 1) * (a.r.rotary_dim / 2) * sizeof(float2);  // (steps are as large as a token's pairs)
    if (a.r.interleaved)
        return launch_pdl(rope_write_kv_kernel<T, VB, true>, dim3(grid), dim3(kRopeThreads), smem, stream, a, per);
    return launch_pdl(rope_write_kv_kernel<T, VB, false>, dim3(grid), dim3(kRopeThreads), smem, stream, a, per);
}

// Whether a row splits into chunks of vb bytes: aligned bases and strides, and slots of two chunks that do not
// straddle the end of the pairs.
bool rope_splits(const RopeArgs& r, int eb, int vb) {
    const int v = vb / eb;
    if (r.head_dim % (2 * v) || r.head_dim / (2 * v) > kRopeThreads || (r.rotary_dim / 2) % v) return false;
    if ((r.head_dim - r.rotary_dim) % (2 * v)) return false;
    for (const void* p : {(const void*)r.query_out, r.query, r.key, r.value})
        if (!multiple(p, vb)) return false;
    return (r.q_stride * eb) % vb == 0 && (r.k_stride * eb) % vb == 0 && (r.v_stride * eb) % vb == 0;
}

template <typename T, int D, int BS, int VB>
cudaError_t append_typed(const RopeAppendArgs& a, cudaStream_t stream) {
    const RopeArgs& r = a.r;
    constexpr int V = VB / (int)sizeof(T), NS = D / (2 * V), RPS = NS < 32 ? 32 / NS : 1;
    // A window is a block long, so that a prompt has one block per window; while a window per token does not fill the
    // GPU, every token has its own, so that the tokens of a decode step do not queue behind one another.  (2240 tokens of 37 requests,
    // 32 kv heads: 59 us, with a window per token 129; 64 decode tokens: 7.4 us on the GPU,
    // 19.6 with warps that took several.  Decode steps either side, in a graph: 304 tokens 8.8 us, 305 9.4, 512 9.5.)
    const int window = r.num_tokens <= 2 * a.num_sms ? 1 : BS;
    const long long windows = (r.num_tokens + window - 1) / window;
    // The rows of a window are shared among parts of CTAs, down to a turn per warp, while that makes at most four CTAs per SM
    // (prompt chunks / 32 kv heads, us: two 50 / 69, four 49 / 55, eight 53 / 59, sixteen 59 / 58).
    const long long items = 2ll * r.num_kv_heads + (long long)window * ((r.num_heads + 2 * RPS - 1) / (2 * RPS));
    const long long parts = std::max(1ll, std::min((items + kAppendWarps - 1) / kAppendWarps, 4ll * a.num_sms / windows));
    const size_t smem = (size_t)(window + BS - 1) * (r.rotary_dim / 2) * sizeof(float2);
    return launch_pdl(rope_append_fp8_kernel<T, D, BS, VB>, dim3((unsigned)(windows * parts)), dim3(kAppendThreads), smem, stream,
                      a, window, (int)parts);
}

template <typename T, int VB>
cudaError_t append_dispatch(const RopeAppendArgs& a, cudaStream_t stream) {
    const int d = a.r.head_dim, bs = a.r.block_size;
    if (d == 128 && bs == 16) return append_typed<T, 128, 16, VB>(a, stream);
    if (d == 128 && bs == 32) return append_typed<T, 128, 32, VB>(a, stream);
    if (d == 64 && bs == 16) return append_typed<T, 64, 16, VB>(a, stream);
    if (d == 64 && bs == 32) return append_typed<T, 64, 32, VB>(a, stream);
    return cudaErrorInvalidValue;
}

template <typename T>
cudaError_t append_split(const RopeAppendArgs& a, cudaStream_t stream) {
    return rope_splits(a.r, sizeof(T), 16) ? append_dispatch<T, 16>(a, stream) : append_dispatch<T, (int)sizeof(T)>(a, stream);
}

}  // namespace

cudaError_t rope_write_kv_launch(const RopeWriteArgs& a, cudaStream_t stream) {
    const int eb = a.r.dtype == 0 ? 4 : 2;
    auto splits = [&](int vb) { return multiple(a.key_cache, vb) && multiple(a.value_cache, vb) && rope_splits(a.r, eb, vb); };
    if (a.r.dtype == 0)
        return splits(16) ? rope_write_typed<float, 16>(a, stream) : rope_write_typed<float, 4>(a, stream);
    const int vb = splits(16) ? 16 : splits(4) ? 4 : 2;
    if (a.r.dtype == 1)
        return vb == 16  ? rope_write_typed<__half, 16>(a, stream)
               : vb == 4 ? rope_write_typed<__half, 4>(a, stream)
                         : rope_write_typed<__half, 2>(a, stream);
    return vb == 16  ? rope_write_typed<__nv_bfloat16, 16>(a, stream)
           : vb == 4 ? rope_write_typed<__nv_bfloat16, 4>(a, stream)
                     : rope_write_typed<__nv_bfloat16, 2>(a, stream);
}

cudaError_t rope_append_fp8_launch(const RopeAppendArgs& a, cudaStream_t stream) {
    switch (a.r.dtype) {
        case 0: return append_split<float>(a, stream);
        case 1: return append_split<__half>(a, stream);
        default: return append_split<__nv_bfloat16>(a, stream);
    }
}

}  // namespace pa
