// Rotary positions of queries and keys, fused with the paged write of keys and values.
//
// Pair i < r / 2 of a head (elements i and i + r / 2, or 2i and 2i + 1), at position p, is turned by the angle
// p * inv_freq[i]:  (a, b) -> factor * (a cos - b sin, a sin + b cos); elements past r pass through.  Products
// are formed in float32 and rounded once to the stored type.
//
// Angles of far positions: p * inv_freq in float32 is off by p * 2^-24 radians, useless at p = 10^6.  A turn is
// therefore a 64-bit fixed-point fraction: u = frac(inv_freq / 2 pi) * 2^64, and p * u modulo 2^64 is the angle
// in turns without whole ones, exactly; its top 32 bits, signed, are within 2^-32 turns of it, and
// sincospi(that / 2^31) is as exact as float32 gives.  One integer product per angle, no reduction.
#include <algorithm>
#include <cstdint>

#include <cuda_fp8.h>

#include "pa_common.cuh"
#include "step_ops.h"

namespace pa {

namespace {

__device__ __forceinline__ uint64_t turn_step(double inv_freq) {
    double t = inv_freq * 0.15915494309189533577;  // 1 / (2 pi)
    t -= floor(t);
    return __double2ull_rz(t * 18446744073709551616.0);  // * 2^64; a double below 1 stays below 2^64
}

__device__ __forceinline__ float2 turn(uint64_t step, int pos, float factor) {
    const int64_t a = (int64_t)(step * (uint64_t)(int64_t)pos + 0x80000000ull);
    float s, c;
    sincospif((float)(int)(a >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31: half turns
    return make_float2(c * factor, s * factor);
}

template <int BYTES>
struct VecOf;
template <>
struct VecOf<16> { using type = uint4; };
template <>
struct VecOf<4> { using type = uint32_t; };
template <>
struct VecOf<2> { using type = uint16_t; };

// VB bytes = V elements of type T.
template <typename T, int VB>
struct Chunk {
    static constexpr int V = VB / (int)sizeof(T);
    typename VecOf<VB>::type raw;
    __device__ __forceinline__ void load(const T* p) { raw = *reinterpret_cast<const typename VecOf<VB>::type*>(p); }
    __device__ __forceinline__ void store(T* p) const { *reinterpret_cast<typename VecOf<VB>::type*>(p) = raw; }
    __device__ __forceinline__ float get(int i) const { return to_float(reinterpret_cast<const T*>(&raw)[i]); }
    __device__ __forceinline__ void set(int i, float x) { reinterpret_cast<T*>(&raw)[i] = from_float<T>(x); }
};

constexpr int kRopeThreads = 256;
constexpr int kRopeTokens = 4;  // tokens of a CTA, at most
constexpr int kRopeBatch = 4;   // rows that a thread has in flight

// Turns the V pairs of one slot of a head row, held in two chunks.  Half layout: chunk 0 holds the pairs' first
// elements, chunk 1 their second; interleaved: the two chunks are 2V neighbours.
template <typename T, int VB, bool INTERLEAVED>
__device__ __forceinline__ void rotate(Chunk<T, VB>& x0, Chunk<T, VB>& x1, const float2* cs) {
    constexpr int V = Chunk<T, VB>::V;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float2 t = cs[i];
        if (INTERLEAVED && V > 1) {
            Chunk<T, VB>& x = 2 * i < V ? x0 : x1;
            const int e = (2 * i) % V;
            const float p = x.get(e), q = x.get(e + 1);
            x.set(e, p * t.x - q * t.y);
            x.set(e + 1, p * t.y + q * t.x);
        } else {
            const float p = x0.get(i), q = x1.get(i);
            x0.set(i, p * t.x - q * t.y);
            x1.set(i, p * t.y + q * t.x);
        }
    }
}

// Rows of a token: its query heads, key heads, value heads.  A row is ns = head_dim / 2V slots of two chunks; a
// thread keeps one slot, so its place in a row and its pairs are fixed, and walks over the rows of the CTA's
// tokens.  The (cos, sin) of a token are computed once per CTA, not once per head.
template <typename T, int VB, bool INTERLEAVED>
__global__ void __launch_bounds__(kRopeThreads) rope_write_kv_kernel(const RopeWriteArgs a, int tokens_per_cta) {
    constexpr int V = Chunk<T, VB>::V;
    extern __shared__ float2 cs[];  // [tokens][rotary_dim / 2]
    __shared__ long long dest[kRopeTokens];
    griddep_wait();
    griddep_launch_dependents();
    const RopeArgs& r = a.r;
    const int half = r.rotary_dim / 2, tid = threadIdx.x;
    const int tok0 = blockIdx.x * tokens_per_cta, ntok = min(tokens_per_cta, r.num_tokens - tok0);
    for (int i = tid; i < ntok * half; i += kRopeThreads) {
        const int t = i / half;
        cs[i] = turn(turn_step(r.inv_freq[i - t * half]), a.positions[tok0 + t], r.factor);
    }
    if (tid < ntok) {
        const long long slot = a.slot_mapping[tok0 + tid];
        long long d = -1;  // in rows of the cache, without the head
        if (slot >= (long long)r.num_blocks * r.block_size) {
            atomicOr(r.err, kErrBadSlot);
        } else if (slot >= 0) {
            const long long blk = slot / r.block_size;
            d = blk * r.num_kv_heads * r.block_size + (slot - blk * r.block_size);
        }
        dest[tid] = d;
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

constexpr int kAppendThreads = 128;
constexpr float kScaleFloor = 7.888609052210118e-31f;  // 2^-100: the scale of a block of zeros

__device__ __forceinline__ uint16_t to_codes(float a, float b) {
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// One unit: the rows of the call that fall into one block of one request, one kv head, K or V.  A warp holds them
// in float32, D / 4 lanes to a row: (2p, 2p + 1) and their partners of two pairs (half layout), or four neighbours.
template <typename T, int D, int BS>
__device__ __forceinline__ void append_unit(const RopeAppendArgs& a, int tok, int n, int off, int pos, long long blk, int h,
                                            bool is_value, int lane) {
    constexpr int LPR = D / 4, RPS = 32 / LPR, STEPS = BS / RPS;
    const RopeArgs& r = a.r;
    const int l = lane % LPR, sub = lane / LPR;
    const int half = r.rotary_dim / 2;
    const T* src = is_value ? static_cast<const T*>(r.value) + h * D + (long long)tok * r.v_stride
                            : static_cast<const T*>(r.key) + h * D + (long long)tok * r.k_stride;
    const long long stride = is_value ? r.v_stride : r.k_stride;
    // element places of this lane: e, e + 1 and f, f + 1
    int e = 4 * l, f = 4 * l + 2;
    const bool turns = !is_value && 4 * l < r.rotary_dim;
    if (turns && !r.interleaved) {
        e = 2 * l;
        f = 2 * l + half;
    }
    uint64_t s0 = 0, s1 = 0;
    if (turns) {  // pairs 2l and 2l + 1 in either layout
        s0 = turn_step(r.inv_freq[2 * l]);
        s1 = turn_step(r.inv_freq[2 * l + 1]);
    }
    float x[STEPS][4];
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int row = i * RPS + sub;
#pragma unroll
        for (int k = 0; k < 4; ++k) x[i][k] = 0.f;
        if (row < n) {
            const T* p = src + row * stride;
            x[i][0] = to_float(p[e]);
            x[i][1] = to_float(p[e + 1]);
            x[i][2] = to_float(p[f]);
            x[i][3] = to_float(p[f + 1]);
        }
    }
    const size_t si = (size_t)blk * r.num_kv_heads + h;
    float* scale_at = (is_value ? a.v_scale : a.k_scale) + si;
    const float held = off > 0 ? *scale_at : 0.f;  // a block that starts here has no scale yet
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int row = i * RPS + sub;
        if (turns && row < n) {
            const float2 t0 = turn(s0, pos + row, r.factor), t1 = turn(s1, pos + row, r.factor);
            float *p0, *q0, *p1, *q1;
            if (r.interleaved) {
                p0 = &x[i][0], q0 = &x[i][1], p1 = &x[i][2], q1 = &x[i][3];
            } else {
                p0 = &x[i][0], q0 = &x[i][2], p1 = &x[i][1], q1 = &x[i][3];
            }
            const float u = *p0 * t0.x - *q0 * t0.y, v = *p0 * t0.y + *q0 * t0.x;
            const float w = *p1 * t1.x - *q1 * t1.y, z = *p1 * t1.y + *q1 * t1.x;
            *p0 = u, *q0 = v, *p1 = w, *q1 = z;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float m = fabsf(x[i][k]);
            if (m <= 3.402823466e38f) most = fmaxf(most, m);  // infinities saturate, NaN stays: neither sets a scale
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    const float scale = fmaxf(fmaxf(held, most / 448.f), kScaleFloor);
    const bool both = a.value_cache == nullptr;
    uint8_t* base = both ? a.key_cache + (si * 2 + (is_value ? 1 : 0)) * BS * D
                         : (is_value ? a.value_cache : a.key_cache) + si * BS * D;
    if (scale > held && off > 0) {  // the codes that the block holds already, in the larger scale
        for (int i = lane; i < off * (D / 4); i += 32) {
            uint32_t* w = reinterpret_cast<uint32_t*>(base) + i;
            const uint32_t c = *w;
            const float2 lo = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xffffu), __NV_E4M3)));
            const float2 hi = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> 16), __NV_E4M3)));
            *w = (uint32_t)to_codes(lo.x * held / scale, lo.y * held / scale) |
                 ((uint32_t)to_codes(hi.x * held / scale, hi.y * held / scale) << 16);
        }
    }
#pragma unroll
    for (int i = 0; i < STEPS; ++i) {
        const int row = i * RPS + sub;
        if (row < n) {
            uint8_t* p = base + (off + row) * D;
            *reinterpret_cast<uint16_t*>(p + e) = to_codes(x[i][0] / scale, x[i][1] / scale);
            *reinterpret_cast<uint16_t*>(p + f) = to_codes(x[i][2] / scale, x[i][3] / scale);
        }
    }
    __syncwarp();
    if (lane == 0 && scale != held) *scale_at = scale;
}

// CTAs [0, kv_ctas): warps over (window of `window` tokens, kv head, K or V), each owning the blocks whose first
// row of this call lies in its window.  The others: a warp per token's query heads.
template <typename T, int D, int BS>
__global__ void __launch_bounds__(kAppendThreads) rope_append_fp8_kernel(const RopeAppendArgs a, int kv_ctas, int window) {
    griddep_wait();
    griddep_launch_dependents();
    const RopeArgs& r = a.r;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int B = a.num_seqs;
    if ((int)blockIdx.x < kv_ctas) {
        long long w = (long long)blockIdx.x * (kAppendThreads / 32) + warp;
        const bool is_value = w & 1;
        w >>= 1;
        const int h = (int)(w % r.num_kv_heads);
        const long long win = w / r.num_kv_heads;
        long long t = win * window;
        const int end = (int)min((long long)r.num_tokens, (win + 1) * window);
        while (t < end) {
            const int b = warp_find(a.q_offsets, B + 1, (int)t, lane);
            if (b < 0 || b >= B) return;  // rows behind the last request
            const int first = a.q_offsets[b], last = min(a.q_offsets[b + 1], r.num_tokens), L = a.context_lens[b];
            const long long start = (long long)L - ((long long)a.q_offsets[b + 1] - first);  // position of its first row
            if (start < 0 || L > (long long)a.max_blocks * BS) {
                if (lane == 0 && t == first) atomicOr(r.err, kErrBadContext);
                t = last;
                continue;
            }
            const int pos = (int)(start + (t - first)), off = pos % BS;
            if (t != first && off != 0) {  // the block belongs to an earlier window
                t += BS - off;
                if (t > last) t = last;
                continue;
            }
            const int n = min(BS - off, last - (int)t);
            const long long blk = a.block_tables[(size_t)b * a.max_blocks + pos / BS];
            if (blk < 0 || blk >= r.num_blocks) {
                if (lane == 0) atomicOr(r.err, kErrBadTable);
            } else {
                append_unit<T, D, BS>(a, (int)t, n, off, pos, blk, h, is_value, lane);
            }
            t += n;
        }
        return;
    }
    // query rows: lanes as in append_unit
    constexpr int LPR = D / 4, RPS = 32 / LPR;
    const int t = (int)(((long long)blockIdx.x - kv_ctas) * (kAppendThreads / 32) + warp);
    if (t >= r.num_tokens) return;
    const int b = warp_find(a.q_offsets, B + 1, t, lane);
    if (b < 0 || b >= B) return;
    const int pos = a.context_lens[b] - (a.q_offsets[b + 1] - t);
    const int l = lane % LPR, sub = lane / LPR, half = r.rotary_dim / 2;
    const bool turns = 4 * l < r.rotary_dim;
    int e = 4 * l, f = 4 * l + 2;
    if (turns && !r.interleaved) {
        e = 2 * l;
        f = 2 * l + half;
    }
    float2 t0 = make_float2(1.f, 0.f), t1 = t0;
    if (turns) {
        t0 = turn(turn_step(r.inv_freq[2 * l]), pos, r.factor);
        t1 = turn(turn_step(r.inv_freq[2 * l + 1]), pos, r.factor);
    }
    const T* src = static_cast<const T*>(r.query) + (long long)t * r.q_stride;
    T* dst = static_cast<T*>(r.query_out) + (long long)t * r.num_heads * D;
#pragma unroll 4
    for (int h = sub; h < r.num_heads; h += RPS) {
        T y[4] = {src[h * D + e], src[h * D + e + 1], src[h * D + f], src[h * D + f + 1]};
        if (turns) {
            const float x0 = to_float(y[0]), x1 = to_float(y[1]), x2 = to_float(y[2]), x3 = to_float(y[3]);
            if (r.interleaved) {
                y[0] = from_float<T>(x0 * t0.x - x1 * t0.y), y[1] = from_float<T>(x0 * t0.y + x1 * t0.x);
                y[2] = from_float<T>(x2 * t1.x - x3 * t1.y), y[3] = from_float<T>(x2 * t1.y + x3 * t1.x);
            } else {
                y[0] = from_float<T>(x0 * t0.x - x2 * t0.y), y[2] = from_float<T>(x0 * t0.y + x2 * t0.x);
                y[1] = from_float<T>(x1 * t1.x - x3 * t1.y), y[3] = from_float<T>(x1 * t1.y + x3 * t1.x);
            }
        }
        dst[h * D + e] = y[0], dst[h * D + e + 1] = y[1], dst[h * D + f] = y[2], dst[h * D + f + 1] = y[3];
    }
}

bool multiple(const void* p, long long bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0; }

template <typename T, int VB>
cudaError_t rope_write_typed(const RopeWriteArgs& a, cudaStream_t stream) {
    // Four tokens share a CTA when that still fills the GPU; few tokens take a CTA each.
    const int per = a.r.num_tokens >= 4096 ? kRopeTokens : 1;
    const unsigned grid = (unsigned)((a.r.num_tokens + per - 1) / per);
    const size_t smem = (size_t)per * (a.r.rotary_dim / 2) * sizeof(float2);
    if (a.r.interleaved)
        return launch_pdl(rope_write_kv_kernel<T, VB, true>, dim3(grid), dim3(kRopeThreads), smem, stream, a, per);
    return launch_pdl(rope_write_kv_kernel<T, VB, false>, dim3(grid), dim3(kRopeThreads), smem, stream, a, per);
}

// Whether a row splits into chunks of vb bytes: aligned bases and strides, and slots of two chunks that do not
// straddle the end of the pairs.
bool rope_splits(const RopeWriteArgs& a, int eb, int vb) {
    const RopeArgs& r = a.r;
    const int v = vb / eb;
    if (r.head_dim % (2 * v) || r.head_dim / (2 * v) > kRopeThreads || (r.rotary_dim / 2) % v) return false;
    if ((r.head_dim - r.rotary_dim) % (2 * v)) return false;
    for (const void* p : {(const void*)r.query_out, r.query, r.key, r.value, (const void*)a.key_cache, (const void*)a.value_cache})
        if (!multiple(p, vb)) return false;
    return (r.q_stride * eb) % vb == 0 && (r.k_stride * eb) % vb == 0 && (r.v_stride * eb) % vb == 0;
}

template <typename T, int D, int BS>
cudaError_t append_typed(const RopeAppendArgs& a, cudaStream_t stream) {
    const RopeArgs& r = a.r;
    constexpr int warps = kAppendThreads / 32;
    // A window is a block long, so that a prompt has one unit per window; while one window per token does not
    // fill the GPU, every token has its own, so that the units of a decode step do not queue behind one another.
    const long long per_token = (long long)r.num_tokens * r.num_kv_heads * 2;
    const int window = per_token <= (long long)a.num_sms * warps * 4 ? 1 : BS;
    const long long kv_warps = (long long)((r.num_tokens + window - 1) / window) * r.num_kv_heads * 2;
    const long long kv_ctas = (kv_warps + warps - 1) / warps;
    const long long q_ctas = (r.num_tokens + warps - 1) / warps;
    return launch_pdl(rope_append_fp8_kernel<T, D, BS>, dim3((unsigned)(kv_ctas + q_ctas)), dim3(kAppendThreads), 0, stream,
                      a, (int)kv_ctas, window);
}

template <typename T>
cudaError_t append_dispatch(const RopeAppendArgs& a, cudaStream_t stream) {
    const int d = a.r.head_dim, bs = a.r.block_size;
    if (d == 128 && bs == 16) return append_typed<T, 128, 16>(a, stream);
    if (d == 128 && bs == 32) return append_typed<T, 128, 32>(a, stream);
    if (d == 64 && bs == 16) return append_typed<T, 64, 16>(a, stream);
    if (d == 64 && bs == 32) return append_typed<T, 64, 32>(a, stream);
    return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t rope_write_kv_launch(const RopeWriteArgs& a, cudaStream_t stream) {
    const int eb = a.r.dtype == 0 ? 4 : 2;
    if (a.r.dtype == 0)
        return rope_splits(a, eb, 16) ? rope_write_typed<float, 16>(a, stream) : rope_write_typed<float, 4>(a, stream);
    const int vb = rope_splits(a, eb, 16) ? 16 : rope_splits(a, eb, 4) ? 4 : 2;
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
        case 0: return append_dispatch<float>(a, stream);
        case 1: return append_dispatch<__half>(a, stream);
        default: return append_dispatch<__nv_bfloat16>(a, stream);
    }
}

}  // namespace pa
