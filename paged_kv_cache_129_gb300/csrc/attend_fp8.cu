// Causal attention of ragged runs of new tokens over an FP8 (E4M3) paged cache.
//
// Request b has the rows q_offsets[b] .. q_offsets[b + 1] - 1, the last n_b positions of its L_b; the row at
// position p attends positions 0 .. p:  out = sum softmax(scale q k_j) v_j, with k_j, v_j = code * scale(block, head).
#include <cstdint>

#include <cuda_fp8.h>

#include "pa_common.cuh"
#include "step_ops.h"

namespace pa {

namespace {

// A warp per (token, query head): the running maximum and sum in float32, D / 32 elements of the head per lane.
template <typename T, int D>
__global__ void __launch_bounds__(128) attend_fp8_kernel(const AttendArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    if (w >= (long long)a.num_tokens * a.num_heads) return;
    const int t = (int)(w / a.num_heads), qh = (int)(w - (long long)t * a.num_heads);
    int lo = -1, hi = a.num_seqs + 1;  // off[lo] <= t < off[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.q_offsets[mid] <= t)
            lo = mid;
        else
            hi = mid;
    }
    if (lo < 0 || lo >= a.num_seqs) return;  // behind the last request
    const int kvh = qh / (a.num_heads / a.num_kv_heads), bs = a.block_size;
    int L = a.context_lens[lo];
    if (L < 0 || L > a.max_blocks * bs) {
        if (lane == 0) atomicOr(a.err, kErrBadContext);
        L = max(0, min(L, a.max_blocks * bs));
    }
    const int seen = L - (a.q_offsets[lo + 1] - t) + 1;
    float q[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        q[i] = to_float(static_cast<const T*>(a.query)[((size_t)t * a.num_heads + qh) * D + lane * E + i]) * a.scale;
        o[i] = 0.f;
    }
    const bool both = a.value_cache == nullptr;
    for (int p = 0; p < seen; ++p) {
        const int blk = a.block_tables[(size_t)lo * a.max_blocks + p / bs];
        if (blk < 0 || blk >= a.num_blocks) {
            if (lane == 0) atomicOr(a.err, kErrBadTable);
            continue;
        }
        const size_t si = (size_t)blk * a.num_kv_heads + kvh;
        const uint8_t* k = a.key_cache + ((both ? 2 * si : si) * bs + p % bs) * D + lane * E;
        const uint8_t* v = both ? k + (size_t)bs * D : a.value_cache + (si * bs + p % bs) * D + lane * E;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) s += q[i] * __half2float(__half(__nv_cvt_fp8_to_halfraw(k[i], __NV_E4M3)));
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= a.k_scale[si];
        const float mn = fmaxf(m, s), f = __expf(m - mn), e = __expf(s - mn), ev = e * a.v_scale[si];
        m = mn;
        l = l * f + e;
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = o[i] * f + ev * __half2float(__half(__nv_cvt_fp8_to_halfraw(v[i], __NV_E4M3)));
    }
#pragma unroll
    for (int i = 0; i < E; ++i)
        static_cast<T*>(a.out)[((size_t)t * a.num_heads + qh) * D + lane * E + i] = from_float<T>(l == 0.f ? 0.f : o[i] / l);
}

template <typename T, int D>
cudaError_t attend_typed(const AttendArgs& a, cudaStream_t stream) {
    const long long warps = (long long)a.num_tokens * a.num_heads;
    return launch_pdl(attend_fp8_kernel<T, D>, dim3((unsigned)((warps + 3) / 4)), dim3(128), 0, stream, a);
}

}  // namespace

size_t attend_fp8_workspace_bytes(int, int, int, int, int, int, int, int) { return 0; }

cudaError_t attend_fp8_launch(const AttendArgs& a, cudaStream_t stream) {
    if (a.dtype == 1) return a.head_dim == 128 ? attend_typed<__half, 128>(a, stream) : attend_typed<__half, 64>(a, stream);
    return a.head_dim == 128 ? attend_typed<__nv_bfloat16, 128>(a, stream) : attend_typed<__nv_bfloat16, 64>(a, stream);
}

}  // namespace pa
