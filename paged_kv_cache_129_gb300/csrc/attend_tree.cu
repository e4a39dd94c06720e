// Attention of the nodes of drafted trees over a paged 16-bit cache.
//
// Request b has the rows q_offsets[b] .. q_offsets[b + 1] - 1, n_b nodes whose keys and values are the last n_b of its L_b positions.  A
// row sees the L_b - n_b positions before them, and node j where bit j of its words of tree_mask is set:
//     out = sum softmax(scale q k_j) v_j over what it sees; zeros where that is nothing.
#include <algorithm>
#include <cstdint>

#include "pa_common.cuh"
#include "tree_ops.h"

namespace pa {

namespace {

constexpr int kThreads = 256;

// A warp per (row, query head), a key at a time; maximum, sum and output in float32 registers.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) attend_tree_kernel(const TreeAttendArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, group = a.num_heads / a.num_kv_heads;
    const int b = blockIdx.y;
    const int lo = a.q_offsets[b], hi = a.q_offsets[b + 1], width = a.max_blocks * a.block_size;
    int L = a.context_lens[b];
    const bool run = is_run(lo, hi, a.num_tokens);
    const int n = run ? hi - lo : 0;
    if ((!run || L < n || L > width || n > 64 * a.mask_words) && blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.err, kErrBadContext);
    L = max(0, min(L, width));
    const long long rows = (long long)n * a.num_heads;
    for (long long x = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); x < rows; x += gridDim.x * (kThreads / 32)) {
        const int t = lo + (int)(x / a.num_heads), h = (int)(x % a.num_heads), kvh = h / group;
        const T* q = static_cast<const T*>(a.query) + ((long long)t * a.num_heads + h) * D + lane * E;
        float qf[E], o[E], m = -INFINITY, l = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) qf[i] = to_float(q[i]) * a.scale, o[i] = 0.f;
        for (int p = 0; p < L; ++p) {
            const int node = p - (L - n);
            if (node >= 0 && (node >= 64 * a.mask_words || !(a.tree_mask[(long long)t * a.mask_words + node / 64] >> (node % 64) & 1)))
                continue;
            const int id = a.block_tables[(long long)b * a.max_blocks + p / a.block_size];
            if (id < 0 || id >= a.num_blocks) {
                if (lane == 0) atomicOr(a.err, kErrBadTable);
                continue;
            }
            const long long at = (((long long)id * a.num_kv_heads + kvh) * a.block_size + p % a.block_size) * D + lane * E;
            const T *k = static_cast<const T*>(a.key_cache) + at, *v = static_cast<const T*>(a.value_cache) + at;
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) s = fmaf(qf[i], to_float(k[i]), s);
#pragma unroll
            for (int w = 16; w > 0; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
            const float mn = fmaxf(m, s), f = m == -INFINITY ? 0.f : __expf(m - mn), e = s == -INFINITY ? 0.f : __expf(s - mn);
            m = mn;
            l = l * f + e;
#pragma unroll
            for (int i = 0; i < E; ++i) o[i] = o[i] * f + e * to_float(v[i]);
        }
        T* out = static_cast<T*>(a.out) + ((long long)t * a.num_heads + h) * D + lane * E;
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int i = 0; i < E; ++i) out[i] = from_float<T>(o[i] * inv);
    }
}

template <typename T, int D>
cudaError_t attend_typed(const TreeAttendArgs& a, cudaStream_t stream) {
    const long long most = ((long long)a.num_tokens * a.num_heads + 7) / 8;  // of one request
    return launch_pdl(attend_tree_kernel<T, D>, dim3((unsigned)std::min(most, 128ll), (unsigned)a.num_seqs), dim3(kThreads), 0, stream, a);
}

}  // namespace

size_t attend_tree_workspace_bytes(int, int, int, int, int, int) { return 0; }

cudaError_t attend_tree_launch(const TreeAttendArgs& a, cudaStream_t stream) {
    if (a.dtype == 1) return a.head_dim == 64 ? attend_typed<__half, 64>(a, stream) : attend_typed<__half, 128>(a, stream);
    return a.head_dim == 64 ? attend_typed<__nv_bfloat16, 64>(a, stream) : attend_typed<__nv_bfloat16, 128>(a, stream);
}

}  // namespace pa
