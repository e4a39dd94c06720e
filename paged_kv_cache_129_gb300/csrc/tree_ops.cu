// Drafted trees of a speculative step: which nodes a node sees, which of them the target confirms, and the confirmed branch
// moved together in the caches.
//
// Request b has the nodes q_offsets[b] .. q_offsets[b + 1] - 1; parents[t] < the node's own index is the index, in the request, of its
// parent (-1: a root).  With a(i) the set of i and its ancestors:
//   masks     bit j of node i's words is set where j is in a(i); position = cached tokens + |a(i)| - 1;
//   accept    the path from node 0 that always goes to the first child whose token is the target's choice at the node;
//   compact   with accepted nodes a_0 < a_1 < .. (so a_j >= j), K and V of node a_j go to the slot of node j, in every layer; the
//             request keeps its cached tokens and the accepted ones, blocks behind them go back on the stack.
// The first two move a few bytes per node: launch and dependent reads bound them (on the GPU, 64 trees of 16 nodes: masks 3.9 us, acceptance 4.6;
// 256 trees of up to 200 nodes: 8.5 and 5.7).
#include <algorithm>
#include <climits>
#include <cstdint>

#include "pa_common.cuh"
#include "tree_ops.h"

namespace pa {

namespace {

// A request's nodes: none if its offsets are no run, or are more than a tree may have.
__device__ __forceinline__ int nodes_of(const int32_t* q_offsets, int b, int num_tokens, int most, int* first, bool* bad) {
    const int lo = q_offsets[b], hi = q_offsets[b + 1];
    *first = lo;
    *bad = !is_run(lo, hi, num_tokens) || hi - lo > most;
    return *bad ? 0 : hi - lo;
}

// ---- masks -------------------------------------------------------------------------------------------

constexpr int kMaskThreads = 128;

// A CTA per request, a thread per node: the ancestors of a node come in descending order, so a thread fills one word after the other,
// from the last, and writes each once.  Nodes whose parent is the one before them form runs, cut at multiples of 32 (so that one lies in one
// word); a thread takes a run at a time: long chains are not followed node by node.  The CTA behind the last request clears the rows behind its
// nodes.
__global__ void __launch_bounds__(kMaskThreads) tree_masks_kernel(const TreeMaskArgs a) {
    __shared__ int parent[kMaxTreeNodes], run[kMaxTreeNodes];  // a node's parent; the first node of its run
    griddep_wait();
    griddep_launch_dependents();
    const int b = blockIdx.x, W = a.mask_words;
    if (b == a.num_seqs) {
        const int end = max(0, min(a.q_offsets[b], a.num_tokens));
        for (long long i = (long long)end * W + threadIdx.x; i < (long long)a.num_tokens * W; i += kMaskThreads) a.tree_mask[i] = 0;
        for (int t = end + threadIdx.x; t < a.num_tokens; t += kMaskThreads) a.positions[t] = 0;
        return;
    }
    int first;
    bool bad;
    const int n = nodes_of(a.q_offsets, b, a.num_tokens, min(kMaxTreeNodes, 64 * W), &first, &bad);
    const int cached = a.context_lens[b] - n;
    if (cached < 0) bad = true;
    for (int i = threadIdx.x; i < (n + 31) / 32 * 32; i += kMaskThreads) {  // (whole warps)
        int p = i < n ? a.parents[first + i] : -1;
        if (p < -1 || p >= i) bad = bad || i < n, p = -1;  // (a node without a parent before it is a root)
        const unsigned starts = __ballot_sync(0xffffffffu, p != i - 1 || i % 32 == 0);
        parent[i] = p;
        run[i] = (i & ~31) + 31 - __clz(starts & (0xffffffffu >> (31 - i % 32)));
    }
    if (bad) atomicOr(a.err, kErrBadContext);
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kMaskThreads) {
        int64_t* row = a.tree_mask + (long long)(first + i) * W;
        int node = i, depth = 0;
        for (int w = W - 1; w >= 0; --w) {
            unsigned long long word = 0;
            while (node >= 64 * w) {
                const int from = run[node];
                word |= (~0ull >> (63 - (node - from))) << (from - 64 * w);
                depth += node - from + 1;
                node = parent[from];
            }
            row[w] = (int64_t)word;
        }
        a.positions[first + i] = max(0, cached) + depth - 1;
    }
}

// ---- acceptance ----------------------------------------------------------------------------------------

constexpr int kAcceptThreads = 128;

// A CTA per request: every node bids for its parent's step, the first child wins; one thread then follows the steps.
template <typename Token>
__global__ void __launch_bounds__(kAcceptThreads) accept_tree_kernel(const AcceptArgs a) {
    __shared__ int next[kMaxTreeNodes];
    griddep_wait();
    griddep_launch_dependents();
    const int b = blockIdx.x;
    const Token* tokens = static_cast<const Token*>(a.tokens);
    const Token* choices = static_cast<const Token*>(a.choices);
    int first;
    bool bad;
    const int n = nodes_of(a.q_offsets, b, a.num_tokens, kMaxTreeNodes, &first, &bad);
    for (int i = threadIdx.x; i < n; i += kAcceptThreads) next[i] = INT_MAX;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kAcceptThreads) {
        const int p = a.parents[first + i];
        if (p < -1 || p >= i || (i == 0 && p != -1)) bad = true;
        if (p >= 0 && p < i && tokens[first + i] == choices[first + p]) atomicMin(&next[p], i);
    }
    if (bad) atomicOr(a.err, kErrBadContext);
    __syncthreads();
    if (threadIdx.x != 0) return;
    int32_t* row = a.accepted + (long long)b * a.max_accepted;
    int count = 0, last = -1;
    for (int node = n > 0 ? 0 : INT_MAX; node != INT_MAX && count < a.max_accepted; node = next[node]) {
        row[count++] = node;
        last = node;
    }
    for (int j = count; j < a.max_accepted; ++j) row[j] = -1;
    a.num_accepted[b] = count;
    static_cast<Token*>(a.next_tokens)[b] = last >= 0 ? choices[first + last] : (Token)-1;
}

// ---- compaction ----------------------------------------------------------------------------------------

constexpr int kCompactThreads = 256, kCompactCtasPerSm = 16;

// Whether request b's accepted nodes are some of its n nodes in ascending order.  Any number of threads, each for itself.
__device__ __forceinline__ bool is_path(const CompactArgs& a, int b, int n, int count) {
    if (count < 0 || count > n || count > a.max_accepted) return false;
    int before = -1;
    bool ok = true;
#pragma unroll 4
    for (int j = 0; j < count; ++j) {  // (loads that do not wait for the comparisons)
        const int node = a.accepted[(long long)b * a.max_accepted + j];
        ok = ok && node > before && node < n;
        before = node;
    }
    return ok;
}

// New lengths, and the blocks given back: one CTA, a contiguous run of requests per thread.
__device__ __forceinline__ void trim(const CompactArgs& a) {
    __shared__ int sums[kCompactThreads + 1];
    const int tid = threadIdx.x, B = a.num_seqs, bs = a.block_size;
    const int per = (B + kCompactThreads - 1) / kCompactThreads, b0 = min(B, tid * per), b1 = min(B, b0 + per);
    const int free0 = *a.num_free;
    unsigned bits = 0;
    // blocks that request b gives back, from which on; -1: it keeps its length
    auto give = [&](int b, int* keep, int* length) {
        int first;
        bool bad;
        const int n = nodes_of(a.q_offsets, b, a.num_tokens, INT_MAX, &first, &bad), L = a.context_lens[b], k = a.num_accepted[b];
        *length = L;
        if (bad || L < n || L > (long long)a.max_blocks * bs || !is_path(a, b, n, k)) {
            bits |= kErrBadContext;
            return -1;
        }
        *keep = (int)(((long long)L - n + k + bs - 1) / bs);
        const int had = (int)(((long long)L + bs - 1) / bs);
        for (int j = *keep; j < had; ++j) {
            const int id = a.block_tables[(long long)b * a.max_blocks + j];
            if (id < 0 || id >= a.num_blocks) {
                bits |= kErrBadTable;
                return -1;
            }
        }
        *length = L - n + k;
        return had - *keep;
    };
    int keep = 0, length = 0, gives = 0, mine = 0;  // (of one request per thread, as nearly always, kept until it is written)
    for (int b = b0; b < b1; ++b) {
        gives = give(b, &keep, &length);
        mine += max(0, gives);
    }
    if (tid == 0) sums[0] = 0;
    sums[tid + 1] = mine;
    __syncthreads();
    if (tid < 32) {  // a run of the threads' sums per lane
        constexpr int kRun = kCompactThreads / 32;
        int sum = 0;
#pragma unroll
        for (int i = 0; i < kRun; ++i) sum += sums[tid * kRun + i + 1];
        int before = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, before, o);
            if (tid >= o) before += x;
        }
        before -= sum;
#pragma unroll
        for (int i = 0; i < kRun; ++i) sums[tid * kRun + i + 1] = before += sums[tid * kRun + i + 1];
    }
    __syncthreads();
    const int total = sums[kCompactThreads];
    const bool room = free0 >= 0 && (long long)free0 + total <= a.num_blocks;
    if (!room) bits |= kErrBadTable;
    int at = free0 + sums[tid];
    for (int b = b0; b < b1; ++b) {
        if (per > 1) gives = give(b, &keep, &length);
        if (room)
            for (int j = 0; j < gives; ++j) a.free_blocks[at++] = a.block_tables[(long long)b * a.max_blocks + keep + j];
        a.context_lens_out[b] = room ? length : a.context_lens[b];
    }
    if (tid == 0) *a.num_free_out = room ? free0 + total : free0;
    if (bits) atomicOr(a.err, bits);
}

// Row (node a_j, layer, K or V, kv head) goes to the place of node j, for the nodes that are not there already: those behind the first that is
// not.  CTA (request, part of its rows); a thread has columns of sizeof(Vec) bytes and takes the nodes in order, kCompactBatch at a time:
// a node's place is written behind every read of it, since a_j >= j.  CTA 0 has the lengths and the blocks.
// The rows are 64 - 512 bytes here and there, each read and written once: HBM bounds many requests, latency few (28 layers of 4 heads of 128, bf16,
// on the GPU: 256 requests with up to 16 accepted nodes 19 us, 64 with up to 5 7.2 us; a CTA per request and a node at a time 168 and 51).
constexpr int kCompactBatch = 8;
template <typename Vec>
__global__ void __launch_bounds__(kCompactThreads) compact_tree_kernel(const CompactArgs a, const __grid_constant__ CachePtrs caches, int parts) {
    __shared__ long long from[kMaxTreeNodes], to[kMaxTreeNodes];  // bytes, of kv head 0
    __shared__ int moving[kCompactThreads / 32];
    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x == 0) {
        trim(a);
        return;
    }
    const int b = (blockIdx.x - 1) / parts, part = (blockIdx.x - 1) - b * parts, H = a.num_kv_heads, bs = a.block_size, tid = threadIdx.x;
    int first;
    bool bad;
    const int n = nodes_of(a.q_offsets, b, a.num_tokens, INT_MAX, &first, &bad), count = a.num_accepted[b];
    if (bad || count <= 0 || count > n || count > a.max_accepted) return;
    const long long slots = (long long)a.num_blocks * bs;
    const int32_t* path = a.accepted + (long long)b * a.max_accepted;
    bool wrong = false;
    int still = 0;  // nodes that are in their place
    for (int j = tid; j < count; j += kCompactThreads) {
        const int node = path[j], before = j > 0 ? path[j - 1] : -1;
        wrong |= node <= before || node >= n;
        if (wrong) break;
        still += node == j;
        long long at[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const long long slot = a.slot_mapping[first + (k ? j : node)];
            const long long blk = slot >= 0 ? slot / bs : 0;
            at[k] = slot < 0 || slot >= slots ? -1 : (blk * H * bs + (slot - blk * bs)) * a.row_bytes;
        }
        if (at[0] < 0 || at[1] < 0) {
            if (node != j) atomicOr(a.err, kErrBadSlot);
            at[0] = -1;
        }
        from[j] = at[0];
        to[j] = at[1];
    }
    if (__syncthreads_or(wrong)) return;
    still = __reduce_add_sync(0xffffffffu, still);
    if ((tid & 31) == 0) moving[tid >> 5] = still;
    __syncthreads();
    still = 0;
#pragma unroll
    for (int w = 0; w < kCompactThreads / 32; ++w) still += moving[w];
    if (still == count) return;
    const int columns = a.row_bytes / (int)sizeof(Vec), items = 2 * a.num_layers * H * columns;
    for (int x = part * kCompactThreads + tid; x < items; x += parts * kCompactThreads) {
        const int unit = x / columns, column = x - unit * columns, cache = unit / H, h = unit - cache * H;
        char* base = (cache & 1 ? caches.value[cache >> 1] : caches.key[cache >> 1]) + (long long)h * bs * a.row_bytes + column * (int)sizeof(Vec);
        for (int j0 = still; j0 < count; j0 += kCompactBatch) {
            Vec v[kCompactBatch];
#pragma unroll
            for (int k = 0; k < kCompactBatch; ++k)
                if (j0 + k < count && from[j0 + k] >= 0) v[k] = *reinterpret_cast<const Vec*>(base + from[j0 + k]);
#pragma unroll
            for (int k = 0; k < kCompactBatch; ++k)
                if (j0 + k < count && from[j0 + k] >= 0) *reinterpret_cast<Vec*>(base + to[j0 + k]) = v[k];
        }
    }
}

}  // namespace

cudaError_t tree_masks_launch(const TreeMaskArgs& a, cudaStream_t stream) {
    return launch_pdl(tree_masks_kernel, dim3((unsigned)a.num_seqs + 1), dim3(kMaskThreads), 0, stream, a);
}

cudaError_t accept_tree_launch(const AcceptArgs& a, cudaStream_t stream) {
    if (a.token_bytes == 4)
        return launch_pdl(accept_tree_kernel<int32_t>, dim3((unsigned)a.num_seqs), dim3(kAcceptThreads), 0, stream, a);
    return launch_pdl(accept_tree_kernel<int64_t>, dim3((unsigned)a.num_seqs), dim3(kAcceptThreads), 0, stream, a);
}

cudaError_t compact_tree_launch(const CompactArgs& a, const CachePtrs& caches, cudaStream_t stream) {
    const int vec = a.vector ? 16 : a.elem_bytes;
    // Parts of a request's rows: about kCompactCtasPerSm CTAs to an SM, but a column for every thread at least.
    const long long items = 2ll * a.num_layers * a.num_kv_heads * (a.row_bytes / vec), most = (items + kCompactThreads - 1) / kCompactThreads;
    const long long wanted = a.num_seqs ? ((long long)kCompactCtasPerSm * a.num_sms + a.num_seqs - 1) / a.num_seqs : 1;
    const int parts = (int)std::max(1ll, std::min(most, wanted));
    const dim3 grid((unsigned)(1 + (long long)a.num_seqs * parts)), block(kCompactThreads);
    if (a.vector) return launch_pdl(compact_tree_kernel<uint4>, grid, block, 0, stream, a, caches, parts);
    if (a.elem_bytes == 4) return launch_pdl(compact_tree_kernel<uint32_t>, grid, block, 0, stream, a, caches, parts);
    return launch_pdl(compact_tree_kernel<uint16_t>, grid, block, 0, stream, a, caches, parts);
}

}  // namespace pa
