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

// CTAs per SM of the rows' parts: 256 requests of 28 layers (see below) 15.8 us with 12, 16.6 with 10, 16.9 with 16.
constexpr int kCompactThreads = 256, kCompactCtasPerSm = 12;

// Whether request b's accepted nodes are some of its n nodes in ascending order.  Any number of threads, each for itself.
__device__ __forceinline__ bool is_path(const CompactArgs& a, int b, int n, int count) {
    if (count < 0 || count > n || count > a.max_accepted) return false;
    const int32_t* path = a.accepted + (long long)b * a.max_accepted;
    constexpr int kAtOnce = 8;
    int before = -1;
    bool ok = true;
    for (int j0 = 0; j0 < count; j0 += kAtOnce) {
        int node[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) node[k] = j0 + k < count ? path[j0 + k] : INT_MAX;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            ok = ok && (j0 + k >= count || (node[k] > before && node[k] < n));
            before = node[k];
        }
    }
    return ok;
}

__device__ __forceinline__ int blocks_of(int positions, int block_size) { return (int)(((unsigned)positions + block_size - 1) / (unsigned)block_size); }

// What becomes of request b: its new length, and how many blocks from which on go back; gives -1: it is left as it is, with these errors.
struct Rest {
    int length, keep, gives;
    unsigned errors;
};
__device__ __forceinline__ Rest rest_of(const CompactArgs& a, int b) {
    int first;
    bool bad;
    const int n = nodes_of(a.q_offsets, b, a.num_tokens, INT_MAX, &first, &bad), L = a.context_lens[b], k = a.num_accepted[b], bs = a.block_size;
    if (bad || L < n || L > (long long)a.max_blocks * bs || !is_path(a, b, n, k)) return Rest{L, 0, -1, kErrBadContext};
    const int keep = blocks_of(L - n + k, bs), had = blocks_of(L, bs);
    const int32_t* table = a.block_tables + (long long)b * a.max_blocks;
    constexpr int kAtOnce = 4;
    bool ids = true;
    for (unsigned j0 = keep; j0 < (unsigned)had; j0 += kAtOnce) {
        int id[kAtOnce];
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) id[k] = j0 + k < (unsigned)had ? table[j0 + k] : 0;
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) ids = ids && id[k] >= 0 && id[k] < a.num_blocks;
    }
    if (!ids) return Rest{L, 0, -1, kErrBadTable};
    return Rest{L - n + k, keep, had - keep, 0u};
}

// Blocks that request b may give back: at most n_b / block_size, rounded up.
__device__ __forceinline__ int may_give(const CompactArgs& a, int b) {
    const int lo = a.q_offsets[b], hi = a.q_offsets[b + 1];
    return is_run(lo, hi, a.num_tokens) ? blocks_of(hi - lo, a.block_size) : 0;
}

// Sums over a warp of what 48 bits hold, in two parts of 32.
__device__ __forceinline__ long long warp_sum(long long x) {
    return __reduce_add_sync(0xffffffffu, (unsigned)x & 0xffffu) + ((long long)__reduce_add_sync(0xffffffffu, (unsigned)(x >> 16)) << 16);
}

// Whether the stack has room for all that goes back, by the requests themselves; a whole CTA.  (Only of a stack that holds more than the
// blocks in use leave, see below.  Runs that overlap may give back more blocks than 31 bits count.)
__device__ __noinline__ bool has_room(const CompactArgs& a, int free0) {
    __shared__ long long sums[32];
    long long sum = 0;
    for (int b = threadIdx.x; b < a.num_seqs; b += blockDim.x) sum += max(0, rest_of(a, b).gives);
    sum = warp_sum(sum);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = sum;
    __syncthreads();
    sum = free0;
    for (int w = 0; w < blockDim.x / 32; ++w) sum += sums[w];
    return sum <= a.num_blocks;
}

// New lengths, and the blocks given back: one CTA, a request per thread, in rounds.  (8192 requests of 16 nodes, captured: the call 134 us, in place 170;
// with a contiguous run of requests per thread, passed twice, 163 and 255.)
__device__ __forceinline__ void trim(const CompactArgs& a) {
    __shared__ long long most[32];
    __shared__ int sums[2][32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x / 32, free0 = *a.num_free;
    long long back = 0;
    for (int b = tid; b < a.num_seqs; b += blockDim.x) back += may_give(a, b);
    back = warp_sum(back);
    if (lane == 0) most[warp] = back;
    __syncthreads();
    back = 0;
    for (int w = 0; w < warps; ++w) back += most[w];
    const bool room = free0 >= 0 && (free0 + back <= a.num_blocks || has_room(a, free0));
    unsigned bits = room ? 0 : kErrBadTable;
    int at = free0;
    for (int b0 = 0, round = 0; b0 < a.num_seqs; b0 += blockDim.x, round ^= 1) {
        const int b = b0 + tid;
        const Rest rest = b < a.num_seqs ? rest_of(a, b) : Rest{};
        bits |= rest.errors;
        const int gives = room ? max(0, rest.gives) : 0;
        int upto = gives;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        if (lane == 31) sums[round][warp] = upto;
        __syncthreads();
        int to = at + upto - gives;
        for (int w = 0; w < warps; ++w) {
            const int x = sums[round][w];
            if (w < warp) to += x;
            at += x;
        }
        for (int j = 0; j < gives; ++j) a.free_blocks[to + j] = a.block_tables[(long long)b * a.max_blocks + rest.keep + j];
        if (b < a.num_seqs) a.context_lens_out[b] = room ? rest.length : a.context_lens[b];
    }
    if (tid == 0) *a.num_free_out = at;
    if (bits) atomicOr(a.err, bits);
}

// Row (node a_j, layer, K or V, kv head) goes to the place of node j, for the nodes that are not there already: those behind the first that is
// not.  CTA (request, part of its rows); a thread has columns of sizeof(Vec) bytes and takes the nodes in order, kCompactBatch at a time:
// a node's place is written behind every read of it, since a_j >= j.  lead 1: CTA 0 has the lengths and the blocks; 0: a launch behind this
// one has them, since they replace what every CTA reads.
// Nothing of a request moves that keeps its length (moved twice, a branch would be lost), so each CTA decides for itself what trim() will.
// What all requests give back matters only for the room on the stack.  Request b holds at least as many blocks as it may give back,
// so that a stack of the blocks that nobody holds has room for the sum of these bounds; it costs less than the exact one, which is left to stacks
// without.
// The rows are 64 - 512 bytes here and there, each read and written once: HBM bounds many requests, latency few (28 layers of 4 heads of 128, bf16,
// captured calls: 256 requests with up to 16 accepted nodes 15.8 us, 64 with up to 5 5.5 us, in place 19.2 and 8.0; without the CTAs' own
// verdicts, moving first, 15.0 and 4.8; a CTA per request and a node at a time was 168 and 51 with the launch).
constexpr int kCompactBatch = 8;
template <typename Vec>
__global__ void __launch_bounds__(kCompactThreads) compact_tree_kernel(const CompactArgs a, const __grid_constant__ CachePtrs caches, int parts,
                                                                       int lead) {
    __shared__ long long from[kMaxTreeNodes], to[kMaxTreeNodes];  // bytes, of kv head 0
    __shared__ int moving[kCompactThreads / 32];
    __shared__ long long most[kCompactThreads / 32];
    griddep_wait();
    griddep_launch_dependents();
    if ((int)blockIdx.x < lead) {
        trim(a);
        return;
    }
    const int at = (int)blockIdx.x - lead, b = at / parts, part = at - b * parts, H = a.num_kv_heads, bs = a.block_size, tid = threadIdx.x;
    long long back = tid < a.num_seqs ? may_give(a, tid) : 0;  // (read beside what follows)
    int first;
    bool bad;
    const int n = nodes_of(a.q_offsets, b, a.num_tokens, INT_MAX, &first, &bad), count = a.num_accepted[b], L = a.context_lens[b], free0 = *a.num_free;
    if (bad || count <= 0 || count > n || count > a.max_accepted || L < n || L > (long long)a.max_blocks * bs || free0 < 0) return;
    const long long slots = (long long)a.num_blocks * bs;
    const int32_t* path = a.accepted + (long long)b * a.max_accepted;
    const int32_t* table = a.block_tables + (long long)b * a.max_blocks;
    bool wrong = false;
    if (tid >= kCompactThreads - 32) {  // a warp that hardly ever has nodes
        const unsigned keep = blocks_of(L - n + count, bs), had = blocks_of(L, bs);
        for (unsigned j = keep + tid % 32; j < had; j += 32) {
            const int id = table[j];
            wrong |= id < 0 || id >= a.num_blocks;
        }
    }
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
            const long long blk = slot < 0 ? 0 : (slot >> 32) == 0 ? (unsigned)slot / (unsigned)bs : slot / bs;
            at[k] = slot < 0 || slot >= slots ? -1 : (blk * H * bs + (slot - blk * bs)) * a.row_bytes;
        }
        if (at[0] < 0 || at[1] < 0) {
            if (node != j) atomicOr(a.err, kErrBadSlot);
            at[0] = -1;
        }
        from[j] = at[0];
        to[j] = at[1];
    }
    for (int i = tid + kCompactThreads; i < a.num_seqs; i += kCompactThreads) back += may_give(a, i);
    still = __reduce_add_sync(0xffffffffu, still);
    back = warp_sum(back);
    if ((tid & 31) == 0) moving[tid >> 5] = still, most[tid >> 5] = back;
    if (__syncthreads_or(wrong)) return;
    still = 0;
    back = 0;
#pragma unroll
    for (int w = 0; w < kCompactThreads / 32; ++w) still += moving[w], back += most[w];
    if (still == count || (free0 + back > a.num_blocks && !has_room(a, free0))) return;
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

constexpr int kTrimThreads = 1024;
__global__ void __launch_bounds__(kTrimThreads) trim_kernel(const CompactArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    trim(a);
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
    const bool in_place = a.context_lens_out == a.context_lens || a.num_free_out == a.num_free;
    const int lead = in_place && a.num_seqs > 0 ? 0 : 1;
    const dim3 grid((unsigned)(lead + (long long)a.num_seqs * parts)), block(kCompactThreads);
    cudaError_t e;
    if (a.vector) e = launch_pdl(compact_tree_kernel<uint4>, grid, block, 0, stream, a, caches, parts, lead);
    else if (a.elem_bytes == 4) e = launch_pdl(compact_tree_kernel<uint32_t>, grid, block, 0, stream, a, caches, parts, lead);
    else e = launch_pdl(compact_tree_kernel<uint16_t>, grid, block, 0, stream, a, caches, parts, lead);
    return e != cudaSuccess || lead ? e : launch_pdl(trim_kernel, dim3(1), dim3((unsigned)std::min(kTrimThreads, (a.num_seqs + 31) / 32 * 32)), 0, stream, a);
}

}  // namespace pa
