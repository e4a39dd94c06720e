// Block tables and slot maps of a serving step, built on the GPU from the requests' lengths.
//
// With L_b tokens held and n_b new ones, block size bs and a stack F of free block ids with top f:
//   give_b = ceil(L_b / bs) for a finished request (n_b < 0), whose ids are pushed in table order;
//   need_b = ceil((L_b + n_b) / bs) - ceil(L_b / bs), the k-th needed block (by request, then position)
//            being F[f1 - 1 - k] with f1 = f + sum give: what popping one id after the other gives;
//   token i of request b sits at position p = L_b + i - off_b, slot table[b, p / bs] * bs + p % bs.
// Everything is three prefix sums over the requests and then independent per block and per token.
//
// The work is a few bytes per token, so the launch and the dependent reads bound it, not bandwidth (64 decode requests 8.0 us,
// 256 requests with 61 700 new prompt tokens 17 us on the GPU).  One
// cluster does it: every CTA of the cluster computes the sums itself (no exchange through memory), a cluster
// barrier separates what is read from what is written, so that outputs may be the inputs' own buffers and a
// faulty step can be refused as a whole, and no state outlives the call.
#include <algorithm>
#include <cooperative_groups.h>

#include "pa_common.cuh"
#include "step_ops.h"

namespace pa {

namespace {

namespace cg = cooperative_groups;

constexpr int kTableThreads = 1024, kTableCtas = 8;
static_assert((long long)kMaxStepRows + kTableCtas * kTableThreads < (1ll << 31), "int counters pass the end by one step");

struct Sums {
    long long tok, need, give;
    int bad;
};

// Inclusive sums over a warp.
__device__ __forceinline__ Sums warp_scan(Sums s, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, s.tok, o);
        const long long n = __shfl_up_sync(0xffffffffu, s.need, o);
        const long long g = __shfl_up_sync(0xffffffffu, s.give, o);
        const int b = __shfl_up_sync(0xffffffffu, s.bad, o);
        if (lane >= o) {
            s.tok += t;
            s.need += n;
            s.give += g;
            s.bad |= b;
        }
    }
    return s;
}

// Largest b with off[b] <= x, for ascending off[0..n] with off[0] <= x < off[n].
__device__ __forceinline__ int find(const int* off, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Dynamic shared memory: lens [B], off_tok, off_need, off_give [B + 1] each.
__global__ void __launch_bounds__(kTableThreads) advance_tables_kernel(const AdvanceArgs a) {
    extern __shared__ int smem[];
    __shared__ Sums warp_sums[32];
    __shared__ unsigned refused;  // error bits found by this CTA; CTA 0's collects the cluster's
    griddep_wait();
    griddep_launch_dependents();
    cg::cluster_group cluster = cg::this_cluster();
    const int B = a.num_seqs, bs = a.block_size, tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    int* lens = smem;
    int* off_tok = lens + B;
    int* off_need = off_tok + B + 1;
    int* off_give = off_need + B + 1;
    const int cta = (int)cluster.block_rank(), ctas = (int)cluster.num_blocks();
    const int t0 = cta * kTableThreads + tid, stride = ctas * kTableThreads;
    if (tid == 0) refused = 0;
    cluster.barrier_arrive();  // waited for before the first access to another CTA's `refused`

    // prefix sums, a contiguous run of requests per thread
    const int per = (B + kTableThreads - 1) / kTableThreads;
    const int b0 = min(B, tid * per), b1 = min(B, b0 + per);
    Sums mine{0, 0, 0, 0};
    const int free0 = *a.num_free;
    for (int b = b0; b < b1; ++b) {
        const int L = a.context_lens[b], n = a.new_lens[b];
        const bool bad = L < 0 || (long long)L + max(n, 0) > (long long)a.max_blocks * bs;
        const int held = bad ? 0 : (int)(((long long)L + bs - 1) / bs);
        lens[b] = bad ? 0 : L;
        mine.bad |= bad;
        if (bad) continue;
        if (n < 0) {
            mine.give += held;
        } else {
            mine.tok += n;
            mine.need += ((long long)L + n + bs - 1) / bs - held;
        }
    }
    Sums incl = warp_scan(mine, lane);
    if (lane == 31) warp_sums[wid] = incl;
    __syncthreads();
    if (wid == 0) warp_sums[lane] = warp_scan(warp_sums[lane], lane);
    __syncthreads();
    const Sums total = warp_sums[31];
    unsigned bits = 0;
    if (total.bad || total.tok > a.num_tokens) bits |= kErrBadContext;
    if (free0 < 0 || free0 + total.give > a.num_blocks) bits |= kErrBadTable;
    if (!bits && total.need > free0 + total.give) bits |= kErrPoolExhausted;
    const int top = free0 + (int)total.give;  // both meaningful only while bits == 0
    unsigned found = 0;
    if (!bits) {
        Sums excl = incl;
        excl.tok -= mine.tok;
        excl.need -= mine.need;
        excl.give -= mine.give;
        if (wid > 0) {
            excl.tok += warp_sums[wid - 1].tok;
            excl.need += warp_sums[wid - 1].need;
            excl.give += warp_sums[wid - 1].give;
        }
        for (int b = b0; b < b1; ++b) {
            off_tok[b] = (int)excl.tok;
            off_need[b] = (int)excl.need;
            off_give[b] = (int)excl.give;
            const long long L = lens[b], n = a.new_lens[b], held = (L + bs - 1) / bs;
            if (n < 0) {
                excl.give += held;
            } else {
                excl.tok += n;
                excl.need += (L + n + bs - 1) / bs - held;
            }
        }
        if (tid == 0) {
            off_tok[B] = (int)total.tok;
            off_need[B] = (int)total.need;
            off_give[B] = (int)total.give;
        }
        __syncthreads();
        // Ids given back go onto the stack (above the old top, where nothing valid lies), and every id that the
        // step will use is looked at before anything that a caller relies on is written.
        for (int i = t0; i < (int)total.give; i += stride) {
            const int b = find(off_give, B, i);
            const int id = a.block_tables[(size_t)b * a.max_blocks + (i - off_give[b])];
            if (id < 0 || id >= a.num_blocks) found = kErrBadTable;
            a.free_blocks[free0 + i] = id;
        }
        for (int k = t0; k < (int)total.need; k += stride) {
            const int at = top - 1 - k;
            if (at < free0) {
                const int id = a.free_blocks[at];
                if (id < 0 || id >= a.num_blocks) found = kErrBadTable;
            }
        }
        for (int b = t0; b < B; b += stride) {
            if (off_tok[b + 1] > off_tok[b] && lens[b] % bs != 0) {
                const int id = a.block_tables[(size_t)b * a.max_blocks + lens[b] / bs];
                if (id < 0 || id >= a.num_blocks) found = kErrBadTable;
            }
        }
    }
    cluster.barrier_wait();
    if (found) atomicOr(cluster.map_shared_rank(&refused, 0), found);
    cluster.sync();  // reads of the inputs and the pushes are done
    if (!bits) bits = *cluster.map_shared_rank(&refused, 0);

    if (bits) {
        if (t0 == 0) {
            atomicOr(a.err, bits);
            *a.num_free_out = free0;
        }
        for (int b = t0; b < B; b += stride)
            if (a.context_lens_out != a.context_lens) a.context_lens_out[b] = a.context_lens[b];
        for (int b = t0; b <= B; b += stride) a.q_offsets[b] = 0;
        for (int t = t0; t < a.num_tokens; t += stride) {
            a.positions[t] = 0;
            a.slot_mapping[t] = -1;
        }
    } else {
        const int need = (int)total.need, tok = (int)total.tok;
        if (t0 == 0) *a.num_free_out = top - need;
        for (int b = t0; b <= B; b += stride) {
            a.q_offsets[b] = off_tok[b];
            if (b == B) break;
            // a finished request with nothing held gives nothing, and has length 0 already
            a.context_lens_out[b] = off_give[b + 1] > off_give[b] ? 0 : lens[b] + off_tok[b + 1] - off_tok[b];
        }
        for (int k = t0; k < need; k += stride) {
            const int b = find(off_need, B, k);
            const int j = (int)(((long long)lens[b] + bs - 1) / bs) + (k - off_need[b]);
            a.block_tables[(size_t)b * a.max_blocks + j] = __ldcg(a.free_blocks + top - 1 - k);
        }
        for (int t = t0; t < a.num_tokens; t += stride) {
            if (t >= tok) {
                a.positions[t] = 0;
                a.slot_mapping[t] = -1;
                continue;
            }
            const int b = find(off_tok, B, t);
            const int p = lens[b] + (t - off_tok[b]), j = p / bs, held = (int)(((long long)lens[b] + bs - 1) / bs);
            const int id = j < held ? a.block_tables[(size_t)b * a.max_blocks + j]
                                    : __ldcg(a.free_blocks + top - 1 - (off_need[b] + j - held));
            a.positions[t] = p;
            a.slot_mapping[t] = (int64_t)id * bs + (p - j * bs);
        }
    }
    if (ctas > 1) cluster.sync();  // CTA 0's shared memory outlives the others' reads of it
}

}  // namespace

cudaError_t advance_tables_launch(const AdvanceArgs& a, cudaStream_t stream) {
    const size_t smem = ((size_t)4 * a.num_seqs + 3) * sizeof(int);
    static_assert((4 * kMaxStepSeqs + 3) * sizeof(int) <= 200 * 1024, "the sums fit shared memory");
    cudaError_t e = cudaFuncSetAttribute(advance_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)((4 * kMaxStepSeqs + 3) * sizeof(int)));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    const unsigned ctas = kTableCtas;
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kTableThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, advance_tables_kernel, a);
}

}  // namespace pa
