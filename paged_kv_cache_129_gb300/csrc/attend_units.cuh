// How the attention kernels share their work among the SMs.
//
// A unit is (request, pair of 128-row tiles, kv head).  All units' key tiles are laid end to end, weighted by their cost, and cut into one
// equal contiguous share per CTA; units cut by a share boundary leave float32 partial results (two slots per CTA), joined by a
// kernel of its own.  A Rule says what a unit costs (kPairedCost, kSplitCost a key tile, kUnitCost besides them, kMinShare), how many key
// tiles rows row0 .. row0 + 255 of a request take (tiles), and which further lengths are reported (refuses).  Args: the arguments of a call.
#pragma once

#include <cstdint>
#include <type_traits>

#include "tcgen05.cuh"

namespace pa {

// ---- work list (made by plan_kernel) ------------------------------------------------------------

struct Entry {
    long long first;  // cost before this entry
    int seq, row0;    // request, first row
    int tiles;        // key tiles, >= 1
    int paired;
};
static_assert(sizeof(Entry) == 24, "packed");

struct PlanHead {
    long long cost;
    int entries, pad;
};

struct Workspace {
    PlanHead* head;
    Entry* entries;   // [max_entries + 1], the last one a sentinel
    float* records;   // [CTAs][2 slots][2 tiles][m 128 | l 128 | o 128 x D]
};

__host__ __device__ inline size_t record_floats(int D) { return (size_t)kTile * (D + 2); }
inline size_t max_entries(int num_seqs, int num_tokens, int group) {
    return (size_t)num_seqs + ((size_t)num_tokens * group) / (2 * kTile);
}
inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// ---- the plan ------------------------------------------------------------------------------------------

template <class Args>
__device__ __forceinline__ int clamped_length(const Args& a, int b) {
    return max(0, min(a.context_lens[b], a.max_blocks * a.block_size));
}
template <class Args>
__device__ __forceinline__ int rows_of(const Args& a, int b) {  // request b's new tokens; none if its offsets are no run
    const int lo = a.q_offsets[b], hi = a.q_offsets[b + 1];
    return is_run(lo, hi, a.num_tokens) ? hi - lo : 0;
}

template <class Rule>
__device__ __forceinline__ long long unit_cost(int tiles, int paired) {
    return Rule::kUnitCost + (long long)tiles * (paired ? Rule::kPairedCost : Rule::kSplitCost);
}

constexpr int kPlanThreads = 1024;

// Exclusive sum of x over the CTA; *total the whole.  scratch: 33 entries.
__device__ __forceinline__ long long block_scan(long long x, long long* scratch, long long* total) {
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    long long s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    __syncthreads();
    if (lane == 31) scratch[wid] = s;
    __syncthreads();
    if (wid == 0) {
        long long w = scratch[lane], t = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += y;
        }
        scratch[lane] = t - w;
        if (lane == 31) scratch[32] = t;
    }
    __syncthreads();
    *total = scratch[32];
    return scratch[wid] + s - x;
}

template <class Args, class Rule>
__global__ void __launch_bounds__(kPlanThreads) attend_plan_kernel(const Args a, const Workspace ws, int entry_cap) {
    extern __shared__ int first_entry[];  // [num_seqs + 1]
    __shared__ long long scratch[33];
    griddep_wait();
    griddep_launch_dependents();
    const int group = a.num_heads / a.num_kv_heads, tid = threadIdx.x;
    long long base = 0, total = 0;
    for (int b0 = 0; b0 < a.num_seqs; b0 += kPlanThreads) {
        const int b = b0 + tid;
        long long n = 0;
        if (b < a.num_seqs) {
            const int L = a.context_lens[b], rows = rows_of(a, b);
            if (L < 0 || L > a.max_blocks * a.block_size || !is_run(a.q_offsets[b], a.q_offsets[b + 1], a.num_tokens) ||
                Rule::refuses(a, L, rows))
                atomicOr(a.err, kErrBadContext);
            n = ((long long)rows * group + 2 * kTile - 1) / (2 * kTile);
        }
        const long long at = base + block_scan(n, scratch, &total);
        if (b < a.num_seqs) first_entry[b] = (int)min(at, (long long)entry_cap);
        base += total;
    }
    int entries = (int)min(base, (long long)entry_cap);
    if (base > entry_cap) {  // runs that overlap
        if (tid == 0) atomicOr(a.err, kErrBadContext);
        entries = 0;
    }
    if (tid == 0) first_entry[a.num_seqs] = entries;
    __syncthreads();
    long long cost = 0;
    for (int e0 = 0; e0 < entries; e0 += kPlanThreads) {
        const int e = e0 + tid;
        Entry x{};
        long long c = 0;
        if (e < entries) {
            int lo = 0, hi = a.num_seqs;  // the last request whose first entry is <= e: one with rows
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (first_entry[mid] <= e)
                    lo = mid;
                else
                    hi = mid;
            }
            const int n = rows_of(a, lo);
            x.seq = lo;
            x.row0 = (e - first_entry[lo]) * 2 * kTile;
            x.paired = n * group - x.row0 > kTile;
            x.tiles = Rule::tiles(clamped_length(a, lo), n, group, x.row0);
            c = unit_cost<Rule>(x.tiles, x.paired) * a.num_kv_heads;
        }
        x.first = cost + block_scan(c, scratch, &total);
        cost += total;
        if (e < entries) ws.entries[e] = x;
    }
    if (tid == 0) {
        ws.entries[entries].first = cost;
        ws.head->cost = cost;
        ws.head->entries = entries;
    }
}

template <class Rule>
__device__ __forceinline__ long long share_of(long long cost, int ctas) {
    const long long s = (cost + ctas - 1) / ctas;
    return s > Rule::kMinShare ? s : Rule::kMinShare;
}

// The entry that cost position x falls into; whole CTA or warp, any number of threads.
__device__ __forceinline__ int find_entry(const Entry* e, int n, long long x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (e[mid].first <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Key tiles of a unit before cost position x inside it (a cut falls between tiles; both sides of a boundary round alike).
template <class Rule>
__device__ __forceinline__ int tiles_in(long long x, int tiles, bool paired) {
    const unsigned cost = (unsigned)max(0ll, min(x - Rule::kUnitCost, (long long)tiles * (paired ? Rule::kPairedCost : Rule::kSplitCost)));
    return (int)(paired ? (cost + Rule::kPairedCost - 1) / Rule::kPairedCost : (cost + Rule::kSplitCost - 1) / Rule::kSplitCost);
}

// The part of one unit that a share covers: key tiles [begin, end) of `tiles`.
struct Piece {
    int seq, row0, kvh, tiles, begin, end;
    bool paired;
};

// Walks over the pieces of share [pos, stop) of the plan.
template <class Rule>
struct UnitWalk {
    const Entry* entries;
    int count, heads, e, kvh;
    long long pos, stop;
    __device__ __forceinline__ UnitWalk(const Workspace& ws, int heads_, int cta, int ctas) : entries(ws.entries), heads(heads_) {
        const long long cost = ws.head->cost, share = share_of<Rule>(cost, ctas);
        count = ws.head->entries;
        pos = share * cta;
        stop = min(pos + share, cost);
        e = kvh = 0;
        if (pos < stop) {
            e = find_entry(entries, count, pos);
            const Entry x = entries[e];
            kvh = (int)((pos - x.first) / unit_cost<Rule>(x.tiles, x.paired));
        }
    }
    __device__ __forceinline__ bool next(Piece* p) {
        while (pos < stop) {
            const Entry x = entries[e];
            const long long cost = unit_cost<Rule>(x.tiles, x.paired), unit = x.first + kvh * cost;
            const long long from = pos > unit ? pos - unit : 0, to = stop - unit;
            p->seq = x.seq;
            p->row0 = x.row0;
            p->kvh = kvh;
            p->tiles = x.tiles;
            p->paired = x.paired != 0;
            p->begin = tiles_in<Rule>(from, x.tiles, p->paired);
            p->end = tiles_in<Rule>(to, x.tiles, p->paired);
            pos = unit + cost;
            if (++kvh == heads) {
                kvh = 0;
                ++e;
            }
            if (p->begin < p->end) return true;
        }
        return false;
    }
};

// What a piece is to every role.
struct Item {
    int L, n, group, rows;  // length, new tokens, heads per kv head, rows of the request
    int first_token;        // row of the request's first new token in query / out
    int jobs;               // score tiles: two streams take them in turn
};
template <class Args>
__device__ __forceinline__ Item item_of(const Args& a, const Piece& p) {
    Item it;
    it.L = clamped_length(a, p.seq);
    it.n = rows_of(a, p.seq);
    it.group = a.num_heads / a.num_kv_heads;
    it.rows = it.n * it.group;
    it.first_token = a.q_offsets[p.seq];
    it.jobs = (p.end - p.begin) * (p.paired ? 2 : 1);
    return it;
}

// Joins the partial results of the units that share boundaries cut.  CTA (boundary, rows): the first boundary inside a unit
// has it; a warp per row, D / 32 elements per lane.
constexpr int kJoinThreads = 256;
template <typename T, int D, class Args, class Rule>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const Args a, const Workspace ws, int ctas) {
    griddep_wait();
    griddep_launch_dependents();
    constexpr int E = D / 32;
    using Vec = typename std::conditional<E == 4, float4, float2>::type;
    const long long cost = ws.head->cost, share = share_of<Rule>(cost, ctas);
    const int c1 = blockIdx.x + 1;  // boundary: the start of CTA c1's share
    const long long x = share * c1;
    if (x >= cost) return;
    const Entry en = ws.entries[find_entry(ws.entries, ws.head->entries, x)];
    const long long each = unit_cost<Rule>(en.tiles, en.paired);
    const int kvh = (int)((x - en.first) / each);
    const long long unit = en.first + kvh * each, end = unit + each;
    if (x == unit || share * (c1 - 1) > unit) return;  // not inside, or not the first inside
    // pieces: CTA c has tiles [cut(c), cut(c + 1))
    auto cut = [&](int c) {
        const long long from = share * c - unit;
        return tiles_in<Rule>(from, en.tiles, en.paired != 0);
    };
    const int first = c1 - 1, last = (int)((end - 1) / share);
    bool parts = false;  // (a boundary inside the cost may still fall before the first tile or behind the last)
    for (int c = first + 1; c <= last; ++c) parts |= cut(c) > 0 && cut(c) < en.tiles;
    if (!parts) return;
    const int n = rows_of(a, en.seq), group = a.num_heads / a.num_kv_heads;
    const int rows = min(n * group - en.row0, 2 * kTile);
    const int lane = threadIdx.x & 31;
    for (int r = blockIdx.y * (kJoinThreads / 32) + (threadIdx.x >> 5); r < rows; r += gridDim.y * (kJoinThreads / 32)) {
        const int tile = r / kTile, rr = r % kTile;
        float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = 0.f;
        for (int c = first; c <= last; ++c) {
            const int from = cut(c);
            if (from >= cut(c + 1)) continue;
            const float* rec = ws.records + ((size_t)c * 4 + (from > 0 ? 0 : 2) + tile) * record_floats(D);
            const float mc = rec[rr], lc = rec[kTile + rr];
            const float mn = fmaxf(m, mc);
            float f = m == -INFINITY ? 0.f : exp2_approx(m - mn), fc = mc == -INFINITY ? 0.f : exp2_approx(mc - mn);
            if (l != l) f = 1.f;
            if (lc != lc) fc = 1.f;
            l = l * f + lc * fc;
            m = mn;
            alignas(16) float x[E];
            *reinterpret_cast<Vec*>(x) = *reinterpret_cast<const Vec*>(rec + 2 * kTile + (size_t)rr * D + lane * E);
#pragma unroll
            for (int i = 0; i < E; ++i) o[i] = o[i] * f + x[i] * fc;
        }
        const int v = en.row0 + r, token = v / group;
        T* dst = static_cast<T*>(a.out) +
                 ((size_t)(a.q_offsets[en.seq] + token) * a.num_heads + kvh * group + (v - token * group)) * D + lane * E;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        alignas(8) T y[E];
#pragma unroll
        for (int i = 0; i < E; ++i) y[i] = from_float<T>(o[i] * inv);
        if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(y);
        else *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(y);
    }
}

}  // namespace pa
