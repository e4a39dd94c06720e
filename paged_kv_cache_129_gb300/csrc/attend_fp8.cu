// Causal attention of ragged runs of new tokens over an FP8 (E4M3) paged cache, on tcgen05 tensor cores.
//
// Request b has the rows q_offsets[b] .. q_offsets[b + 1] - 1, the last n_b positions of its L_b; the row at
// position p attends positions 0 .. p:  out = sum softmax(scale q k_j) v_j, with k_j, v_j = code * scale(block, head).
//
// Rows.  The g query heads of a kv head and the request's tokens form R = n_b * g rows (row v: token v / g, head
// v % g), cut into tiles of 128, the M of the products; keys come in tiles of 128 tokens, whose scores are made and
// used in halves of 64 columns: while the softmax warps work on one half, the other half's products run.
// A CTA has two streams of softmax warps:
//   paired  two row tiles share every key tile (it is widened once for both);
//   split   a single row tile (few rows: verification, decode, the rest of a run): the streams take alternate key
//           tiles, and join their results at the end.
// Work.  A unit is (request, pair of row tiles, kv head).  All units' key tiles are laid end to end, weighted by their
// cost, and cut into one equal contiguous share per SM, so every SM works equally long whatever the length mix; units cut by a
// share boundary leave float32 partial results (two slots per CTA), joined by a third kernel.
// Numbers.  E4M3 codes widen to f16 exactly; a query row is moved into f16 range by a power of two (f16 queries as they
// are), undone in the score factor.  A block's K scale multiplies its scores; its V scale multiplies P, so that V goes into the
// products as codes.  Scores, maxima, sums and the output accumulate in float32; P alone is rounded to f16, relative to a power of
// two (vref) near the row's largest exponential times V scale: half a step 2^-11 of a weight (below the half step 2^-9 of a bf16
// output), and 2^-25 of the largest one for weights below 2^-14 of it.  Only what a row sees counts for that: neither a block behind its
// position nor one of a negligible weight takes bits from it.  Both references, the maximum that exponents are taken from and vref, follow
// the true ones by steps of 2^8 at least: rescaling the output in tensor memory is rare that way.
// Bound.  Shared memory: a split key tile at D = 128 moves 256 KB through it (codes in and out, widened, query rows for two halves,
// K, V), 2048 of the 3000 cycles that it takes; a paired one 384 KB.  Prompt chunks (four requests of 1500 - 2048 new tokens on
// 2048 - 6144) take 616 us, 0.90 PFLOP/s, issue slots 51 % and the tensor pipe 39 % busy; few rows on long contexts (eight
// requests of 32k - 128k tokens) 394 us, 3.15 TB/s.  That bound is the 128-row tile's: few rows pay for all of it.  64 requests of four
// tokens take 117 us, pa_decode_multi over a 16-bit cache, twice the bytes, 68; of one token 108 us, pa_decode_fp8 46.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include <cuda_fp8.h>

#include "pa_common.cuh"
#include "step_ops.h"
#include "tcgen05.cuh"

namespace pa {

namespace {

constexpr int kSoftmaxWarps = 8;       // four per stream
constexpr int kWidenWarps = 4;
constexpr int kIssueWarp = kSoftmaxWarps + kWidenWarps;  // two, one per stream
constexpr int kCopyWarp = kIssueWarp + 2, kLookWarp = kCopyWarp + 1;
constexpr int kThreads = (kLookWarp + 1) * 32;
constexpr int kBuffers = 3;            // f16 operand tiles (K or V) in shared memory
constexpr int kRing = 16;              // slots of per-tile side data (block ids, scales), see look_ahead()
constexpr int kAhead = kRing - 6;      // key tiles that look_ahead() may be ahead of the copies
constexpr int kNanRing = 2;            // V of tile i is widened once the scores of tile i (i - 1) are done: the softmax of i - 2 too
// Cost of work in shares: of a key tile of a pair, of a split tile (half the products and exponentials, but the same loads and
// widening), and of a unit besides its tiles (queries staged, streams joined, output written: about six split tiles).  Measured when chosen
// (verification / prompt chunks / long contexts / short mixed D = 64, us): 6, 4, 24: 115 / 625 / 387 / 95; 4, 3, 8: 135 / 656 / 412 /
// 98.  With prefetches as in look_ahead()'s note, 4, 3, 0 (no cost of a unit) took 175 / 694 / 430 / 125, 4, 3, 8 143 / 675 / 439 / 99.
constexpr int kPairedCost = 6, kSplitCost = 4, kUnitCost = 24;
constexpr int kMinShare = kUnitCost + 4 * kSplitCost;  // a CTA's share is not worth less than the pieces' overhead

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

// ---- PTX ------------------------------------------------------------------------------------------

// Four rows y of a tensor map whose box is one row, into shared memory one after the other; x in elements.  One elected lane.
__device__ __forceinline__ void gather4(void* dst, const CUtensorMap* map, int x, int4 y, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];\n\t}" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w), "r"(smem_addr(bar))
        : "memory");
}
// ---- the plan ------------------------------------------------------------------------------------------

__device__ __forceinline__ int clamped_length(const AttendArgs& a, int b) {
    return max(0, min(a.context_lens[b], a.max_blocks * a.block_size));
}
__device__ __forceinline__ int rows_of(const AttendArgs& a, int b) {  // request b's new tokens; none if its offsets are no run
    const int lo = a.q_offsets[b], hi = a.q_offsets[b + 1];
    return is_run(lo, hi, a.num_tokens) ? hi - lo : 0;
}

// Key tiles of rows row0 .. row0 + 255 of a request: up to the last row's position.
__device__ __forceinline__ int tiles_of(int L, int n, int group, int row0) {
    const int last = min(n * group, row0 + 2 * kTile) - 1;
    const int bound = L - n + last / group;
    return max(1, (bound + kTile) / kTile);
}

__device__ __forceinline__ long long unit_cost(int tiles, int paired) {
    return kUnitCost + (long long)tiles * (paired ? kPairedCost : kSplitCost);
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

__global__ void __launch_bounds__(kPlanThreads) attend_plan_kernel(const AttendArgs a, const Workspace ws, int entry_cap) {
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
            const int L = a.context_lens[b];
            if (L < 0 || L > a.max_blocks * a.block_size || !is_run(a.q_offsets[b], a.q_offsets[b + 1], a.num_tokens))
                atomicOr(a.err, kErrBadContext);
            n = ((long long)rows_of(a, b) * group + 2 * kTile - 1) / (2 * kTile);
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
            x.tiles = tiles_of(clamped_length(a, lo), n, group, x.row0);
            c = unit_cost(x.tiles, x.paired) * a.num_kv_heads;
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

__device__ __forceinline__ long long share_of(long long cost, int ctas) {
    const long long s = (cost + ctas - 1) / ctas;
    return s > kMinShare ? s : kMinShare;
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
__device__ __forceinline__ int tiles_in(long long x, int tiles, bool paired) {
    const unsigned cost = (unsigned)max(0ll, min(x - kUnitCost, (long long)tiles * (paired ? kPairedCost : kSplitCost)));
    return (int)(paired ? (cost + kPairedCost - 1) / kPairedCost : (cost + kSplitCost - 1) / kSplitCost);
}

// The part of one unit that a share covers: key tiles [begin, end) of `tiles`.
struct Piece {
    int seq, row0, kvh, tiles, begin, end;
    bool paired;
};

// Walks over the pieces of share [pos, stop) of the plan.
struct Walk {
    const Entry* entries;
    int count, heads, e, kvh;
    long long pos, stop;
    __device__ __forceinline__ Walk(const Workspace& ws, int heads_, int cta, int ctas) : entries(ws.entries), heads(heads_) {
        const long long cost = ws.head->cost, share = share_of(cost, ctas);
        count = ws.head->entries;
        pos = share * cta;
        stop = min(pos + share, cost);
        e = kvh = 0;
        if (pos < stop) {
            e = find_entry(entries, count, pos);
            const Entry x = entries[e];
            kvh = (int)((pos - x.first) / unit_cost(x.tiles, x.paired));
        }
    }
    __device__ __forceinline__ bool next(Piece* p) {
        while (pos < stop) {
            const Entry x = entries[e];
            const long long cost = unit_cost(x.tiles, x.paired), unit = x.first + kvh * cost;
            const long long from = pos > unit ? pos - unit : 0, to = stop - unit;
            p->seq = x.seq;
            p->row0 = x.row0;
            p->kvh = kvh;
            p->tiles = x.tiles;
            p->paired = x.paired != 0;
            p->begin = tiles_in(from, x.tiles, p->paired);
            p->end = tiles_in(to, x.tiles, p->paired);
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

// ---- shared memory of the attention kernel -----------------------------------------------------------------

template <int D>
struct Smem {
    static constexpr int kOperand = kTile * D * 2;      // one f16 tile
    static constexpr int kRaw = D == 128 ? 3 : 6;       // tiles of codes on their way or waiting: 48 KB in flight per SM
    unsigned char q[2][kOperand];
    unsigned char kv[kBuffers][kOperand];
    unsigned char raw[kRaw][kTile * D];
    float ks[kRing][8], vs[kRing][8], lv[kRing][8];     // scales of the tile's blocks; the exponent of the V scale
    int rows[kRing][8];                                 // and their rows of the K map (of the V map: the next)
    unsigned present[kRing], masked[kRing];             // blocks of the tile: there; with an id outside the pool
    unsigned nan_any[kNanRing][kWidenWarps];            // whether a warp found NaN in V of a tile that some row sees in part,
    uint16_t nan_at[kNanRing][kTile][D / 16];           // and where: per token and 16 elements
    uint32_t nan_row[2][kTile][D / 32];                 // per row: elements of the output that are NaN, if its thread says so
    float4 state[2][kTile];                             // at the end of a split piece: both streams' m, l, vref, has_nan
    uint64_t side_full[kRing], copied[kRing], q_full[2], raw_full[kRaw], raw_empty[kRaw], kv_full[kBuffers], kv_empty[kBuffers];
    uint64_t s_full[2][2], p_full[2][2], pv_done[2][2], o_full[2], join_full, join_done, drain[2];
    uint32_t tmem;
    volatile int abort;
};

// The order in which a piece's n key tiles go through the buffers.  Paired: K0 V0 K1 V1 ...  Split: K one tile ahead, K0 K1 V0 K2
// V1 ... V(n-2) V(n-1), because the scores of a tile are issued before the output of the tile before it.
struct Fill {
    int tile;
    bool value;
};
__device__ __forceinline__ Fill fill_of(bool paired, int n, int i) {
    if (paired) return {i >> 1, (i & 1) != 0};
    if (i == 2 * n - 1) return {n - 1, true};
    if (i == 0) return {0, false};
    return (i & 1) ? Fill{(i + 1) >> 1, false} : Fill{(i >> 1) - 1, true};
}
__device__ __forceinline__ int key_fill(bool paired, int tile) { return paired ? 2 * tile : tile == 0 ? 0 : 2 * tile - 1; }
__device__ __forceinline__ int value_fill(bool paired, int n, int tile) {
    return paired ? 2 * tile + 1 : tile == n - 1 ? 2 * n - 1 : 2 * tile + 2;
}

static_assert(sizeof(Smem<128>) + 1024 <= 227 * 1024, "fits an SM");

// What a piece is to every role.
struct Item {
    int L, n, group, rows;  // length, new tokens, heads per kv head, rows of the request
    int first_token;        // row of the request's first new token in query / out
    int jobs;               // score tiles: two streams take them in turn
};
__device__ __forceinline__ Item item_of(const AttendArgs& a, const Piece& p) {
    Item it;
    it.L = clamped_length(a, p.seq);
    it.n = rows_of(a, p.seq);
    it.group = a.num_heads / a.num_kv_heads;
    it.rows = it.n * it.group;
    it.first_token = a.q_offsets[p.seq];
    it.jobs = (p.end - p.begin) * (p.paired ? 2 : 1);
    return it;
}

// Sixteen E4M3 codes as f16 (exact), in two 16-byte units.
__device__ __forceinline__ void widen_store(unsigned char* unit0, unsigned char* unit1, uint4 c) {
    uint32_t h[8];
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, lo;\n\tcvt.rn.f16x2.e4m3x2 %1, hi;\n\t}"
            : "=r"(h[2 * i]), "=r"(h[2 * i + 1])
            : "r"(w[i]));
    *reinterpret_cast<uint4*>(unit0) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4*>(unit1) = make_uint4(h[4], h[5], h[6], h[7]);
}

// Per byte of w: 0x80 where the code is NaN.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// The look-ahead warp: block ids and scales of tile after tile into the side ring, up to kAhead tiles before they are copied and
// across the ends of pieces, so that the tables' and scales' latencies are not waited for.  (It also prefetched the codes into L2 at
// first, line by line: 144 / 676 / 439 us on verification, chunks, long contexts with, 134 / 656 / 412 without; the raw ring's
// 48 KB in flight per SM cover HBM's latency.)
// Side data of tile i sits in slot i % kRing, which was tile i - kRing's.  When K of tile j is copied, at least 2j - 1 fills went before
// (see fill_of()).  The raw slot that it takes was widened: fill 2j - 1 - kRaw; so the f16 buffer that this one went to was released by
// the products of fill 2j - 1 - kRaw - kBuffers and all before it.  V of tile g is fill 2g + 2 at most: with 2g <= 2j - 3 - kRaw - kBuffers,
// the outputs of tile g are issued, so its softmax, the last to look at its side data, is done.  Tile i is looked at once K of tile
// i - kAhead is copied, so g = i - kRing has to satisfy that for j = i - kAhead.
template <int D, int BS>
__device__ __forceinline__ void look_ahead(const AttendArgs& a, const Workspace& ws, Smem<D>& sm) {
    constexpr int BLOCKS = kTile / BS;
    static_assert(2 * (kRing - kAhead) >= Smem<D>::kRaw + kBuffers + 3, "a slot's tile is done with when it is written again");
    const int lane = threadIdx.x & 31;
    const bool both = a.value_cache == nullptr;
    Walk walk(ws, a.num_kv_heads, blockIdx.x, gridDim.x);
    Piece p;
    unsigned tiles = 0;
    while (walk.next(&p)) {
        const int used = (clamped_length(a, p.seq) + BS - 1) / BS;
        const int32_t* table = a.block_tables + (size_t)p.seq * a.max_blocks;
        // lane j < BLOCKS has block j of a tile
        auto wanted = [&](int tile) { return lane < BLOCKS && tile < p.end && tile * BLOCKS + lane < used; };
        int id = wanted(p.begin) ? table[p.begin * BLOCKS + lane] : -1;
        for (int tile = p.begin; tile < p.end; ++tile, ++tiles) {
            const bool mine = wanted(tile), in = mine && id >= 0 && id < a.num_blocks;
            if (mine && !in) atomicOr(a.err, kErrBadTable);
            // (blocks that are not there take record 0's place: whatever it brings is not used)
            const int record = (in ? id : 0) * a.num_kv_heads + p.kvh;
            const float ks = in ? a.k_scale[record] : 0.f, vs = in ? a.v_scale[record] : 0.f;
            id = wanted(tile + 1) ? table[(tile + 1) * BLOCKS + lane] : -1;
            const unsigned present = __ballot_sync(0xffffffffu, in), masked = __ballot_sync(0xffffffffu, mine && !in);
            if (tiles >= kAhead) {
                const unsigned before = tiles - kAhead;
                if (!warp_wait(&sm.copied[before % kRing], (before / kRing) & 1, a.err, &sm.abort)) return;
            }
            const int slot = tiles % kRing;
            if (lane < 8) {
                sm.ks[slot][lane] = ks;
                sm.vs[slot][lane] = vs;
                sm.lv[slot][lane] = (float)((int)(__float_as_uint(vs) >> 23) - 127);  // (of zero and subnormal ones -127)
                sm.rows[slot][lane] = both ? 2 * record : record;
            }
            if (lane == 0) {
                sm.present[slot] = present;
                sm.masked[slot] = masked;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.side_full[slot]);
        }
    }
}

// The copy warp: K or V of four blocks by one gather (a block's rows of a head are one row of the tensor map), into the raw ring.
// Registers and L1 could not hold what has to be in flight: with 200 KB of shared memory taken, L1 has room for about
// 14 KB, and plain loads stalled at 2.2 TB/s over all SMs.  One copy per block, from a lane each, took 1900 cycles a tile to issue.
template <int D, int BS>
__device__ __forceinline__ void copy_tiles(const AttendArgs& a, const Workspace& ws, Smem<D>& sm, const CUtensorMap* kmap,
                                           const CUtensorMap* vmap) {
    constexpr int BLOCKS = kTile / BS, RAW = Smem<D>::kRaw;
    constexpr int kRowBytes = BS * D, kBox = kRowBytes < 2048 ? kRowBytes : 2048, PARTS = kRowBytes / kBox;  // 8-byte elements
    const int lane = threadIdx.x & 31;
    const int next_row = a.value_cache == nullptr ? 1 : 0;
    Walk walk(ws, a.num_kv_heads, blockIdx.x, gridDim.x);
    Piece p;
    unsigned fills = 0, tiles = 0;
    bool ok = true;
    while (ok && walk.next(&p)) {
        const int n = p.end - p.begin;
#pragma unroll 1
        for (int i = 0; i < 2 * n; ++i, ++fills) {
            const Fill f = fill_of(p.paired, n, i);
            const int slot = fills % RAW;
            const unsigned tile = tiles + f.tile, side = tile % kRing;
            ok = f.value || warp_wait(&sm.side_full[side], (tile / kRing) & 1, a.err, &sm.abort);
            ok = ok && warp_wait(&sm.raw_empty[slot], ((fills / RAW) & 1) ^ 1, a.err, &sm.abort);
            if (!ok) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(&sm.raw_full[slot], kTile * D);
                if (!f.value) mbar_arrive(&sm.copied[side]);
            }
            __syncwarp();
            const CUtensorMap* map = f.value ? vmap : kmap;
#pragma unroll
            for (int g = 0; g < BLOCKS / 4; ++g) {
                int4 y = *reinterpret_cast<const int4*>(&sm.rows[side][4 * g]);
                if (f.value) y = make_int4(y.x + next_row, y.y + next_row, y.z + next_row, y.w + next_row);
#pragma unroll
                for (int part = 0; part < PARTS; ++part)
                    gather4(sm.raw[slot] + (part * BLOCKS + 4 * g) * kBox, map, part * (kBox / 8), y, &sm.raw_full[slot]);
            }
        }
        tiles += n;
    }
    if (!ok) {  // copies still under way must land before the CTA's shared memory goes
        int never = 0;
        for (unsigned f = fills > RAW ? fills - RAW : 0; f < fills; ++f)
            mbar_wait_bounded(&sm.raw_full[f % RAW], (f / RAW) & 1, a.err, &never);
    }
}

// The four widen warps: tile after tile of codes from the raw ring to a swizzled f16 buffer.
template <int D, int BS>
__device__ __forceinline__ void widen_tiles(const AttendArgs& a, const Workspace& ws, Smem<D>& sm) {
    constexpr int RPP = 128 / (D / 16), N = kTile / RPP, RAW = Smem<D>::kRaw;  // rows per pass, passes
    const int tid = threadIdx.x - kSoftmaxWarps * 32, lane = tid & 31;
    // A thread's sixteen codes of a row, the same in every pass.  The eight lanes that load or store together hold half a row each
    // of an even and an odd row, the halves apart: eight different 16-byte columns of the codes (128-byte lines), and
    // eight different swizzled units of the buffer.
    const int chunk = D == 128 ? (lane & 3) + 4 * ((lane >> 2 ^ lane >> 3) & 1) : lane & 3;
    const int row0 = D == 128 ? 4 * (tid >> 5) + (lane >> 2 & 1) + 2 * (lane >> 4) : tid >> 2;
    const uint32_t line = (chunk / 4) * kPanel + row0 * 128, u = (chunk % 4) * 2;
    const uint32_t unit0 = line + ((u ^ (row0 & 7)) << 4), unit1 = line + (((u + 1) ^ (row0 & 7)) << 4);
    Walk walk(ws, a.num_kv_heads, blockIdx.x, gridDim.x);
    Piece p;
    unsigned fills = 0, tiles = 0;
    while (walk.next(&p)) {
        const Item it = item_of(a, p);
        const int n = p.end - p.begin;
        const int seen_by_all = it.L - it.n + p.row0 / it.group;  // the first row's position
        for (int i = 0; i < 2 * n; ++i, ++fills) {
            const Fill f = fill_of(p.paired, n, i);
            const int slot = fills % RAW, buf = fills % kBuffers, p0 = (p.begin + f.tile) * kTile;
            if (!warp_wait(&sm.raw_full[slot], (fills / RAW) & 1, a.err, &sm.abort)) return;
            const unsigned present = sm.present[(tiles + f.tile) % kRing];
            const int left = it.L - p0;  // rows of the tile inside the context; the others' codes may be anything
            if (!warp_wait(&sm.kv_empty[buf], ((fills / kBuffers) & 1) ^ 1, a.err, &sm.abort)) return;
            // rows row0 + 16 k (32 k); a block of 4 KB came as two halves, all first halves before all second ones
            const unsigned char* from = sm.raw[slot] + row0 * D + chunk * 16;
            auto pass = [&](int k) { return BS * D > 2048 ? ((k & 1) * 4 + (k >> 1)) * 2048 : k * RPP * D; };
            unsigned char *to0 = sm.kv[buf] + unit0, *to1 = sm.kv[buf] + unit1;
            const bool seen_in_part = p0 + kTile - 1 > seen_by_all;
            if (left >= kTile && present == (1u << (kTile / BS)) - 1 && !(f.value && seen_in_part)) {
#pragma unroll 1
                for (int k = 0; k < N; k += 4) {
                    uint4 c[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) c[j] = *reinterpret_cast<const uint4*>(from + pass(k + j));
#pragma unroll
                    for (int j = 0; j < 4; ++j) widen_store(to0 + (k + j) * RPP * 128, to1 + (k + j) * RPP * 128, c[j]);
                }
                if (f.value && lane == 0) sm.nan_any[(tiles + f.tile) % kNanRing][tid >> 5] = 0;
            } else {
                // Rows past the context are zeros.  Where some row sees the tile in part, a NaN of V behind its position must not
                // reach it through 0 * NaN: NaN become zeros too, and the softmax warps are told where they were.
                const int at_slot = (tiles + f.tile) % kNanRing;
                bool any = false;
#pragma unroll 1
                for (int k = 0; k < N; ++k) {
                    const int r = row0 + k * RPP;
                    uint4 c = *reinterpret_cast<const uint4*>(from + pass(k));
                    if (r >= left || !(present >> (r / BS) & 1)) c = make_uint4(0u, 0u, 0u, 0u);
                    if (f.value && seen_in_part) {
                        unsigned at = 0;
                        auto clean = [&](uint32_t w, int j) {
                            const uint32_t t = nan_bytes(w) >> 7;
                            at |= ((t * 0x01020408u >> 24) & 0xfu) << (4 * j);
                            return w & ~(t * 0xffu);
                        };
                        c = make_uint4(clean(c.x, 0), clean(c.y, 1), clean(c.z, 2), clean(c.w, 3));
                        any |= at != 0;
                        sm.nan_at[at_slot][r][chunk] = (uint16_t)at;
                    }
                    widen_store(to0 + k * RPP * 128, to1 + k * RPP * 128, c);
                }
                any = __any_sync(0xffffffffu, any);
                if (f.value && lane == 0) sm.nan_any[at_slot][tid >> 5] = any;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.raw_empty[slot]);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.kv_full[buf]);
        }
        tiles += n;
    }
}

// One warp per stream issues its products; while one waits, the other's keep the tensor cores busy.  Job j of a piece is a
// score tile of stream j % 2, in two halves of 64 columns (64 tokens): a half's scores are issued right behind the output of the
// same half of the stream's previous job, which has then read the P that they overwrite, and are ready while the softmax warps are
// still at the other half.  (Scores of 64 columns cost 768 cycles a tile instead of 512: the query rows are read twice.)
template <int D>
__device__ __forceinline__ void issue_products(const AttendArgs& a, const Workspace& ws, Smem<D>& sm, int t) {
    volatile int* abort = &sm.abort;
    const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0), s_at = tmem + t * kTile, o_at = tmem + 2 * kTile + t * D;
    const uint64_t qd = desc_of(smem_addr(sm.q[t]), 16, 1024), k0 = desc_of(smem_addr(sm.kv[0]), 16, 1024),
                   v0 = desc_of(smem_addr(sm.kv[0]), kPanel, 1024);
    Walk walk(ws, a.num_kv_heads, blockIdx.x, gridDim.x);
    Piece p;
    unsigned fills = 0, pieces = 0, steps = 0;
    while (walk.next(&p)) {
        const int n = p.end - p.begin, jobs = n * (p.paired ? 2 : 1);
        // A buffer is free after two arrivals: one from either stream, or two from the only one that reads it.  A wait tells a
        // phase from the one before it alone, so no thread may skip a buffer's turn without knowing that it came: within a
        // piece the fills that a stream waits for are at most three apart, and a piece of one tile, stream 0's, is waited for
        // and released by stream 1 too.
        const bool alone = !p.paired && jobs > 1;
        auto release = [&](unsigned buf) {
            tc_commit(&sm.kv_empty[buf]);
            if (alone) tc_commit(&sm.kv_empty[buf]);
        };
        if (jobs <= t) {
            for (unsigned f = fills; f < fills + 2; ++f) {
                if (!warp_wait(&sm.kv_full[f % kBuffers], (f / kBuffers) & 1, a.err, abort)) return;
                if ((threadIdx.x & 31) == 0) mbar_arrive(&sm.kv_empty[f % kBuffers]);
            }
        }
        // unit u: half u % 2 of the stream's job u / 2
        const int units = 2 * ((jobs + 1 - t) / 2);
#pragma unroll 1
        for (int u = -2; u < units; ++u) {
            const int half = u & 1;
            if (u >= 0) {
                const int tile = p.paired ? u >> 1 : u - half + t;
                const unsigned f = fills + value_fill(p.paired, n, tile), buf = f % kBuffers;
                if (half == 0 && !warp_wait(&sm.kv_full[buf], (f / kBuffers) & 1, a.err, abort)) return;
                if (!warp_wait(&sm.p_full[t][half], steps & 1, a.err, abort)) return;
                tc_fence_after();
                const uint64_t vd = v0 + buf * (Smem<D>::kOperand >> 4) + half * (kTile * 64 >> 4);
#pragma unroll
                for (int k = 0; k < kTile / 32; ++k)
                    mma_ts(o_at, s_at + 64 * half + 8 * k, vd + (k * 2048 >> 4), idesc_of(D, true), u > 0 || k > 0);
                tc_commit(&sm.pv_done[t][half]);
                if (half == 1) {
                    release(buf);
                    ++steps;
                }
                if (u == units - 1) tc_commit(&sm.o_full[t]);
            }
            const int next = u + 2;
            if (next < units) {
                const int tile = p.paired ? next >> 1 : next - half + t;
                const unsigned f = fills + key_fill(p.paired, tile), buf = f % kBuffers;
                if (half == 0 && !warp_wait(&sm.kv_full[buf], (f / kBuffers) & 1, a.err, abort)) return;
                if (next == 0 && !warp_wait(&sm.q_full[t], pieces++ & 1, a.err, abort)) return;
                tc_fence_after();
                const uint64_t kd = k0 + buf * (Smem<D>::kOperand >> 4) + half * (kTile * 64 >> 4);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = ((k / 4) * kPanel + (k % 4) * 32) >> 4;
                    mma_ss(s_at + 64 * half, qd + off, kd + off, idesc_of(kTile / 2, false), k > 0);
                }
                if (half == 1) release(buf);
                tc_commit(&sm.s_full[t][half]);
            }
        }
        fills += 2 * n;
    }
}

// A warp's 32 query rows to f16, into the swizzled tile; row_at: where this lane's row begins (live: if it exists).  D / 8 lanes load a
// row together.  Returns what undoes the power of two that this lane's row was moved by.
template <typename T, int D>
__device__ __forceinline__ float stage_query(const T* query, size_t row_at, bool live, bool negate, unsigned char* tile, int row0) {
    constexpr int LPR = D / 8, RPS = 32 / LPR, BATCH = 8;
    const int lane = threadIdx.x & 31, sub = lane / LPR, i = lane % LPR;
    const unsigned alive = __ballot_sync(0xffffffffu, live);
    float undo = 1.f;
#pragma unroll 1
    for (int b = 0; b < 32; b += BATCH * RPS) {
        uint4 raw[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k)  // (rows that do not exist read the first one: a branch would wait for each load)
            raw[k] = *reinterpret_cast<const uint4*>(query + __shfl_sync(0xffffffffu, row_at, b + k * RPS + sub) + 8 * i);
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int r = b + k * RPS + sub, row = row0 + r;
            if (!(alive >> r & 1)) raw[k] = make_uint4(0u, 0u, 0u, 0u);
            float x[8];
            unpack16<T>(raw[k], x);
            float mul = negate ? -1.f : 1.f;
            if (!std::is_same<T, __half>::value) {
                float most = 0.f;
#pragma unroll
                for (int j = 0; j < 8; ++j) most = fmaxf(most, fabsf(x[j]));
#pragma unroll
                for (int o = LPR / 2; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
                // most = f * 2^ex, f in [1, 2): the row's largest goes to [2^14, 2^15)
                const int ex = (int)(__float_as_uint(most) >> 23) - 127;
                const int e = most > 0.f && ex < 128 ? min(14 - ex, 126) : 0;
                mul *= __int_as_float((e + 127) << 23);
                const float back = __int_as_float((127 - e) << 23);
#pragma unroll
                for (int o = 0; o < RPS; ++o) {
                    const float y = __shfl_sync(0xffffffffu, back, o * LPR);
                    if (lane == b + k * RPS + o) undo = y;
                }
            }
            uint32_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const __half2 y = __floats2half2_rn(x[2 * j] * mul, x[2 * j + 1] * mul);
                h[j] = *reinterpret_cast<const uint32_t*>(&y);
            }
            *reinterpret_cast<uint4*>(tile + row * 128 + (i / 8) * kPanel + (((i & 7) ^ (row & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
    }
    return undo;
}

// 64 scores of a lane's row that it does not see become -inf: cols of them are seen, less the blocks in masked.
template <int BS>
__device__ __forceinline__ void mask_scores(uint32_t (&s)[64], int cols, unsigned masked) {
#pragma unroll
    for (int i = 0; i < 64; ++i)
        if (i >= cols || (masked >> (i / BS) & 1)) s[i] = 0xff800000u;
}

// Largest of 64 scores, times the factors of their blocks; weight: the largest sum of such a score and its block's lv.
template <int BS>
__device__ __forceinline__ float row_max(const uint32_t (&s)[64], const float (&kf)[64 / BS], const float (&lv)[64 / BS], float& weight) {
    float top = -INFINITY;
    weight = -INFINITY;
#pragma unroll
    for (int h = 0; h < 64 / BS; ++h) {
        float x = -INFINITY, y = -INFINITY;  // two chains
#pragma unroll
        for (int k = 0; k < BS; k += 4) {
            x = fmaxf(x, fmaxf(__uint_as_float(s[BS * h + k]), __uint_as_float(s[BS * h + k + 1])));
            y = fmaxf(y, fmaxf(__uint_as_float(s[BS * h + k + 2]), __uint_as_float(s[BS * h + k + 3])));
        }
        const float most = fmaxf(x, y) * kf[h];
        top = fmaxf(top, most);
        weight = fmaxf(weight, most + lv[h]);
    }
    return top;
}

// P of 64 scores: exp2(score - mu) times its block's factor vf, as f16, over the scores in tensor memory; returns the sum of the
// exponentials.
template <int BS>
__device__ __forceinline__ float row_exp(uint32_t (&s)[64], uint32_t s_at, const float (&kf)[64 / BS], const float (&vf)[64 / BS], float mu) {
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int c = 0; c < 64; c += 32) {
#pragma unroll
        for (int i = c; i < c + 32; i += 2) {
            const int h = i / BS;
            const float2 x = fma2(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), make_float2(kf[h], kf[h]),
                                  make_float2(-mu, -mu));
            const float2 e = make_float2(exp2_approx(x.x), exp2_approx(x.y));
            sum = add2(sum, e);
            const float2 w = mul2(e, make_float2(vf[h], vf[h]));
            const __half2 p = __floats2half2_rn(w.x, w.y);
            s[i / 2] = *reinterpret_cast<const uint32_t*>(&p);
        }
        tmem_st16(s_at + c / 2, *reinterpret_cast<uint32_t(*)[16]>(&s[c / 2]));
    }
    return sum.x + sum.y;
}

// What the side ring holds of a half's blocks.
template <int N>
__device__ __forceinline__ void load_blocks(float (&x)[N], const float* from) {
    static_assert(N == 4 || N == 2, "blocks of 16 or 32 tokens");
    if constexpr (N == 4) *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(from);
    else *reinterpret_cast<float2*>(x) = *reinterpret_cast<const float2*>(from);
}
__device__ __forceinline__ float inverse(float p) { return __int_as_float(0x7f000000 - __float_as_int(p)); }  // of 2^-126 .. 2^126
__device__ __forceinline__ float power_of_two(float e) { return __int_as_float(((int)e + 127) << 23); }  // |e| <= 126, whole
// log2 of the power of two that P is relative to, from the references of weights and of exponents: P of the former's weight is in [1, 4).
__device__ __forceinline__ float reference(float weight, float m) {
    const float e = floorf(weight - m);
    return e == e ? fminf(fmaxf(e, -126.f), 126.f) : 0.f;  // (nothing seen yet, or an infinite score)
}

// A softmax warp: 32 rows of a stream's row tile, one per lane.
template <typename T, int D, int BS>
__device__ __forceinline__ void softmax_rows(const AttendArgs& a, const Workspace& ws, Smem<D>& sm) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = warp >> 2, r = (warp & 3) * 32 + lane;
    volatile int* abort = &sm.abort;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = sm.tmem + lanes + t * kTile, o_at = sm.tmem + lanes + 2 * kTile + t * D;
    const uint32_t other_o_at = sm.tmem + lanes + 2 * kTile + (t ^ 1) * D;
    Walk walk(ws, a.num_kv_heads, blockIdx.x, gridDim.x);
    unsigned pieces = 0, steps = 0, joins = 0, tiles_before = 0;  // so far
    // what the result of a piece needs; it is written after the next piece's queries are staged, which waits for nothing
    struct Result {
        size_t row_at;
        float* rec;
        bool live, warp_live, cut, join;
    } res{};
    // the row's references of exponents and of weights; the sum of its exponentials; 1 / the power of two that P is relative to
    float m = -INFINITY, w = -INFINITY, l = 0.f, vinv = 1.f;
    bool has_nan = false, pending = false;
#pragma unroll 1
    for (;;) {
        Piece p;
        Item it{};
        int n = 0, my_jobs = 0, bound = -1, seen_by_all = 0;
        float qf = 0.f;
        Result now{};
        const bool have = walk.next(&p);
        if (have) {
            it = item_of(a, p);
            n = p.end - p.begin;
            my_jobs = (it.jobs + 1 - t) / 2;
            if (my_jobs == 0 && !pending) {  // a single tile in a split piece is stream 0's
                tiles_before += n;
                continue;
            }
            const int first = p.row0 + (p.paired ? t * kTile : 0), v = first + r;  // row of the request
            const int token = v / it.group;
            now.live = v < it.rows;
            now.warp_live = first + (warp & 3) * 32 < it.rows;
            now.cut = p.begin > 0 || p.end < p.tiles;
            now.join = !p.paired && it.jobs > 1;
            now.rec = ws.records + ((size_t)blockIdx.x * 4 + (p.begin > 0 ? 0 : 2) + (p.paired ? t : 0)) * record_floats(D);
            now.row_at = now.live ? ((size_t)(it.first_token + token) * a.num_heads + p.kvh * it.group + (v - token * it.group)) * D : 0;
            if (now.live) bound = it.L - it.n + token;  // last position that the row sees
            seen_by_all = it.L - it.n + p.row0 / it.group;
            if (my_jobs > 0) {
                // the stream's last scores were waited for, so its query tile is free
                const float undo =
                    stage_query<T, D>(static_cast<const T*>(a.query), now.row_at, now.live, a.scale < 0.f, sm.q[t], (warp & 3) * 32);
                fence_proxy_async_smem();
                mbar_arrive(&sm.q_full[t]);
                qf = fabsf(a.scale) * 1.4426950408889634f * undo;
            }
        }

        if (pending) {  // the previous piece's result
            if (!warp_wait(&sm.o_full[t], pieces & 1, a.err, abort)) return;
            tc_fence_after();
            ++pieces;
            const float vref = inverse(vinv);
            float f0 = vref, f1 = 0.f;  // factors of this stream's output and of the other's
            uint32_t nan_from = has_nan ? 1u << t : 0u;
            if (res.join) {  // both streams have a part of the same rows, in the same lanes of tensor memory
                sm.state[t][r] = make_float4(m, l, vref, has_nan ? 1.f : 0.f);
                tc_fence_before();
                mbar_arrive(&sm.join_full);
                if (!warp_wait(&sm.join_full, joins & 1, a.err, abort)) return;
                tc_fence_after();
                const float4 o = sm.state[t ^ 1][r];
                const float mn = fmaxf(m, o.x);
                // a state without a maximum is empty, unless its sum is NaN
                const float w0 = m == -INFINITY ? (l != l ? 1.f : 0.f) : exp2_approx(m - mn);
                const float w1 = o.x == -INFINITY ? (o.y != o.y ? 1.f : 0.f) : exp2_approx(o.x - mn);
                f0 = vref * w0;
                f1 = o.z * w1;
                l = l * w0 + o.y * w1;
                m = mn;
                if (o.w != 0.f) nan_from |= 2u >> t;
            }
            if (res.warp_live) {
                const float inv = res.cut ? 1.f : (l == 0.f ? 0.f : 1.f / l);
                const int c0 = res.join ? t * (D / 2) : 0, c1 = res.join ? c0 + D / 2 : D;
#pragma unroll 1
                for (int c = c0; c < c1; c += 32) {
                    uint32_t s[32];
                    tmem_ld32(o_at + c, s);
                    tc_wait_ld(s);
#pragma unroll
                    for (int k = 0; k < 32; ++k) s[k] = __float_as_uint(__uint_as_float(s[k]) * f0);
                    if (res.join) {
                        uint32_t o[32];
                        tmem_ld32(other_o_at + c, o);
                        tc_wait_ld(o);
#pragma unroll
                        for (int k = 0; k < 32; ++k) s[k] = __float_as_uint(fmaf(__uint_as_float(o[k]), f1, __uint_as_float(s[k])));
                    }
                    if (nan_from) {
                        const uint32_t nan = (nan_from & 1 ? sm.nan_row[0][r][c / 32] : 0u) | (nan_from & 2 ? sm.nan_row[1][r][c / 32] : 0u);
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (nan >> k & 1) s[k] = 0x7fc00000u;
                    }
                    if (res.live && res.cut) {
                        uint4* d = reinterpret_cast<uint4*>(res.rec + 2 * kTile + (size_t)r * D + c);
#pragma unroll
                        for (int k = 0; k < 8; ++k) d[k] = make_uint4(s[4 * k], s[4 * k + 1], s[4 * k + 2], s[4 * k + 3]);
                    } else if (res.live) {
                        uint4* d = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + res.row_at + c);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            T y[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) y[i] = from_float<T>(__uint_as_float(s[8 * k + i]) * inv);
                            d[k] = *reinterpret_cast<const uint4*>(y);
                        }
                    }
                }
                if (res.cut && res.live && c0 == 0) {
                    res.rec[r] = m;
                    res.rec[kTile + r] = l;
                }
            }
            tc_fence_before();
            if (res.join) {  // neither stream's output is written again before both have read it
                mbar_arrive(&sm.join_done);
                if (!warp_wait(&sm.join_done, joins & 1, a.err, abort)) return;
                ++joins;
            }
            pending = false;
        }
        if (!have) return;
        if (my_jobs == 0) {
            tiles_before += n;
            continue;
        }

        res = now;
        pending = true;
        m = w = -INFINITY;
        l = 0.f;
        has_nan = false;
#pragma unroll 1
        for (int step = 0; step < my_jobs; ++step, ++steps) {
            const int local = p.paired ? step : 2 * step + t;
            const unsigned count = tiles_before + local;
            const int p0 = (p.begin + local) * kTile, slot = count % kRing;
#pragma unroll 1
            for (int half = 0; half < 2; ++half) {
                if (!warp_wait(&sm.s_full[t][half], steps & 1, a.err, abort)) return;
                tc_fence_after();
                if (!now.warp_live) {  // rows that nobody reads: whatever lies there may be multiplied
                    if (lane == 0) mbar_arrive(&sm.p_full[t][half]);
                    continue;
                }
                const uint32_t at = s_at + 64 * half;
                uint32_t s[64];
                tmem_ld32(at, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
                tmem_ld32(at + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
                alignas(16) float ks[64 / BS], vs[64 / BS], lv[64 / BS];
                load_blocks(ks, sm.ks[slot] + half * (64 / BS));
                load_blocks(lv, sm.lv[slot] + half * (64 / BS));
                // factors of the scores; kept above zero, so that masked scores stay -inf
                float kf[64 / BS];
#pragma unroll
                for (int k = 0; k < 64 / BS; ++k) kf[k] = fmaxf(ks[k] * qf, 1e-38f);
                const unsigned masked = sm.masked[slot] >> (half * (64 / BS));
                const int cols = bound - p0 - 64 * half + 1;  // columns that the row sees, if below 64
                const bool whole = __all_sync(0xffffffffu, !now.live || cols >= 64) && (masked & ((1u << (64 / BS)) - 1)) == 0;
                tc_wait_ld(s);
                if (!whole) mask_scores<BS>(s, cols, masked);
                float weight;  // log2 of the row's largest exponential times V scale, less what the scale has past its power of two
                const float top = row_max<BS>(s, kf, lv, weight);
                if (step == 0 && half == 0) {
                    m = top;
                    w = weight;
                    vinv = power_of_two(-reference(w, m));
                } else if (__any_sync(0xffffffffu, top > m + 8.f || weight > w + 8.f)) {
                    // The output so far has to be there.  (Its barrier is waited for only here: the phase before the one that is
                    // meant is over, because this half's scores were issued after the output of the half before the last.)
                    const unsigned last = half ? steps : steps - 1;
                    if (!warp_wait(&sm.pv_done[t][half ^ 1], last & 1, a.err, abort)) return;
                    tc_fence_after();
                    const float mn = fmaxf(m, top), wn = fmaxf(w, weight), vn = -reference(wn, mn);
                    const float f = mn == -INFINITY ? 1.f : exp2_approx(m - mn);
                    // (one power: the two that it is made of may be past float32's ends where it is not)
                    const float of = mn == -INFINITY ? 1.f : exp2_approx(m - mn + (vn + reference(w, m)));
                    l *= f;
                    m = mn;
                    w = wn;
                    vinv = power_of_two(vn);
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t o[16];
                        tmem_ld16(o_at + c, o);
                        tc_wait_ld(o);
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * of);
                        tmem_st16(o_at + c, o);
                    }
                }
                // Factors of P.  (One past float32's end is that of a block that the row does not see, or of one whose exponentials are below
                // 2^-110: kept finite, it leaves their zeros zeros.)
                load_blocks(vs, sm.vs[slot] + half * (64 / BS));
                float vf[64 / BS];
#pragma unroll
                for (int k = 0; k < 64 / BS; ++k) vf[k] = fminf(vs[k] * vinv, 1e38f);
                l += row_exp<BS>(s, at, kf, vf, m == -INFINITY ? 0.f : m);
                if (half == 1 && p0 + kTile - 1 > seen_by_all) {  // a tile whose V was searched for NaN
                    const unsigned f = 2 * tiles_before + value_fill(p.paired, n, local);
                    if (!warp_wait(&sm.kv_full[f % kBuffers], (f / kBuffers) & 1, a.err, abort)) return;
                    const int at_slot = count % kNanRing, all = min(kTile, bound - p0 + 1);
                    if (sm.nan_any[at_slot][0] | sm.nan_any[at_slot][1] | sm.nan_any[at_slot][2] | sm.nan_any[at_slot][3]) {
#pragma unroll 1
                        for (int i = 0; i < D / 32; ++i) {
                            uint32_t bits = has_nan ? sm.nan_row[t][r][i] : 0u;
#pragma unroll 1
                            for (int k = 0; k < all; ++k)
                                if (!(sm.masked[slot] >> (k / BS) & 1))
                                    bits |= (uint32_t)sm.nan_at[at_slot][k][2 * i] | ((uint32_t)sm.nan_at[at_slot][k][2 * i + 1] << 16);
                            sm.nan_row[t][r][i] = bits;
                        }
                        has_nan = true;
                    }
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.p_full[t][half]);
            }
        }
        tiles_before += n;
    }
}

template <typename T, int D, int BS>
__global__ void __launch_bounds__(kThreads, 1) attend_fp8_kernel(const AttendArgs a, const Workspace ws,
                                                                 const __grid_constant__ CUtensorMap kmap,
                                                                 const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ unsigned char raw_smem[];
    Smem<D>& sm = *reinterpret_cast<Smem<D>*>(((uintptr_t)raw_smem + 1023) & ~(uintptr_t)1023);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.q_full[i], 128);
            for (int h = 0; h < 2; ++h) {
                mbar_init(&sm.s_full[i][h], 1);
                mbar_init(&sm.p_full[i][h], 4);
                mbar_init(&sm.pv_done[i][h], 1);
            }
            mbar_init(&sm.o_full[i], 1);
        }
        for (int i = 0; i < kRing; ++i) {
            mbar_init(&sm.side_full[i], 1);
            mbar_init(&sm.copied[i], 1);
        }
        for (int i = 0; i < Smem<D>::kRaw; ++i) {
            mbar_init(&sm.raw_full[i], 1);
            mbar_init(&sm.raw_empty[i], kWidenWarps);
        }
        for (int i = 0; i < kBuffers; ++i) {
            mbar_init(&sm.kv_full[i], kWidenWarps);
            mbar_init(&sm.kv_empty[i], 2);
        }
        mbar_init(&sm.join_full, kSoftmaxWarps * 32);
        mbar_init(&sm.join_done, kSoftmaxWarps * 32);
        mbar_init(&sm.drain[0], 1);
        mbar_init(&sm.drain[1], 1);
        sm.abort = 0;
        fence_barrier_init();
    }
    if (warp == kIssueWarp) tmem_alloc(&sm.tmem, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    griddep_wait();
    griddep_launch_dependents();
    if (warp < kSoftmaxWarps) {
        softmax_rows<T, D, BS>(a, ws, sm);
    } else if (warp < kSoftmaxWarps + kWidenWarps) {
        widen_tiles<D, BS>(a, ws, sm);
    } else if (warp == kCopyWarp) {
        copy_tiles<D, BS>(a, ws, sm, &kmap, &vmap);
    } else if (warp == kLookWarp) {
        look_ahead<D, BS>(a, ws, sm);
    } else {
        const int t = __shfl_sync(0xffffffffu, warp - kIssueWarp, 0);
        issue_products<D>(a, ws, sm, t);
        if (__any_sync(0xffffffffu, sm.abort)) {  // products still in flight read shared and tensor memory
            int never = 0;
            tc_commit(&sm.drain[t]);
            mbar_wait_bounded(&sm.drain[t], 0, a.err, &never);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kIssueWarp) tmem_free(sm.tmem, 512);
}

// Joins the partial results of the units that share boundaries cut.  CTA (boundary, rows): the first boundary inside a unit
// has it; a warp per row, D / 32 elements per lane.
constexpr int kJoinThreads = 256;
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) attend_join_kernel(const AttendArgs a, const Workspace ws, int ctas) {
    griddep_wait();
    griddep_launch_dependents();
    constexpr int E = D / 32;
    using Vec = typename std::conditional<E == 4, float4, float2>::type;
    const long long cost = ws.head->cost, share = share_of(cost, ctas);
    const int c1 = blockIdx.x + 1;  // boundary: the start of CTA c1's share
    const long long x = share * c1;
    if (x >= cost) return;
    const Entry en = ws.entries[find_entry(ws.entries, ws.head->entries, x)];
    const long long each = unit_cost(en.tiles, en.paired);
    const int kvh = (int)((x - en.first) / each);
    const long long unit = en.first + kvh * each, end = unit + each;
    if (x == unit || share * (c1 - 1) > unit) return;  // not inside, or not the first inside
    // pieces: CTA c has tiles [cut(c), cut(c + 1))
    auto cut = [&](int c) {
        const long long from = share * c - unit;
        return tiles_in(from, en.tiles, en.paired != 0);
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

template <typename T, int D, int BS>
cudaError_t attend_typed(const AttendArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t stream) {
    const int group = a.num_heads / a.num_kv_heads, ctas = a.num_sms;
    const size_t cap = max_entries(a.num_seqs, a.num_tokens, group);
    char* base = static_cast<char*>(a.workspace);
    Workspace ws;
    ws.head = reinterpret_cast<PlanHead*>(base);
    ws.entries = reinterpret_cast<Entry*>(base + 256);
    ws.records = reinterpret_cast<float*>(base + 256 + align256((cap + 1) * sizeof(Entry)));
    cudaError_t e = launch_pdl(attend_plan_kernel, dim3(1), dim3(kPlanThreads), (size_t)(a.num_seqs + 1) * sizeof(int), stream, a, ws,
                               (int)cap);
    if (e != cudaSuccess) return e;
    const size_t smem = sizeof(Smem<D>) + 1024;
    e = cudaFuncSetAttribute(attend_fp8_kernel<T, D, BS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(attend_fp8_kernel<T, D, BS>, dim3((unsigned)ctas), dim3(kThreads), smem, stream, a, ws, kmap, vmap);
    if (e != cudaSuccess || ctas < 2) return e;
    // (a boundary's 256 rows on 8 CTAs, four rows a warp, measured when chosen: short mixed requests 88.7 us; 4 CTAs 95, 16 89.7, 32 93)
    return launch_pdl(attend_join_kernel<T, D>, dim3((unsigned)(ctas - 1), 8), dim3(kJoinThreads), 0, stream, a, ws, ctas);
}

}  // namespace

size_t attend_fp8_workspace_bytes(int num_sms, int num_seqs, int num_tokens, int num_heads, int num_kv_heads, int head_dim, int,
                                  int) {
    const size_t cap = max_entries(num_seqs, num_tokens, num_heads / num_kv_heads);
    return 256 + align256((cap + 1) * sizeof(Entry)) + (size_t)num_sms * 4 * record_floats(head_dim) * sizeof(float);
}

cudaError_t attend_fp8_launch(const AttendArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t stream) {
    const int pick = (a.dtype == 1 ? 4 : 0) + (a.head_dim == 64 ? 2 : 0) + (a.block_size == 32 ? 1 : 0);
    switch (pick) {
        case 0: return attend_typed<__nv_bfloat16, 128, 16>(a, kmap, vmap, stream);
        case 1: return attend_typed<__nv_bfloat16, 128, 32>(a, kmap, vmap, stream);
        case 2: return attend_typed<__nv_bfloat16, 64, 16>(a, kmap, vmap, stream);
        case 3: return attend_typed<__nv_bfloat16, 64, 32>(a, kmap, vmap, stream);
        case 4: return attend_typed<__half, 128, 16>(a, kmap, vmap, stream);
        case 5: return attend_typed<__half, 128, 32>(a, kmap, vmap, stream);
        case 6: return attend_typed<__half, 64, 16>(a, kmap, vmap, stream);
        default: return attend_typed<__half, 64, 32>(a, kmap, vmap, stream);
    }
}

}  // namespace pa
