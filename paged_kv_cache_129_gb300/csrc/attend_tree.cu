// Attention of the nodes of drafted trees over a paged 16-bit cache, on tcgen05 tensor cores.
//
// Request b has the rows q_offsets[b] .. q_offsets[b + 1] - 1, n_b nodes whose keys and values are the last n_b of its L_b positions.  A
// row sees the L_b - n_b positions before them, and node j where bit j of its words of tree_mask is set:
//     out = sum softmax(scale q k_j) v_j over what it sees; zeros where that is nothing.
//
// Rows.  The g query heads of a kv head and the request's nodes form n_b * g rows (row v: node v / g, head v % g), cut into tiles of 128,
// the M of the products; keys come in tiles of 128 positions.  A CTA has two streams of softmax warps:
//   paired  two row tiles share every key tile, a stream each;
//   split   a single row tile (small trees, single tokens, the rest of a wide tree): each stream takes one half, 64 positions, of every key
//           tile, and they join their results at the end.
// Work.  A unit is (request, kv head, pair of row tiles).  All units' key tiles are laid end to end, weighted by their cost, and cut into one
// equal contiguous share per CTA, of which there is one per SM; every CTA adds up the requests' costs for itself and finds its own.  Units
// cut by a share boundary leave float32 partial results (two slots per CTA), joined by a second kernel.
// Operands.  K and V go from the cache's blocks straight into operand tiles, one bulk tensor copy per block: a block's rows as groups of
// eight by panels of 64 elements, which is the order that both products read (K by rows, V by columns) with uniform strides.  A block
// that is not there is copied from behind the pool, as zeros.
// What a row does not see.  Its scores become -inf, its weights zeros; but 0 * NaN is NaN, so V must be finite there.  Blocks behind the
// context are zeros; in the tiles that hold nodes or the context's end a warp clears the rows behind the end, and looks for infinities and
// NaN in the nodes' V: these are taken out, noted, and put into the outputs of the rows that see them.
// Numbers.  Scores, maxima, sums and the output accumulate in float32.  A weight is rounded to the cache's type for the second
// product (half a step: bf16 2^-8 of it, as the output; f16 2^-11, and 2^-25 of the reference below 2^-14).  The sum that divides takes the
// rounded weights, so that those that multiply V sum to one: a row over equal values returns them, and a dominant weight's rounding cancels (what weights
// alone put in, restated in float64: as much as with the sum of the unrounded ones where scores are flat, half of it and less where their deviation
// is 3 or 6).  The reference of a row's exponents is its maximum when it was last moved: all rows of a warp move to their maxima once
// one of them is 2^8 above its own, so that rescaling the output in tensor memory is rare, and weights are 2^8 at most.
// Bound.  Long contexts (eight requests of 32k - 128k positions with 1 - 8 nodes) HBM: 475 us, 7.0 TB/s.  Steps (64 requests of 512 - 4096 with 16
// nodes) 68 us, 4.6 TB/s: of an SM's 120 000 cycles 85 000 are its share of HBM's time, 15 000 pass before the first scores and the rest at the
// pieces' ends.  Wide trees (16 requests of 2k - 8k with 48 - 128 nodes) 134 us, 0.90 PFLOP/s, tensor pipe 51 % busy: the softmax warps, whose code is
// fetched as slowly as it is run.  Short mixed requests of D = 64 28 us: the same 15 000 cycles, the pieces' ends, the second launch.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "pa_common.cuh"
#include "tcgen05.cuh"
#include "tree_ops.h"

namespace pa {

namespace {

constexpr int kJoinThreads = 128;
size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
__host__ __device__ inline size_t record_floats(int D) { return (size_t)kTile * (D + 2); }

constexpr int kSoftmaxWarps = 8;  // four per stream
constexpr int kIssueWarp = kSoftmaxWarps;  // two, one per stream
constexpr int kCopyWarp = kIssueWarp + 2, kLookWarp = kCopyWarp + 1, kCleanWarp = kLookWarp + 1, kQueryWarp = kCleanWarp + 1;
constexpr int kThreads = (kQueryWarp + 1) * 32;
constexpr int kPieces = 4;  // pieces of the share that the look-ahead warp may be ahead of the others

// Cost of work in shares: of a key tile of a pair and of a split piece, and of a unit besides its tiles.  Measured when chosen (steps / wide
// trees / short mixed D = 64, us): 6, 4, 12: 68.8 / 137 / 27.8; 6, 4, 16: 69.2 / 136 / 30.5; 6, 4, 20: 69.2 / 137 / 31.4; 5, 4, 16: 69.0 / 138 / 31.3;
// 7, 4, 16: 68.9 / 135 / 30.8.  (By the clock of an SM a split tile takes 2100 - 2600 cycles, a paired one 3000 - 3400, a piece 7000 - 9500 besides.)
constexpr int kPairedCost = 6, kSplitCost = 4, kUnitCost = 12;
constexpr int kMinShare = kUnitCost + 4 * kSplitCost;  // a CTA's share is not worth less than the pieces' overhead

// A request as the shares see it: n nodes on L positions.
struct Request {
    int L, n, first_token, rows, tiles;
    bool bad;  // its lengths or offsets are none
    Request() = default;
    __device__ __forceinline__ Request(const TreeAttendArgs& a, int b) {
        const int given = a.context_lens[b], lo = a.q_offsets[b], hi = a.q_offsets[b + 1], most = a.max_blocks * a.block_size;
        const bool run = is_run(lo, hi, a.num_tokens);
        L = max(0, min(given, most));
        n = run ? hi - lo : 0;
        bad = !run || given < n || given > most;
        first_token = lo;
        rows = n * a.group;
        tiles = max(1, (L + kTile - 1) / kTile);
    }
    __device__ __forceinline__ int entries() const { return (rows + 2 * kTile - 1) / (2 * kTile); }  // pairs of row tiles
    __device__ __forceinline__ bool paired(int e) const { return rows - e * 2 * kTile > kTile; }
    __device__ __forceinline__ long long cost(bool pair) const { return kUnitCost + (long long)tiles * (pair ? kPairedCost : kSplitCost); }
    __device__ __forceinline__ long long head_cost() const {  // of a kv head's units
        const int full = rows / (2 * kTile), rest = rows % (2 * kTile);
        return full * cost(true) + (rest ? cost(rest > kTile) : 0);
    }
};

// Key tiles of a unit before cost position x inside it (a cut falls between tiles; both sides of a boundary round alike).  A cut so near to
// an end of the unit that the piece would cost more than its tiles goes to the end (1, that is not at all: 74.5 / 158 / 36.9 us where 3 took 72.5 / 157 /
// 35.2, 2 72.1 / 158 / 37.1, 4 73.4 / 157 / 35.1).
constexpr int kSnap = 3;
__device__ __forceinline__ int tiles_in(long long x, int tiles, bool paired) {  // (a unit's tiles: below 2^24)
    const unsigned cost = (unsigned)max(0ll, min(x - kUnitCost, (long long)tiles * (paired ? kPairedCost : kSplitCost)));
    const int cut = (int)(paired ? (cost + kPairedCost - 1) / kPairedCost : (cost + kSplitCost - 1) / kSplitCost);
    return cut == tiles ? tiles : cut < kSnap ? 0 : cut > tiles - kSnap ? tiles : cut;
}

// x / y; of what fits 32 bits, which is nearly all, in a fifth of the time.
__device__ __forceinline__ long long quotient(long long x, long long y) {
    return ((unsigned long long)(x | y) >> 32) == 0 ? (long long)((unsigned)x / (unsigned)y) : x / y;
}

// Where a CTA's share [pos, stop) of the total cost begins: a unit that starts at `unit`.
struct Start {
    long long pos, stop, unit, share;
    int seq, kvh, entry;
    Request r;
};

// A boundary that cuts a unit: what the joining kernel needs.  CTAs first .. last have parts of it; last 0: nothing to join.
struct Seam {
    long long unit, share;
    int seq, kvh, row0, rows, tiles, paired, first, last;
};

struct Scratch {
    long long cost[kThreads / 32], rows[kThreads / 32];
    Start start;
};

// The share of this CTA; all its threads.  A run of requests per thread, their costs summed over the CTA; whoever's run the share begins
// in finds the unit.
__device__ __forceinline__ Start find_share(const TreeAttendArgs& a, Scratch& sc) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = a.num_seqs, H = a.num_kv_heads;
    const int per = (B + kThreads - 1) / kThreads, b0 = min(B, tid * per), b1 = min(B, b0 + per);
    long long cost = 0, rows = 0, head = 0;
    Request r{};
    for (int b = b0; b < b1; ++b) {
        r = Request(a, b);
        head = r.head_cost();
        cost += head * H;
        rows += r.n;
        if (blockIdx.x == 0 && (r.bad || r.n > 64 * a.mask_words)) atomicOr(a.err, kErrBadContext);
    }
    long long sum = cost;  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, sum, o), y = __shfl_xor_sync(0xffffffffu, rows, o);
        if (lane >= o) sum += x;
        rows += y;
    }
    if (lane == 31) sc.cost[warp] = sum, sc.rows[warp] = rows;
    if (tid == 0) sc.start.seq = -1;
    __syncthreads();
    long long total = 0, before = 0, all_rows = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w == warp) before = total;
        total += sc.cost[w];
        all_rows += sc.rows[w];
    }
    if (all_rows > a.num_tokens) {  // runs that overlap
        if (blockIdx.x == 0 && tid == 0) atomicOr(a.err, kErrBadContext);
        total = 0;
    }
    const long long even = quotient(total + gridDim.x - 1, gridDim.x), share = even > kMinShare ? even : kMinShare, pos = share * blockIdx.x;
    long long at = before + sum - cost;
    if (pos < total && at <= pos && pos < at + cost) {
        int b = b1 - 1;
        if (per > 1)  // (else the only request is at hand)
            for (b = b0;; ++b) {
                r = Request(a, b);
                head = r.head_cost();
                if (pos < at + head * H) break;
                at += head * H;
            }
        const int kvh = (int)quotient(pos - at, head);
        at += kvh * head;
        const long long pair = r.cost(true);
        const int e = min((int)quotient(pos - at, pair), r.rows / (2 * kTile));
        sc.start = Start{pos, min(pos + share, total), at + e * pair, share, b, kvh, e, r};
    }
    __syncthreads();
    return sc.start;
}

// Sizes and places of the operand tiles.  A key tile is 16 groups of 8 positions; a group is D / 64 panels of 8 rows by 128 bytes,
// swizzled (16-byte unit u of row r at u ^ r), which is how a block's copy leaves it.
template <int D>
struct Tile {
    static constexpr int kOperand = kTile * D * 2;
    static constexpr int kBuffers = D == 128 ? 5 : 10;            // K or V tiles in shared memory: 160 KB
    static constexpr int kRing = D == 128 ? 8 : 16;               // slots of per-tile side data (places of blocks), see look_ahead()
    static constexpr int kAhead = kRing - (kBuffers + 4) / 2;     // key tiles that look_ahead() may be ahead of the copies
    static constexpr int kCleanRing = D == 128 ? 4 : 8;           // cleaned V tiles whose notes are kept, see clean_tiles()
    static constexpr int kGroup = D * 16;                         // bytes of a group
    // offset of 16 bytes (8 elements, unit u) of row r
    static __device__ __forceinline__ int at(int r, int u) { return (r >> 3) * kGroup + (u >> 3) * 1024 + (r & 7) * 128 + (((u & 7) ^ (r & 7)) << 4); }
};

// What a piece of the share is to every role; begin == end behind the last one.
struct Job {
    int L, n, first_token, seq;  // length, nodes, row of the first node
    int row0, kvh, tiles, begin, end, paired;
};

template <int D>
struct Smem {
    unsigned char q[2][Tile<D>::kOperand];  // row tiles, used in turn: of a split piece one, of a pair both
    unsigned char kv[Tile<D>::kBuffers][Tile<D>::kOperand];
    float2 state[2][kTile];                // at the end of a split piece: both streams' m and l (sign bit: there is a note)
    int place[Tile<D>::kRing][8];          // a tile's blocks: their first group of eight rows
    unsigned masked[Tile<D>::kRing];       // which have an id outside the pool; bit 31: the tile's V is cleaned
    unsigned special[Tile<D>::kCleanRing]; // whether a cleaned tile had infinities or NaN
    Job jobs[kPieces];
    uint64_t job_full[kPieces], job_free[kPieces], side_full[Tile<D>::kRing], copied[Tile<D>::kRing];
    uint64_t q_full[2], q_free[2], kv_full[Tile<D>::kBuffers], kv_empty[Tile<D>::kBuffers];
    uint64_t dirty_full[Tile<D>::kCleanRing], clean_full[Tile<D>::kCleanRing];
    uint64_t s_full[2][2], p_full[2][2], pv_done[2][2], o_full[2], join_full, join_done, drain[2];
    uint32_t tmem;
    volatile int abort;
};
static_assert(sizeof(Smem<128>) <= 227 * 1024, "fits an SM");

// Notes of infinities and NaN, in the workspace (there is hardly ever one): bit set where an element was +inf or NaN, and where it was
// -inf or NaN.  at: per cleaned tile and position; row: per row of a stream, the elements of its output that they reach.
template <int D>
struct Notes {
    uint8_t at[Tile<D>::kCleanRing][2][kTile][D / 8];
    uint32_t row[2][2][kTile][D / 32];
};

// The order in which a piece's n key tiles go through the buffers.  Paired: K0 V0 K1 V1 ...  Split: K one tile ahead, K0 K1 V0 K2
// V1 ... V(n-2) V(n-1), because the scores of a tile are made before the output of the tile before it.
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
__device__ __forceinline__ int value_fill(bool paired, int n, int tile) {
    return paired ? 2 * tile + 1 : tile == n - 1 ? 2 * n - 1 : 2 * tile + 2;
}

// The first key tile whose V is cleaned: the one with the request's first node (or the context's end).
__device__ __forceinline__ int first_cleaned(const Job& j) { return max(0, j.L - j.n) / kTile; }

// Tensor memory: per stream two buffers of 64 columns, used in turn, for the scores of a half and then, over the first of them, the 32 columns of
// weights P made of them; behind both streams' D columns of output each.  The scores of a half are issued right behind the output of the half
// before the last, which has then read the P that they overwrite, and are ready when their turn comes.  (Scores of a pair in products of 128
// columns, 66 cycles where two of 64 take 100: every tile waited for its products, 4570 cycles a tile, and as long with the streams
// taking turns.)
template <int D>
__device__ __forceinline__ uint32_t output_at(int t) { return 256 + t * D; }

// A bounded wait by a whole warp: all lanes go on, or none.  (Tried once before warp_wait()'s loop: 157 to 150 us for wide trees when added.)
__device__ __forceinline__ bool ready(uint64_t* bar, unsigned parity, unsigned* err, volatile int* abort) {
    return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || warp_wait(bar, parity, err, abort);
}

// Piece i of the share, for a warp of any role but the look-ahead's, which writes them; false if a wait gave up.
constexpr int kReaders = kQueryWarp;  // (all roles' warps but one)
template <int D>
__device__ __forceinline__ bool read_job(Smem<D>& sm, unsigned i, Job* job, unsigned* err) {
    if (!ready(&sm.job_full[i % kPieces], (i / kPieces) & 1, err, &sm.abort)) return false;
    *job = sm.jobs[i % kPieces];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&sm.job_free[i % kPieces]);
    return true;
}

// The boundary at a share's start, if it is the first inside its unit: the share before begins at the unit, or before it.
__device__ __forceinline__ Seam seam_of(const Start& s) {
    if (s.seq < 0 || s.pos <= s.unit || s.pos - s.share > s.unit) return Seam{};
    const bool pair = s.r.paired(s.entry);
    return Seam{s.unit, s.share, s.seq, s.kvh, s.entry * 2 * kTile, min(2 * kTile, s.r.rows - s.entry * 2 * kTile), s.r.tiles, pair,
                (int)blockIdx.x - 1, (int)quotient(s.unit + s.r.cost(pair) - 1, s.share)};
}

// The look-ahead warp: the places of block after block into the side ring, up to kAhead tiles before they are copied and across the ends
// of pieces, so that the tables' latency is not waited for.
// Side data of tile i sits in slot i % kRing, which was tile i - kRing's, last looked at by the softmax before P of that tile is there, so before
// its V's buffer is released.  When K of tile j is copied, fill 2j - 1 at least (see fill_of()), fill 2j - 1 - kBuffers was released by both
// streams, which release in order; V of tile g is fill 2g + 2 at most.  Tile i is looked at once K of tile i - kAhead is copied: with g = i - kRing,
// 2 (i - kRing) + 2 <= 2 (i - kAhead) - 1 - kBuffers.
template <int D, int BS>
__device__ __forceinline__ void look_ahead(const TreeAttendArgs& a, Seam* seams, Smem<D>& sm, const Start& start) {
    constexpr int BLOCKS = kTile / BS, RING = Tile<D>::kRing, AHEAD = Tile<D>::kAhead;
    static_assert(2 * (RING - AHEAD) >= Tile<D>::kBuffers + 3 && AHEAD > 1, "a slot's tile is done with when it is written again");
    const int lane = threadIdx.x & 31;
    const int behind = a.num_blocks * a.num_kv_heads * (BS / 8);  // the first group behind the pool: copied as zeros
    int seq = start.seq, kvh = start.kvh, e = start.entry;
    long long unit = start.unit;  // where the unit begins
    bool more = seq >= 0, taken = false;  // taken: the unit at hand is behind us
    Request r = start.r;
    unsigned tiles = 0;
    // The unit behind the one at hand; false: there is none.  Requests without nodes, which a captured batch may hold by the thousand, are
    // passed 32 at a time, a lane each, and behind the end of the share not at all (32 requests alone 46 us, in front of 8160 empty slots 56; passed
    // one by one, before the piece at hand was given to the other roles, 747).
    auto next_unit = [&] {
        if (++e < r.entries()) return true;
        e = 0;
        if (++kvh < a.num_kv_heads) return true;
        kvh = 0;
        for (++seq; seq < a.num_seqs; seq += 32) {
            const unsigned nodes = __ballot_sync(0xffffffffu, seq + lane < a.num_seqs && Request(a, min(seq + lane, a.num_seqs - 1)).rows > 0);
            if (nodes) {
                seq += __ffs(nodes) - 1;
                r = Request(a, seq);
                return true;
            }
        }
        return false;
    };
#pragma unroll 1
    for (unsigned i = 0;; ++i) {
        Job j{};
        while (more && j.begin == j.end) {  // the next unit with tiles in the share
            if (taken && !next_unit()) break;
            const bool pair = r.paired(e);
            j = Job{r.L, r.n, r.first_token, seq, e * 2 * kTile, kvh, r.tiles, tiles_in(start.pos - unit, r.tiles, pair),
                    tiles_in(start.stop - unit, r.tiles, pair), pair};
            unit += r.cost(pair);
            more = unit < start.stop;
            taken = true;
        }
        const bool have = j.begin < j.end;
        if (i >= kPieces && !ready(&sm.job_free[i % kPieces], (i / kPieces - 1) & 1, a.err, &sm.abort)) return;
        if (lane == 0) {
            sm.jobs[i % kPieces] = j;
            mbar_arrive(&sm.job_full[i % kPieces]);
        }
        if (i == 0 && lane == 0) seams[blockIdx.x] = seam_of(start);
        if (!have) return;
        const int used = (j.L + BS - 1) / BS, cleaned = first_cleaned(j);
        const int32_t* table = a.block_tables + (size_t)j.seq * a.max_blocks;
        // lane l < BLOCKS has block l of a tile
        auto wanted = [&](int tile) { return lane < BLOCKS && tile < j.end && tile * BLOCKS + lane < used; };
        int id = wanted(j.begin) ? table[j.begin * BLOCKS + lane] : -1;
        for (int tile = j.begin; tile < j.end; ++tile, ++tiles) {
            const bool mine = wanted(tile), in = mine && id >= 0 && id < a.num_blocks;
            if (mine && !in) atomicOr(a.err, kErrBadTable);
            const int place = in ? (id * a.num_kv_heads + j.kvh) * (BS / 8) : behind;
            id = wanted(tile + 1) ? table[(tile + 1) * BLOCKS + lane] : -1;
            const unsigned masked = __ballot_sync(0xffffffffu, mine && !in) | (tile >= cleaned ? 1u << 31 : 0u);
            if (tiles >= AHEAD) {
                const unsigned before = tiles - AHEAD;
                if (!ready(&sm.copied[before % RING], (before / RING) & 1, a.err, &sm.abort)) return;
            }
            const int slot = tiles % RING;
            if (lane < 8) sm.place[slot][lane] = place;
            if (lane == 0) sm.masked[slot] = masked;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.side_full[slot]);
        }
    }
}

// One block of a kv head, K or V: box (64 elements, 8 rows, panels, groups) at group `place`.  One elected lane.
__device__ __forceinline__ void copy_block(void* dst, const CUtensorMap* map, int place, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\t"
        "@q cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %2, %2, %3}], [%4];\n\t}" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(place), "r"(smem_addr(bar))
        : "memory");
}

// The copy warp.  V that is cleaned arrives on a barrier of the cleaning warp's, which then says that the buffer is full.
template <int D, int BS>
__device__ __forceinline__ void copy_tiles(const TreeAttendArgs& a, Smem<D>& sm, const CUtensorMap* kmap, const CUtensorMap* vmap) {
    constexpr int BLOCKS = kTile / BS, N = Tile<D>::kBuffers, RING = Tile<D>::kRing, kCleanRing = Tile<D>::kCleanRing;
    const int lane = threadIdx.x & 31;
    unsigned fills = 0, tiles = 0, cleaned = 0, dirty = 0;  // dirty: buffers whose last fill is one that is cleaned
    bool ok = true;
#pragma unroll 1
    for (unsigned piece = 0; ok; ++piece) {
        Job job;
        ok = read_job(sm, piece, &job, a.err);
        if (ok && job.begin == job.end) return;
        const int n = ok ? job.end - job.begin : 0;
#pragma unroll 1
        for (int i = 0; i < 2 * n; ++i, ++fills) {
            const Fill f = fill_of(job.paired, n, i);
            const int buf = fills % N;
            const unsigned tile = tiles + f.tile, side = tile % RING;
            ok = f.value || ready(&sm.side_full[side], (tile / RING) & 1, a.err, &sm.abort);
            ok = ok && ready(&sm.kv_empty[buf], ((fills / N) & 1) ^ 1, a.err, &sm.abort);
            if (!ok) break;
            const bool clean = f.value && (sm.masked[side] >> 31);
            uint64_t* bar = clean ? &sm.dirty_full[cleaned % kCleanRing] : &sm.kv_full[buf];
            dirty = (dirty & ~(1u << buf)) | ((unsigned)clean << buf);
            cleaned += clean;
            const int place = sm.place[side][lane & 7];
            if (lane == 0) {
                mbar_arrive_expect_tx(bar, Tile<D>::kOperand);
                if (!f.value) mbar_arrive(&sm.copied[side]);
            }
            __syncwarp();
            const CUtensorMap* map = f.value ? vmap : kmap;
#pragma unroll
            for (int j = 0; j < BLOCKS; ++j)
                copy_block(sm.kv[buf] + j * (BS * D * 2), map, __shfl_sync(0xffffffffu, place, j), bar);
        }
        tiles += n;
    }
    if (!ok) {  // copies still under way must land before the CTA's shared memory goes
        int never = 0;
        for (unsigned f = fills; f > 0 && f + N > fills; --f) {
            const int buf = (f - 1) % N;
            if (dirty >> buf & 1) {
                --cleaned;
                mbar_wait_bounded(&sm.dirty_full[cleaned % kCleanRing], (cleaned / kCleanRing) & 1, a.err, &never);
            } else {
                mbar_wait_bounded(&sm.kv_full[buf], ((f - 1) / N) & 1, a.err, &never);
            }
        }
    }
}

// Per element of a word of two: bit 15 set where it is infinite or NaN.
template <typename T>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
    constexpr uint32_t kStep = std::is_same<T, __half>::value ? 0x0400u : 0x0080u;  // from the largest exponent to bit 15
    return ((w & 0x7fff7fffu) + (kStep * 0x10001u)) & 0x80008000u;
}

// The cleaning warp: V tiles from the first one with a node (or the context's end) on.  Rows between the context's end and its block's
// become zeros (what lies there may be anything); infinities and NaN of nodes too, with notes.
// Slots of dirty_full, clean_full, special and the notes are used in turn by cleaned tiles.  Slot c % kCleanRing is free when V of cleaned
// tile c arrives: its buffer, and those of all fills kBuffers or more before it, were released, so the softmax of tiles
// c - kCleanRing and older is done (V's fills are two apart, or one at a piece's end).
template <typename T, int D, int BS>
__device__ __forceinline__ void clean_tiles(const TreeAttendArgs& a, Smem<D>& sm, Notes<D>& notes) {
    constexpr int N = Tile<D>::kBuffers, kCleanRing = Tile<D>::kCleanRing, UNITS = D / 8, RPP = 32 / UNITS;  // rows per pass
    static_assert(2 * kCleanRing - 1 >= N, "see above");
    const int lane = threadIdx.x & 31, u = lane % UNITS, sub = lane / UNITS;
    unsigned fills = 0, cleaned = 0;
#pragma unroll 1
    for (unsigned piece = 0;; ++piece) {
        Job it;
        if (!read_job(sm, piece, &it, a.err) || it.begin == it.end) return;
        const int n = it.end - it.begin, base = it.L - it.n;
        for (int tile = max(it.begin, first_cleaned(it)); tile < it.end; ++tile, ++cleaned) {
            const unsigned fill = fills + value_fill(it.paired, n, tile - it.begin), slot = cleaned % kCleanRing;
            unsigned char* v = sm.kv[fill % N];
            if (!ready(&sm.dirty_full[slot], (cleaned / kCleanRing) & 1, a.err, &sm.abort)) return;
            const int p0 = tile * kTile, end = min(kTile, it.L - p0), first = max(0, base - p0);
            const int block_end = min(kTile, (end + BS - 1) / BS * BS);
            for (int r = end + sub; r < block_end; r += RPP) *reinterpret_cast<uint4*>(v + Tile<D>::at(r, u)) = make_uint4(0u, 0u, 0u, 0u);
            uint32_t found = 0;
#pragma unroll 4
            for (int r = first + sub; r < end; r += RPP) {
                const uint4 x = *reinterpret_cast<const uint4*>(v + Tile<D>::at(r, u));
                found |= not_finite<T>(x.x) | not_finite<T>(x.y) | not_finite<T>(x.z) | not_finite<T>(x.w);
            }
            const bool any = __any_sync(0xffffffffu, found != 0);
            if (any) {
                constexpr uint32_t kMantissa = std::is_same<T, __half>::value ? 0x03ffu : 0x007fu;
                for (int r = first + sub; r < end; r += RPP) {
                    uint4* at = reinterpret_cast<uint4*>(v + Tile<D>::at(r, u));
                    uint32_t w[4] = {at->x, at->y, at->z, at->w}, plus = 0, minus = 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t x = w[i / 2] >> (16 * (i & 1));
                        if (!(not_finite<T>(x & 0xffffu))) continue;
                        const bool nan = (x & kMantissa) != 0;
                        if (nan || !(x & 0x8000u)) plus |= 1u << i;
                        if (nan || (x & 0x8000u)) minus |= 1u << i;
                        w[i / 2] &= i & 1 ? 0x0000ffffu : 0xffff0000u;
                    }
                    *at = make_uint4(w[0], w[1], w[2], w[3]);
                    notes.at[slot][0][r][u] = (uint8_t)plus;
                    notes.at[slot][1][r][u] = (uint8_t)minus;
                }
            }
            if (lane == 0) sm.special[slot] = any;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sm.kv_full[fill % N]);
                mbar_arrive(&sm.clean_full[slot]);
            }
        }
        fills += 2 * n;
    }
}

// One warp per stream issues its products.  Both streams read every K and V tile, in the order in which they come; a buffer is free when
// both have committed what reads it, a query tile too (a pair's tile, read by one stream, is committed twice).
template <typename T, int D>
__device__ __forceinline__ void issue_products(const TreeAttendArgs& a, Smem<D>& sm, int t) {
    constexpr int N = Tile<D>::kBuffers;
    constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
    volatile int* abort = &sm.abort;
    const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0), s_at = tmem + t * 128, o_at = tmem + output_at<D>(t);
    const uint64_t q0 = desc_of(smem_addr(sm.q[0]), 16, 1024), k0 = desc_of(smem_addr(sm.kv[0]), 16, Tile<D>::kGroup),
                   v0 = desc_of(smem_addr(sm.kv[0]), 1024, Tile<D>::kGroup);
    constexpr uint32_t kHalf = Tile<D>::kOperand / 2 >> 4;
    const uint32_t negate = a.scale < 0.f ? 1u << 13 : 0u;  // the query rows are negated instead of the scale
    unsigned buf = 0, phase = 0, query = 0;  // the next fill's buffer and the parity of its phase; the piece's first query tile
    unsigned p_phase = 0;                    // parities of the next phases of p_full: bit b of buffer b's
    // waits for the next fill; its buffer, or -1
    auto take = [&] {
        if (!ready(&sm.kv_full[buf], phase, a.err, abort)) return -1;
        tc_fence_after();
        const int got = (int)buf;
        if (++buf == N) buf = 0, phase ^= 1;
        return got;
    };
    // scores of 64 rows of K, into buffer b
    const uint32_t desc = idesc_of(kTile / 2, false, kBf16) | negate;
    auto scores = [&](int b, uint64_t qd, uint64_t kd) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
            mma_ss(s_at + 64 * b, qd + (((k / 4) * kPanel + (k % 4) * 32) >> 4), kd + (((k / 4) * 1024 + (k % 4) * 32) >> 4), desc, k > 0);
        tc_commit(&sm.s_full[t][b]);
    };
    // output of P buffer b times 64 rows of V
    auto output = [&](int b, uint64_t vd, bool add) {
        if (!ready(&sm.p_full[t][b], p_phase >> b & 1, a.err, abort)) return false;
        p_phase ^= 1u << b;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < kTile / 32; ++k)
            mma_ts(o_at, s_at + 64 * b + 8 * k, vd + (k * 2 * Tile<D>::kGroup >> 4), idesc_of(D, true, kBf16), add || k > 0);
        tc_commit(&sm.pv_done[t][b]);
        return true;
    };
#pragma unroll 1
    for (unsigned piece = 0;; ++piece) {
        Job job;
        if (!read_job(sm, piece, &job, a.err) || job.begin == job.end) return;
        const int n = job.end - job.begin;
        const unsigned mine = query + (job.paired ? t : 0), qbuf = mine & 1;
        query += job.paired ? 2 : 1;
        // (a stream that skips a pair's other tile: the phase before the one that it waits for is over, staged before one that it has seen)
        if (!ready(&sm.q_full[qbuf], mine >> 1 & 1, a.err, abort)) return;
        const uint64_t qd = q0 + (qbuf * Tile<D>::kOperand >> 4);
        // (both buffers are free: their weights were waited for, and the outputs that read them issued)
        // Step u of a pair is half u % 2 of tile u / 2; of a split piece this stream's half of tile u.  Its scores are issued two steps ahead.
        const int steps = job.paired ? 2 * n : n;
        int k_at = 0, v_at = 0;
#pragma unroll 1
        for (int u = -2; u < steps; ++u) {
            const int b = u & 1;
            const bool second = job.paired && b == 1;  // the tile is there already, and done with behind this half
            const uint32_t half = (job.paired ? b : t) * kHalf;
            if (u >= 0) {
                if (!second && (v_at = take()) < 0) return;
                if (!output(b, v0 + (v_at * Tile<D>::kOperand >> 4) + half, u > 0)) return;
                if (!job.paired || second) tc_commit(&sm.kv_empty[v_at]);
            }
            if (u + 2 < steps) {
                if (!second && (k_at = take()) < 0) return;
                scores(b, qd, k0 + (k_at * Tile<D>::kOperand >> 4) + half);
                if (!job.paired || second) tc_commit(&sm.kv_empty[k_at]);
            }
        }
        if (job.paired) tc_commit(&sm.q_free[qbuf]);
        tc_commit(&sm.q_free[qbuf]);
        tc_commit(&sm.o_full[t]);
    }
}

// The query warp: row tile after row tile, up to one piece ahead.  D / 8 lanes copy a row together; rows of a live softmax warp that do not
// exist become zeros.
template <typename T, int D>
__device__ __forceinline__ void stage_queries(const TreeAttendArgs& a, Smem<D>& sm) {
    constexpr int LPR = D / 8, RPS = 32 / LPR;
    const int lane = threadIdx.x & 31, sub = lane / LPR, i = lane % LPR, group = a.group;
    const T* query = static_cast<const T*>(a.query);
    unsigned tile = 0;
#pragma unroll 1
    for (unsigned piece = 0;; ++piece) {
        Job job;
        if (!read_job(sm, piece, &job, a.err) || job.begin == job.end) return;
#pragma unroll 1
        for (int k = 0; k < (job.paired ? 2 : 1); ++k, ++tile) {
            const int buf = tile & 1, first = job.row0 + k * kTile, rows = min(kTile, job.n * group - first);
            if (!ready(&sm.q_free[buf], ((tile >> 1) & 1) ^ 1, a.err, &sm.abort)) return;
#pragma unroll 1
            for (int b = 0; b < rows; b += 32) {
                const int v = first + b + lane, node = v / group;  // this lane's row; its address goes to the lanes that copy it
                const bool live = b + lane < rows;
                const long long row_at =
                    live ? ((long long)(job.first_token + node) * a.num_heads + job.kvh * group + (v - node * group)) * D : 0;
                const unsigned alive = __ballot_sync(0xffffffffu, live);
#pragma unroll
                for (int r = 0; r < 32; r += RPS) {
                    const int row = b + r + sub;
                    const T* src = query + __shfl_sync(0xffffffffu, row_at, r + sub) + 8 * i;
                    cp_async_16_or_zero(sm.q[buf] + row * 128 + (i / 8) * kPanel + (((i & 7) ^ (row & 7)) << 4), src, alive >> (r + sub) & 1);
                }
            }
            cp_async_commit();
            cp_async_wait_all();
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.q_full[buf]);
        }
    }
}

// Which of the 64 positions from `at` on a row sees: those before the nodes (base), and its nodes; less the blocks in masked.
// word0: the row's first word, read ahead.
template <int BS>
__device__ __forceinline__ uint64_t seen_from(const uint64_t* words, uint64_t word0, int num_words, int at, int base, int n, unsigned masked) {
    auto word = [&](int w) {
        const int left = n - 64 * w;
        return w >= num_words || left <= 0 ? 0ull : (w == 0 ? word0 : words[w]) & (left >= 64 ? ~0ull : (1ull << left) - 1);
    };
    const int node = at - base;
    uint64_t seen;
    if (node <= -64) {
        seen = ~0ull;
    } else if (node < 0) {
        seen = (word(0) << -node) | ((1ull << -node) - 1);
    } else {
        seen = word(node >> 6) >> (node & 63);
        if (node & 63) seen |= word((node >> 6) + 1) << (64 - (node & 63));
    }
    constexpr uint64_t kBlock = BS == 16 ? 0xffffull : 0xffffffffull;
#pragma unroll
    for (int k = 0; k < 64 / BS; ++k)
        if (masked >> k & 1) seen &= ~(kBlock << (k * BS));
    return seen;
}

__device__ __forceinline__ float max3(float x, float y, float z) {
    float m;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(x), "f"(y), "f"(z));
    return m;
}
template <typename T>
__device__ __forceinline__ uint32_t round2(float2 x);
template <>
__device__ __forceinline__ uint32_t round2<__half>(float2 x) {
    const __half2 h = __floats2half2_rn(x.x, x.y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t round2<__nv_bfloat16>(float2 x) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// sum += the halves of w, in float32.  (Additions that take 16-bit operands: wide trees 134.3 us; widened first 137.6; the unrounded weights 133.4.)
template <typename T>
__device__ __forceinline__ void add_halves(uint32_t w, float2& sum) {
    if constexpr (std::is_same<T, __half>::value)
        asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tadd.rn.f32.f16 %0, x, %0;\n\tadd.rn.f32.f16 %1, y, %1;\n\t}" : "+f"(sum.x), "+f"(sum.y) : "r"(w));
    else
        asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tadd.rn.f32.bf16 %0, x, %0;\n\tadd.rn.f32.bf16 %1, y, %1;\n\t}" : "+f"(sum.x), "+f"(sum.y) : "r"(w));
}

// Eight 16-byte units of a row per lane become, in groups of eight lanes, one unit of each of the group's rows: x[r] is unit lane % 8 of
// row r.  Stores of x[r] then write whole 128-byte lines (a row to a lane, each store of a warp touched 32 of them, and the results of
// a piece took 4000 cycles).
__device__ __forceinline__ void transpose8(uint4 (&x)[8]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int step = 4; step > 0; step >>= 1) {
        const bool up = lane & step;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j & step) continue;
            const uint4 give = up ? x[j] : x[j + step];
            const uint4 got = make_uint4(__shfl_xor_sync(0xffffffffu, give.x, step), __shfl_xor_sync(0xffffffffu, give.y, step),
                                         __shfl_xor_sync(0xffffffffu, give.z, step), __shfl_xor_sync(0xffffffffu, give.w, step));
            if (up) x[j] = got;
            else x[j + step] = got;
        }
    }
}

// A softmax warp: 32 rows of a stream's row tile, one per lane.
template <typename T, int D, int BS>
__device__ __forceinline__ void softmax_rows(const TreeAttendArgs& a, float* records, Smem<D>& sm, Notes<D>& notes) {
    constexpr int RING = Tile<D>::kRing, kCleanRing = Tile<D>::kCleanRing;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, t = warp >> 2, r = (warp & 3) * 32 + lane, group = a.group;
    volatile int* abort = &sm.abort;
    const uint32_t lanes = sm.tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t s_at = lanes + t * 128, o_at = lanes + output_at<D>(t), other_o_at = lanes + output_at<D>(t ^ 1);
    // (kept above zero, so that masked scores stay -inf)
    const float factor = fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1e-38f);
    unsigned pieces = 0, joins = 0, tiles_before = 0, cleaned = 0;  // so far
    unsigned s_phase = 0, pv_phase = 3;  // parities of the next phases of s_full, of the last ones of pv_done: bit b of buffer b's
#pragma unroll 1
    for (unsigned piece = 0;; ++piece) {
        Job job;
        if (!read_job(sm, piece, &job, a.err) || job.begin == job.end) return;
        const bool paired = job.paired;
        const int n = job.end - job.begin, base = job.L - job.n;
        const int first = job.row0 + (paired ? t * kTile : 0), v = first + r, node = v / group;  // row of the request
        const bool live = v < job.n * group, warp_live = first + (warp & 3) * 32 < job.n * group;
        const uint64_t* words = reinterpret_cast<const uint64_t*>(a.tree_mask) + (live ? (size_t)(job.first_token + node) * a.mask_words : 0);
        const uint64_t word0 = words[0];
        float m = -INFINITY, l = 0.f;  // the row's reference of exponents, the sum of its exponentials
        bool noted = false;
        uint64_t seen0 = 0, seen1 = 0;  // of the tile's halves, where V is cleaned (of a split piece this stream's)
        const int steps = paired ? 2 * n : n;
#pragma unroll 1
        for (int step = 0; step < steps; ++step) {
            const int half = paired ? step & 1 : t, local = paired ? step >> 1 : step, b = step & 1;
            const int p0 = (job.begin + local) * kTile;
            if (!ready(&sm.s_full[t][b], s_phase >> b & 1, a.err, abort)) return;
            s_phase ^= 1u << b;
            tc_fence_after();
            const unsigned masked = sm.masked[(tiles_before + local) % RING];
            const bool clean = (masked >> 31) && (!paired || half == 1);  // V of this tile is cleaned
            if (!warp_live) {  // rows that nobody reads: whatever lies there may be multiplied
                if (clean) {
                    if (!ready(&sm.clean_full[cleaned % kCleanRing], (cleaned / kCleanRing) & 1, a.err, abort)) return;
                    ++cleaned;
                }
                if (lane == 0) mbar_arrive(&sm.p_full[t][b]);
                pv_phase ^= 1u << b;
                continue;
            }
            // The half's weights, from its scores, in two passes of two chunks of 32 columns; the second reads the scores again.  (Softmax warps run
            // through this code once a step, and fetching it is what bounds them: all 64 scores in registers, one pass, 145 us
            // for wide trees; two steps unrolled 183.)  A body for either case of edge.
            auto weigh = [&](auto edge) {
                constexpr bool kEdge = decltype(edge)::value;
                const uint32_t at = s_at + 64 * b;
                uint64_t mine = ~0ull;
                if constexpr (kEdge) {
                    mine = live ? seen_from<BS>(words, word0, a.mask_words, p0 + 64 * half, base, job.n, (masked & 0xffu) >> (half * (64 / BS))) : 0ull;
                    if (half == 0) seen0 = mine;
                    else seen1 = mine;
                }
                auto chunk = [&](int c, uint32_t (&s)[32]) {
                    tmem_ld32(at + 32 * c, s);
                    tc_wait_ld(s);
                    if constexpr (kEdge) {
                        const uint32_t w = (uint32_t)(mine >> (32 * c));
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(w >> i & 1)) s[i] = 0xff800000u;
                    }
                };
                float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // four chains
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t s[32];
                    chunk(c, s);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) x[i / 2 % 4] = max3(x[i / 2 % 4], __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
                }
                const float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) * factor;
                if (step == 0) {
                    m = top;
                } else if (__any_sync(0xffffffffu, top > m + 8.f)) {
                    // The output so far has to be there.  (The phase before the one that is meant is over: these scores were issued behind the
                    // output before the last, and a commit waits for all products before it.  So P's place is free too.)
                    if (!ready(&sm.pv_done[t][b ^ 1], pv_phase >> (b ^ 1) & 1, a.err, abort)) return false;
                    tc_fence_after();
                    const float mn = fmaxf(m, top);
                    const float f = mn == -INFINITY ? 1.f : exp2_approx(m - mn);
                    l *= f;
                    m = mn;
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t o[16];
                        tmem_ld16(o_at + c, o);
                        tc_wait_ld(o);
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                        tmem_st16(o_at + c, o);
                    }
                }
                // P: exp2(score * factor - mu), rounded, over the scores of the first chunk, which are in registers by then
                const float mu = m == -INFINITY ? 0.f : m;
                float2 sum = make_float2(0.f, 0.f);
                const float2 f2 = make_float2(factor, factor), m2 = make_float2(-mu, -mu);
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    uint32_t s[32];
                    chunk(c, s);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float2 y = fma2(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), f2, m2);
                        const float2 e = make_float2(exp2_approx(y.x), exp2_approx(y.y));
                        s[i / 2] = round2<T>(e);
                        add_halves<T>(s[i / 2], sum);
                    }
                    tmem_st16(at + 16 * c, *reinterpret_cast<uint32_t(*)[16]>(&s[0]));
                }
                l += sum.x + sum.y;
                return true;
            };
            // edge: a block that is not there, or (bit 31) a tile with nodes or the context's end
            if (!masked) {
                if (!weigh(std::false_type{})) return;
            } else if (!weigh(std::true_type{})) {
                return;
            }
            pv_phase ^= 1u << b;
            if (clean) {
                const unsigned note = cleaned % kCleanRing;
                if (!ready(&sm.clean_full[note], (cleaned / kCleanRing) & 1, a.err, abort)) return;
                ++cleaned;
                if (sm.special[note]) {
                    const int from = max(0, base - p0);
#pragma unroll 1
                    for (int sign = 0; sign < 2; ++sign) {
#pragma unroll 1
                        for (int i = 0; i < D / 32; ++i) {
                            uint32_t bits = noted ? notes.row[t][sign][r][i] : 0u;
#pragma unroll 1
                            for (int k = from; k < kTile; ++k)
                                if ((k < 64 ? seen0 : seen1) >> (k & 63) & 1)
                                    bits |= *reinterpret_cast<const uint32_t*>(&notes.at[note][sign][k][4 * i]);
                            notes.row[t][sign][r][i] = bits;
                        }
                    }
                    noted = true;
                }
            }
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.p_full[t][b]);
        }
        tiles_before += n;

        // the piece's result
        const bool cut = job.begin > 0 || job.end < job.tiles, join = !paired;
        if (!ready(&sm.o_full[t], pieces & 1, a.err, abort)) return;
        tc_fence_after();
        ++pieces;
        float f0 = 1.f, f1 = 0.f;  // factors of this stream's output and of the other's
        uint32_t notes_from = noted ? 1u << t : 0u;
        if (join) {  // both streams have a part of the same rows, in the same lanes of tensor memory
            sm.state[t][r] = make_float2(m, __uint_as_float((__float_as_uint(l) & 0x7fffffffu) | (noted ? 0x80000000u : 0u)));
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.join_full);
            if (!ready(&sm.join_full, joins & 1, a.err, abort)) return;
            tc_fence_after();
            const float2 o = sm.state[t ^ 1][r];
            const float ol = __uint_as_float(__float_as_uint(o.y) & 0x7fffffffu);
            const float mn = fmaxf(m, o.x);
            // a state without a maximum is empty, unless its sum is NaN
            f0 = m == -INFINITY ? (l != l ? 1.f : 0.f) : exp2_approx(m - mn);
            f1 = o.x == -INFINITY ? (ol != ol ? 1.f : 0.f) : exp2_approx(o.x - mn);
            l = l * f0 + ol * f1;
            m = mn;
            if (__float_as_uint(o.y) >> 31) notes_from |= 2u >> t;
        }
        if (warp_live) {
            float* rec = records + ((size_t)blockIdx.x * 4 + (job.begin > 0 ? 0 : 2) + (paired ? t : 0)) * record_floats(D);
            const long long row_at = live ? ((long long)(job.first_token + node) * a.num_heads + job.kvh * group + (v - node * group)) * D : 0;
            if (!cut) f0 *= l == 0.f ? 0.f : 1.f / l, f1 *= l == 0.f ? 0.f : 1.f / l;
            if (l != l) notes_from = 0;  // (NaN everywhere)
            const unsigned alive = __ballot_sync(0xffffffffu, live);
            const int c0 = join ? t * (D / 2) : 0, c1 = join ? c0 + D / 2 : D;
            // 32 columns from c on, in float32
            auto columns = [&](int c, uint32_t (&s)[32]) {
                tmem_ld32(o_at + c, s);
                if (join) {
                    uint32_t o[32];
                    tmem_ld32(other_o_at + c, o);
                    tc_wait_ld(s);
                    tc_wait_ld(o);
#pragma unroll
                    for (int k = 0; k < 32; ++k) s[k] = __float_as_uint(fmaf(__uint_as_float(o[k]), f1, __uint_as_float(s[k]) * f0));
                } else {
                    tc_wait_ld(s);
#pragma unroll
                    for (int k = 0; k < 32; ++k) s[k] = __float_as_uint(__uint_as_float(s[k]) * f0);
                }
                if (notes_from) {
                    uint32_t plus = 0, minus = 0;
#pragma unroll
                    for (int k = 0; k < 2; ++k)
                        if (notes_from >> k & 1) {
                            plus |= notes.row[k][0][r][c / 32];
                            minus |= notes.row[k][1][r][c / 32];
                        }
#pragma unroll
                    for (int k = 0; k < 32; ++k)
                        if ((plus | minus) >> k & 1) s[k] = !(minus >> k & 1) ? 0x7f800000u : !(plus >> k & 1) ? 0xff800000u : 0x7fc00000u;
                }
            };
            if (cut) {
#pragma unroll 1
                for (int c = c0; c < c1; c += 32) {
                    uint32_t s[32];
                    columns(c, s);
                    uint4 x[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[k] = make_uint4(s[4 * k], s[4 * k + 1], s[4 * k + 2], s[4 * k + 3]);
                    transpose8(x);
                    float* to = rec + 2 * kTile + (size_t)((warp & 3) * 32 + (lane & 24)) * D + c + 4 * (lane & 7);
#pragma unroll
                    for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4*>(to + k * D) = x[k];
                }
                if (c0 == 0) {
                    rec[r] = m;
                    rec[kTile + r] = l;
                }
            } else {
#pragma unroll 1
                for (int c = c0; c < c1; c += 64) {
                    uint4 x[8];
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        if (join && D == 64 && part == 1) {  // (a stream has 32 columns)
                            x[4] = x[5] = x[6] = x[7] = make_uint4(0u, 0u, 0u, 0u);
                            break;
                        }
                        uint32_t s[32];
                        columns(c + 32 * part, s);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t y[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                y[i] = round2<T>(make_float2(__uint_as_float(s[8 * k + 2 * i]), __uint_as_float(s[8 * k + 2 * i + 1])));
                            x[4 * part + k] = make_uint4(y[0], y[1], y[2], y[3]);
                        }
                    }
                    const bool mine = !(join && D == 64) || (lane & 7) < 4;
                    transpose8(x);
                    T* out = static_cast<T*>(a.out) + c + 8 * (lane & 7);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int row = (lane & 24) + k;
                        const long long at = __shfl_sync(0xffffffffu, row_at, row);
                        if (mine && (alive >> row & 1)) *reinterpret_cast<uint4*>(out + at) = x[k];
                    }
                }
            }
        }
        tc_fence_before();
        if (join) {  // neither stream's output is written again before both have read it
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.join_done);
            if (!ready(&sm.join_done, joins & 1, a.err, abort)) return;
            ++joins;
        }
    }
}

template <typename T, int D, int BS>
__global__ void __launch_bounds__(kThreads, 1) attend_tree_kernel(const TreeAttendArgs a, Seam* seams, float* records, Notes<D>* all_notes,
                                                                  const __grid_constant__ CUtensorMap kmap,
                                                                  const __grid_constant__ CUtensorMap vmap) {
    extern __shared__ __align__(1024) unsigned char raw_smem[];
    Smem<D>& sm = *reinterpret_cast<Smem<D>*>(raw_smem);
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 32) {
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
    }
    if (warp == 0) {  // a lane per place
        const int i = threadIdx.x;
        if (i < 2) {
            mbar_init(&sm.q_full[i], 1);
            mbar_init(&sm.q_free[i], 2);
            mbar_init(&sm.o_full[i], 1);
            mbar_init(&sm.drain[i], 1);
            mbar_init(i ? &sm.join_full : &sm.join_done, kSoftmaxWarps);
        }
        if (i < 4) {
            mbar_init(&sm.s_full[i >> 1][i & 1], 1);
            mbar_init(&sm.p_full[i >> 1][i & 1], 4);
            mbar_init(&sm.pv_done[i >> 1][i & 1], 1);
        }
        if (i < kPieces) {
            mbar_init(&sm.job_full[i], 1);
            mbar_init(&sm.job_free[i], kReaders);
        }
        if (i < Tile<D>::kRing) {
            mbar_init(&sm.side_full[i], 1);
            mbar_init(&sm.copied[i], 1);
        }
        if (i < Tile<D>::kBuffers) {
            mbar_init(&sm.kv_full[i], 1);
            mbar_init(&sm.kv_empty[i], 2);
        }
        if (i < Tile<D>::kCleanRing) {
            mbar_init(&sm.dirty_full[i], 1);
            mbar_init(&sm.clean_full[i], 1);
        }
        sm.abort = 0;
        fence_barrier_init();
    }
    if (warp == kIssueWarp) tmem_alloc(&sm.tmem, 512);
    griddep_wait();
    griddep_launch_dependents();
    static_assert(sizeof(Scratch) <= sizeof(sm.state), "the sums lie where the states will");
    tc_fence_before();
    const Start start = find_share(a, *reinterpret_cast<Scratch*>(&sm.state));  // (synchronises the CTA)
    tc_fence_after();
    Notes<D>& notes = all_notes[blockIdx.x];
    if (warp < kSoftmaxWarps) {
        softmax_rows<T, D, BS>(a, records, sm, notes);
    } else if (warp == kCopyWarp) {
        copy_tiles<D, BS>(a, sm, &kmap, &vmap);
    } else if (warp == kLookWarp) {
        look_ahead<D, BS>(a, seams, sm, start);
    } else if (warp == kCleanWarp) {
        clean_tiles<T, D, BS>(a, sm, notes);
    } else if (warp == kQueryWarp) {
        stage_queries<T, D>(a, sm);
    } else {
        const int t = __shfl_sync(0xffffffffu, warp - kIssueWarp, 0);
        issue_products<T, D>(a, sm, t);
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

// Joins the partial results of the units that share boundaries cut: CTA (boundary, rows), a warp per row, D / 32 elements per lane.  The
// parts' maxima and sums are read by a lane each.
constexpr int kJoinRows = kJoinThreads / 32, kJoinSplit = 32;
template <typename T, int D>
__global__ void __launch_bounds__(kJoinThreads) join_tree_kernel(const TreeAttendArgs a, const Seam* seams, const float* records) {
    griddep_wait();
    griddep_launch_dependents();
    constexpr int E = D / 32;
    using Vec = typename std::conditional<E == 4, float4, float2>::type;
    const Seam s = seams[blockIdx.x + 1];
    if (s.last == 0) return;
    const int lane = threadIdx.x & 31, group = a.group, first_token = a.q_offsets[s.seq];
    auto cut = [&](int c) { return tiles_in(s.share * c - s.unit, s.tiles, s.paired); };  // CTA c has tiles [cut(c), cut(c + 1))
    bool parts = false;  // (a boundary inside the cost may still fall before the first tile or behind the last)
    for (int c = s.first + 1; c <= s.last; ++c) parts |= cut(c) > 0 && cut(c) < s.tiles;
    if (!parts) return;
    // Lane i has part i of 32: whether it is there, and where its record is (nearly always there is no second round of 32).
    int at = 0;
    auto look = [&](int c0) {
        const int c = c0 + lane, from = cut(c);
        at = (int)((c * 4 + (from > 0 ? 0 : 2)) * record_floats(D));
        return __ballot_sync(0xffffffffu, c <= s.last && from < cut(c + 1));
    };
    unsigned there = look(s.first);
    for (int r = blockIdx.y * kJoinRows + (threadIdx.x >> 5); r < s.rows; r += gridDim.y * kJoinRows) {
        const int rr = r % kTile;
        const float* of_tile = records + (r / kTile) * record_floats(D);
        const float* of_row = of_tile + 2 * kTile + (size_t)rr * D + lane * E;
        float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = 0.f;
        for (int c0 = s.first; c0 <= s.last; c0 += 32) {
            if (s.last - s.first >= 32) there = look(c0);
            unsigned left = there;
            constexpr int kAtOnce = 2;
            alignas(16) float x[kAtOnce][E];
            int part[kAtOnce];  // whose; -1: none
            auto fetch = [&] {
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    part[k] = __ffs(left) - 1;
                    const int of = __shfl_sync(0xffffffffu, at, max(0, part[k]));
                    if (part[k] >= 0) *reinterpret_cast<Vec*>(x[k]) = *reinterpret_cast<const Vec*>(of_row + of);
                    left &= left - 1;
                }
            };
            const bool has = there >> lane & 1;
            const float mc = has ? of_tile[at + rr] : -INFINITY, lc = has ? of_tile[at + kTile + rr] : 0.f;
            fetch();  // (on their way while the weights are made)
            float mn = mc;
#pragma unroll
            for (int w = 16; w > 0; w >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, w));
            mn = fmaxf(mn, m);
            // a part without a maximum is empty, unless its sum is NaN
            const float weight = lc != lc ? 1.f : mc == -INFINITY ? 0.f : exp2_approx(mc - mn), f = l != l ? 1.f : m == -INFINITY ? 0.f : exp2_approx(m - mn);
            float sum = lc * weight;
#pragma unroll
            for (int w = 16; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            l = l * f + sum;
            m = mn;
#pragma unroll
            for (int i = 0; i < E; ++i) o[i] *= f;
            for (;;) {
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    const float wk = __shfl_sync(0xffffffffu, weight, max(0, part[k]));
                    if (part[k] >= 0)
#pragma unroll
                        for (int i = 0; i < E; ++i) o[i] = fmaf(x[k][i], wk, o[i]);
                }
                if (!left) break;
                fetch();
            }
        }
        const int v = s.row0 + r, node = v / group;
        T* dst = static_cast<T*>(a.out) + ((size_t)(first_token + node) * a.num_heads + s.kvh * group + (v - node * group)) * D + lane * E;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint32_t y[E / 2];
#pragma unroll
        for (int i = 0; i < E / 2; ++i) y[i] = round2<T>(make_float2(o[2 * i] * inv, o[2 * i + 1] * inv));
        if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(y[0], y[1]);
        else *reinterpret_cast<uint32_t*>(dst) = y[0];
    }
}

// Places in the workspace of a call: seams, then records [CTAs][2 slots][2 tiles][m 128 | l 128 | o 128 x D], then notes.
template <int D>
size_t lay_out(int num_sms, char* base, Seam** seams, float** records, Notes<D>** notes) {
    const size_t first = align256((size_t)num_sms * sizeof(Seam)), second = first + (size_t)num_sms * 4 * record_floats(D) * sizeof(float);
    if (base) {
        *seams = reinterpret_cast<Seam*>(base);
        *records = reinterpret_cast<float*>(base + first);
        *notes = reinterpret_cast<Notes<D>*>(base + second);
    }
    return second + (size_t)num_sms * sizeof(Notes<D>);
}

template <typename T, int D, int BS>
cudaError_t attend_typed(const TreeAttendArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t stream) {
    const int ctas = a.num_sms;
    Seam* seams;
    float* records;
    Notes<D>* notes;
    lay_out<D>(ctas, static_cast<char*>(a.workspace), &seams, &records, &notes);
    const size_t smem = sizeof(Smem<D>);
    cudaError_t e = cudaFuncSetAttribute(attend_tree_kernel<T, D, BS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(attend_tree_kernel<T, D, BS>, dim3((unsigned)ctas), dim3(kThreads), smem, stream, a, seams, records, notes, kmap, vmap);
    if (e != cudaSuccess || ctas < 2) return e;
    return launch_pdl(join_tree_kernel<T, D>, dim3((unsigned)(ctas - 1), kJoinSplit), dim3(kJoinThreads), 0, stream, a, seams, records);
}

}  // namespace

size_t attend_tree_workspace_bytes(int num_sms, int head_dim) {
    return head_dim == 64 ? lay_out<64>(num_sms, nullptr, nullptr, nullptr, nullptr) : lay_out<128>(num_sms, nullptr, nullptr, nullptr, nullptr);
}

cudaError_t attend_tree_launch(const TreeAttendArgs& a, const CUtensorMap& kmap, const CUtensorMap& vmap, cudaStream_t stream) {
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
