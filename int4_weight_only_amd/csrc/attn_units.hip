// attn_units.hip -- attention of sequences that share prefixes (w4_attn_shared), and cross attention
// (w4_attn_cross).
//
// The softmax of a row over prefix and own keys is the join of two partial ones, and the rows of all
// sequences over one prefix can be stacked: its keys are then read and multiplied once for many rows,
// not once per sequence. Work is cut into units of stacked rows of one key-value head:
//   prefix units: rows of all sequences over prefix g, its keys
//   own units:    rows of one sequence, its own keys; of a sequence that fills a wide unit by itself (or
//                 has no prefix) all of its keys, by both tables. (Such sequences share nothing, and the
//                 rows past their last full unit take one for themselves: 64 of 18 tokens after 8000
//                 shared keys, 28 heads over 4 of 128, 177 us, of 19 tokens, 133 rows, 238.)
// The unit of a prefix or sequence with up to 16 rows is narrow, a wave's work (attn_narrow.h: bound by
// reading keys), others are wide, 128 rows each, a workgroup's (attn_tile.h: bound by the products).
//
// The workgroups that the card holds at once are divided between wide and narrow work by what it
// costs. The key tiles of all wide (narrow) units, one unit after the other, form a line, and the
// workgroups (their waves) take equal pieces of it, whatever the lengths are; each goes through the
// units in its piece one after the other. Where there are workers enough, every unit has pieces of its
// own instead, so that none begins two. A unit that lies in several pieces leaves weighted sums,
// maximum and sum of weights in the workspace, as do rows with two units, and a second kernel joins
// them in order. Lengths live on the device, so that every workgroup sums up the line for itself.
//
// 28 heads over 4 of 128, in a graph: 256 sequences over 32768 shared keys 155 to 163 us (121 GFLOP, 740
// to 780 TFLOP/s; matrix cores 36 %, vector units 39 % busy), 100 over five prefixes of up to 8000, with
// 1500 keys of their own, 73 us (256 MB, 3.5 TB/s), 64 over 2048 28 us, 4 over 1000 16 us. Of the last,
// 2.7 us go by until the line is summed up, 1.5 until a worker has its rows, 6 for the keys' way and two
// tiles, one for the sums, 4 for the join: waits one after the other. Wide units take 5 us from their
// rows to the first weights and 2 for their sums. A launch for each line instead of one for both: 64
// sequences 44 us for 29, five prefixes 94 for 73, 256 sequences 181 for 158.
#include <algorithm>

#include "attn_narrow.h"
#include "attn_tile.h"

namespace w4 {

namespace {

// Rows of a prefix or sequence whose units are narrow, at most. (Up to 64, so that keys are read once per
// 16 rows: 32 sequences of 4 tokens, 28 heads over 4 of 128, 4096 shared keys and up to 1000 of their
// own 47 us for 37. At 256 dims the narrow body's registers do not fit beside the wide one's.)
template <int DP>
constexpr int kNarrowMost = DP > 128 ? 0 : kNarrowRows;
constexpr int kThreads = kTileWaves * kWave;
static_assert(kTileWaves == kNarrowWaves, "one workgroup for both");
// Entries of the line: each prefix, and each bucket of sequences (of one up to kBuckets sequences).
constexpr int kMostPrefixes = 256, kBuckets = 256, kEntries = kMostPrefixes + kBuckets;
// Costs, on either line: of a tile, and of what a unit takes besides (rows, queries, the first keys'
// way, sums), in halves of a tile. (Wide start 6: 4 sequences over 1000 keys 19 us for 17; 16 gives
// nothing. Narrow start 6: 17.4 for 16.9.)
constexpr int kTileCost = 2, kWideStart = 10, kNarrowStart = 3;
// A narrow tile's cost in wide ones, where the card is full of them: a wave's 32 keys from memory, over
// the products of 128 rows and the keys of a tile. (A quarter: four waves. Half of it: 256 sequences over
// 32768 keys 182 us for 154; twice: five prefixes of up to 8000 85 us for 73.)
template <int DP>
constexpr float kNarrowWeight = DP > 64 ? 0.4f : 0.25f;
// The shortest pieces, without a unit's start: workers that share less than this are better fewer. (A
// piece that may have one inside is longer by it, so that none is without tiles. Wide: 8 tiles 24 us for
// 17 with 4 sequences over 1000 keys, 2 tiles 35 for 31 with 16 over 16384. Narrow: one tile 31 us for 24,
// 4 tiles 22, with 8 sequences of 8 heads over 4096; but 18.3 for 16.9 with 4 over 1000.)
constexpr int kWideLeast = 4 * kTileCost, kNarrowLeast = 2 * kTileCost;

struct UnitArgs {
    AttnArgs a;
    KvView c;
    Prefixes x;  // x.n = 0: none
    bool every;  // each row sees all keys of its sequence
    int grid;             // workgroups
    int bucket, buckets;  // sequences of a bucket, and how many buckets
    int heads;            // of a key-value head
};

// a / b of numbers below 2^30 where the quotient is below 2^21 (within 5/8 before it is cut).
__device__ __forceinline__ int divide(int a, int b) {
    const float q = static_cast<float>(a) * __builtin_amdgcn_rcpf(static_cast<float>(b));
    int r = static_cast<int>(q);
    r -= r * b > a ? 1 : 0;
    return r + (a - r * b >= b ? 1 : 0);
}

// A sequence in this call: its rows, its keys, and the prefix that holds the first of them (-1: none).
struct Sequence {
    int q0, n_keys, packed;  // packed: tokens, and the prefix + 1
    __device__ __forceinline__ int tokens() const { return packed >> 9; }
    __device__ __forceinline__ int prefix() const { return (packed & 511) - 1; }
};
constexpr int kMostTokens = 1 << 21;
// (a worker looks through a bucket of them for each unit)
constexpr int kMostSequences = 1 << 16;
__device__ __forceinline__ Sequence sequence(const UnitArgs &s, int b) {
    const AttnArgs &a = s.a;
    Sequence r;
    int tokens = 1, prefix = -1;
    r.q0 = b;
    if (a.q_start) {
        r.q0 = max(read_const(a.q_start + b), 0);
        tokens = max(min(read_const(a.q_start + b + 1), static_cast<int>(a.T)) - r.q0, 0);
    }
    if (s.x.n > 0) prefix = read_const(s.x.of + b);
    r.n_keys = kv_length(s.c, b);
    r.packed = tokens << 9 | (prefix >= 0 && prefix < s.x.n ? prefix + 1 : 0);
    return r;
}

// Oldest and newest of 64 positions, -kRowsMost .. kNewest.
constexpr int kRowsMost = 1 << 24, kNewest = 1 << 30;
__device__ __forceinline__ int wave_oldest(int v) { return kNewest - wave_max_dpp(kNewest - v); }
__device__ __forceinline__ int wave_newest(int v) {
    return wave_max_dpp(v + kRowsMost) - kRowsMost;
}

// The workspace. Each (token row, head) pair has a record of its partial results, of the own unit's
// and of the prefix unit's pieces: how many there are (kNarrowRecord added where workers are waves), and
// the row of partial sums of the second one. The first piece's is the pair's own; every workgroup has
// kTileRows rows, a quarter for each wave, for the one unit that began before its piece.
struct Record {
    int parts, rest;
};
constexpr int kNarrowRecord = 1 << 20, kWaveRows = kTileRows / kTileWaves;
struct Workspace {
    float *o, *ml;         // [rows][D], [rows][2]
    Record *own, *prefix;  // [pairs]; own[pair].parts < 0: written, nothing to join
    int64_t pairs, rows;
};
__host__ __device__ __forceinline__ int64_t work_rows(int64_t pairs, int grid) {
    return 2 * pairs + static_cast<int64_t>(grid) * kTileRows;
}
__device__ __forceinline__ Workspace workspace(const UnitArgs &s) {
    Workspace w;
    w.pairs = s.a.T * s.a.n_heads;
    w.rows = work_rows(w.pairs, s.grid);
    w.o = static_cast<float *>(s.a.work);
    w.ml = w.o + w.rows * s.c.head_dim;
    w.own = reinterpret_cast<Record *>(w.ml + w.rows * 2);
    w.prefix = w.own + w.pairs;
    return w;
}

// A worker's place on its line. (In LDS: what the loops over keys do not use takes no registers
// there.)
struct Place {
    int x, end;      // what is left of its piece
    int span;        // length of all pieces
    int worker;      // number of its piece
    int slot;        // its first row of partial sums
    int whole;       // units of whole pieces: each begins where a piece does
};

// The line, in LDS. Entries: the prefixes, then the buckets.
struct Line {
    int upto[kEntries];   // lengths up to and with each entry
    int tiles[kEntries];  // key tiles of each of its units (of a bucket of one sequence)
    int cut[kMostPrefixes], tokens[kMostPrefixes];  // of a prefix: keys, tokens of its rows
    Sequence seq[kBuckets];                         // of a bucket of one sequence
    int cost[2][kTileWaves], units[2][kTileWaves];  // sums of a wave's wide and narrow entries
    Place place[kTileWaves];                        // of each wave (those of a wide workgroup: alike)
};

// A piece of a unit.
struct Piece {
    int next;   // where the one after it begins on the line
    int group;  // prefix or sequence
    bool of_prefix, first;
    int hk, row0, rows;  // key-value head, first stacked row, stacked rows of the group
    int tiles, t0, t1;   // key tiles of the unit as planned, those of the piece
    int parts;           // pieces of the unit (where `first`)
};

template <int DP, bool NARROW>
struct Units {
    static constexpr int KT = tile_keys(DP);
    const UnitArgs &s;
    Line &line;

    __device__ __forceinline__ Place place() const {
        const Place &p = line.place[threadIdx.x / kWave];
        return {uniform(p.x),      uniform(p.end),  uniform(p.span),
                uniform(p.worker), uniform(p.slot), uniform(p.whole)};
    }

    __device__ __forceinline__ static bool is_narrow(int rows) { return rows <= kNarrowMost<DP>; }
    __device__ __forceinline__ static int unit_rows(bool narrow) {
        return narrow ? kNarrowRows : kTileRows;
    }
    __device__ __forceinline__ int first_position(const Sequence &q) const {
        return s.every ? q.n_keys - 1 : q.n_keys - q.tokens();
    }
    // Keys that the sequence's prefix holds, and whether its rows go with the prefix' units. (Not those of
    // a sequence without keys: its rows see nothing, and position -1 would have a unit under a window begin
    // at key 0. 64 sequences, 48 of them ended, after 32768 keys, 28 heads over 4 of 128: 42 us with them
    // left out, 76 with them stacked; window 1024 24 and 75.)
    __device__ __forceinline__ int cut_of(const Sequence &q) const {
        return q.prefix() >= 0 ? line.cut[q.prefix()] : 0;
    }
    __device__ __forceinline__ bool shares(const Sequence &q, int cut) const {
        return cut > 0 && q.n_keys > 0 && q.packed >= 512 && q.tokens() * s.heads < kTileRows;
    }
    // Units of `rows` stacked rows, and what each costs.
    __device__ __forceinline__ int units_of(int rows) const {
        const int n = unit_rows(is_narrow(rows));
        return (rows + n - 1) / n * s.c.n_kv;
    }
    __device__ __forceinline__ static int unit_cost(int rows, int tiles) {
        return (is_narrow(rows) ? kNarrowStart : kWideStart) + tiles * kTileCost;
    }
    // Length of each on the line; of all of them.
    __device__ __forceinline__ static int length(const Place &at, int rows, int tiles) {
        const int cost = unit_cost(rows, tiles);
        // (no piece without a tile but the first)
        return at.whole ? min(divide(cost + at.span - 1, at.span), max(tiles, 1)) * at.span : cost;
    }
    __device__ __forceinline__ int lengths(const Place &at, bool narrow, int rows, int tiles) const {
        return is_narrow(rows) == narrow ? units_of(rows) * length(at, rows, tiles) : 0;
    }
    // Key tiles of a unit whose rows stand at first .. last.
    __device__ __forceinline__ int key_tiles(int rows, int first, int last, int cut, bool from_cut,
                                             bool to_cut) const {
        const int shift = is_narrow(rows) ? __builtin_ctz(kNarrowTile) : __builtin_ctz(KT);
        const int window = s.a.window;
        last = to_cut ? min(last, cut - 1) : last;
        const int begin = from_cut ? cut : 0;
        if (last < begin) return 0;
        // (both tables: the tile of the border twice)
        const int twice =
            !from_cut && !to_cut && last >= cut && (cut & ((1 << shift) - 1)) != 0 ? 1 : 0;
        if (window == 0) return (last >> shift) - (begin >> shift) + 1 + twice;
        const int lo = max(max(first - window + 1, 0), begin);
        const int early = min(s.a.sinks, lo);
        const int sink_end = early > begin ? ((early - 1) >> shift) + 1 : begin >> shift;
        return max((last >> shift) + 1 - max(lo >> shift, sink_end), 0) + sink_end -
               (begin >> shift) + twice;
    }
    __device__ __forceinline__ int own_tiles(const Sequence &q) const {
        const int cut = cut_of(q);
        return key_tiles(q.tokens() * s.heads, first_position(q), q.n_keys - 1, cut, shares(q, cut),
                         false);
    }
    __device__ __forceinline__ Sequence sequence_at(int b) const {
        return s.bucket == 1 ? line.seq[b] : sequence(s, b);
    }
    // Sums up the lines, for NARROW of either kind, and finds the workers' places; is this workgroup one
    // of the narrow line's? `oldest`: LDS of kMostPrefixes words.
    __device__ __forceinline__ bool plan(int *oldest) const {
        static_assert(kMostPrefixes <= kThreads && kBuckets <= kThreads, "a thread each");
        static_assert(kEntries == 2 * kThreads, "two each");
        const int tid = threadIdx.x, lane = tid & (kWave - 1), wid = uniform(tid / kWave);
        const int n_prefixes = s.x.n, n_seqs = s.c.n_seqs, bucket = s.bucket;
        const int buckets = s.buckets, entries = n_prefixes + buckets;
        const int b0 = tid * bucket, b1 = min(b0 + bucket, n_seqs);
        Sequence q = {0, 0, 0};
        if (tid < buckets) q = sequence(s, b0);  // (on its way with the prefix')
        if (n_prefixes > 0) {
            if (tid < n_prefixes) {
                line.cut[tid] = prefix_length(s.x, tid);
                line.tokens[tid] = 0;
                oldest[tid] = INT32_MAX;
            }
            __syncthreads();
        }
        // What wide and narrow units cost.
        int cost[2] = {0, 0}, units[2] = {0, 0}, rows = 0, tiles = 0;
        const auto count = [&](int rows, int tiles) {
            const int n = units_of(rows), all = n * unit_cost(rows, tiles);
            const bool narrow = is_narrow(rows);
            cost[0] += narrow ? 0 : all;
            cost[1] += narrow ? all : 0;
            units[0] += narrow ? 0 : n;
            units[1] += narrow ? n : 0;
        };
        if (tid < buckets) {
            line.seq[tid] = q;
#pragma unroll 1
            for (int b = b0;;) {
                rows = q.tokens() * s.heads;
                tiles = own_tiles(q);
                count(rows, tiles);
                if (n_prefixes > 0 && shares(q, cut_of(q))) {
                    atomicAdd(&line.tokens[q.prefix()], q.tokens());
                    if (s.a.window > 0) atomicMin(&oldest[q.prefix()], first_position(q));
                }
                if (++b >= b1) break;
                q = sequence(s, b);
            }
            line.tiles[n_prefixes + tid] = tiles;
        }
        int shared_rows = 0, shared_tiles = 0;
        if (n_prefixes > 0) {
            __syncthreads();
            if (tid < n_prefixes) {
                shared_rows = line.tokens[tid] * s.heads;
                shared_tiles =
                    key_tiles(shared_rows, oldest[tid], INT32_MAX, line.cut[tid], false, true);
                line.tiles[tid] = shared_tiles;
                count(shared_rows, shared_tiles);
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            cost[i] = wave_sum_dpp(cost[i]);
            units[i] = wave_sum_dpp(units[i]);
            if (lane == 0) {
                line.cost[i][wid] = cost[i];
                line.units[i][wid] = units[i];
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            cost[i] = units[i] = 0;
#pragma unroll
            for (int w = 0; w < kTileWaves; ++w) {
                cost[i] += line.cost[i][w];
                units[i] += line.units[i][w];
            }
            cost[i] = uniform(cost[i]);
            units[i] = uniform(units[i]);
        }
        // Workgroups of the wide line: by what it costs, no more than make sense where the other one can
        // use them.
        const int block = blockIdx.x;
        const int grid = s.grid;
        int wide = grid;
        if (cost[0] == 0) {
            wide = 0;
        } else if (cost[1] > 0) {
            const int most_wide = min(divide(cost[0], kWideLeast) + 1, grid);
            const int most_narrow = min(divide(cost[1], kTileWaves * kNarrowLeast) + 1, grid);
            const float of_wide = static_cast<float>(cost[0]);
            const float of_all = of_wide + kNarrowWeight<DP> * static_cast<float>(cost[1]);
            wide = min(static_cast<int>(of_wide / of_all * static_cast<float>(grid)), most_wide);
            wide = max(wide, min(grid - most_narrow, most_wide));
            wide = min(max(wide, 1), grid - 1);
        }
        wide = uniform(wide);
        const bool narrow = block >= wide;
        const int workers = narrow ? (grid - wide) * kTileWaves : wide;
        const int my_cost = narrow ? cost[1] : cost[0], my_units = narrow ? units[1] : units[0];
        // Pieces of one unit each, where there are workers enough (every unit rounds up once).
        Place at;
        at.worker = narrow ? (block - wide) * kTileWaves + wid : block;
        at.slot = (narrow ? wide * kTileRows : 0) +
                  at.worker * (narrow ? kWaveRows : kTileRows);
        at.whole = 2 * my_units <= workers && my_cost < 1 << 27;
        const int pieces = at.whole ? workers - my_units : workers;
        const int least = (narrow ? kNarrowLeast : kWideLeast) +
                          (at.whole ? 0 : narrow ? kNarrowStart : kWideStart);
        at.span = uniform(max((my_cost + max(pieces, 1) - 1) / max(pieces, 1), least));
        // Lengths, and their sums: two entries of a thread.
        if (tid < n_prefixes) line.upto[tid] = lengths(at, narrow, shared_rows, shared_tiles);
        if (tid < buckets) {
            int sum = bucket == 1 ? lengths(at, narrow, rows, tiles) : 0;
            if (bucket > 1)
#pragma unroll 1
                for (int b = b0; b < b1; ++b) {
                    q = sequence(s, b);
                    sum += lengths(at, narrow, q.tokens() * s.heads, own_tiles(q));
                }
            line.upto[n_prefixes + tid] = sum;
        }
        __syncthreads();
        const int v0 = 2 * tid < entries ? line.upto[2 * tid] : 0;
        const int v1 = 2 * tid + 1 < entries ? line.upto[2 * tid + 1] : 0;
        const int scan = wave_scan_dpp(v0 + v1);
        if (lane == kWave - 1) line.cost[0][wid] = scan;
        __syncthreads();
        int before = scan - v0 - v1, all = 0;
#pragma unroll
        for (int w = 0; w < kTileWaves; ++w) {
            before += w < wid ? line.cost[0][w] : 0;
            all += line.cost[0][w];
        }
        if (2 * tid < entries) line.upto[2 * tid] = before + v0;
        if (2 * tid + 1 < entries) line.upto[2 * tid + 1] = before + v0 + v1;
        // (a worker without a piece: at the line's end)
        at.x = static_cast<int>(min(static_cast<int64_t>(at.worker) * at.span,
                                    static_cast<int64_t>(all)));
        at.end = min(at.x + at.span, all);
        if (lane == 0) line.place[wid] = at;
        __syncthreads();
        return narrow;
    }

    // Tiles of a unit that begin before `at` of its cost.
    __device__ __forceinline__ static int tiles_before(int at, int tiles) {
        if (at <= 0) return 0;
        at -= NARROW ? kNarrowStart : kWideStart;
        return min(max((at + kTileCost - 1) / kTileCost, 1), tiles);
    }

    // The piece at the worker's place.
    __device__ __forceinline__ Piece piece() const {
        const Place st = place();
        const int lane = threadIdx.x & (kWave - 1), x = st.x;
        const int n_prefixes = s.x.n, entries = n_prefixes + s.buckets;
        constexpr int kEach = kEntries / kWave;
        static_assert(kEach <= kWave, "two steps");
        constexpr uint64_t kLast = 1ull << 63;
        Piece p;
        // the first entry that ends after x
        uint64_t hit = __ballot(line.upto[min(lane * kEach + kEach - 1, entries - 1)] > x);
        const int from = static_cast<int>(__builtin_ctzll(hit | kLast)) * kEach;
        hit = __ballot(line.upto[min(from + lane, entries - 1)] > x);
        const int entry = min(from + static_cast<int>(__builtin_ctzll(hit | kLast)), entries - 1);
        int base = entry > 0 ? line.upto[entry - 1] : 0;
        p.of_prefix = entry < n_prefixes;
        p.group = p.of_prefix ? entry : (entry - n_prefixes) * s.bucket;
        p.tiles = line.tiles[entry];
        int tokens = p.of_prefix ? line.tokens[entry] : line.seq[entry - n_prefixes].tokens();
        if (__builtin_expect(s.bucket > 1 && !p.of_prefix, 0)) {
            // the sequence of its bucket
            int b = p.group;
            for (;; b += kWave) {
                int n = 0;
                if (b + lane < s.c.n_seqs) {
                    const Sequence q = sequence(s, b + lane);
                    n = lengths(st, NARROW, q.tokens() * s.heads, own_tiles(q));
                }
                const int scan = wave_scan_dpp(n);
                hit = __ballot(base + scan > x);
                if (hit || b + kWave >= s.c.n_seqs) {
                    const int w = hit ? __builtin_ctzll(hit) : 0;
                    base += __builtin_amdgcn_readlane(scan - n, w);
                    b += w;
                    break;
                }
                base += __builtin_amdgcn_readlane(scan, kWave - 1);
            }
            p.group = uniform(b);
            const Sequence q = sequence(s, p.group);
            tokens = q.tokens();
            p.tiles = own_tiles(q);
        }
        p.tiles = uniform(p.tiles);
        p.rows = uniform(tokens) * s.heads;
        base = uniform(base);
        const int cost = uniform(length(st, p.rows, p.tiles));
        const int unit = uniform(divide(x - base, cost)), unit_at = base + unit * cost;
        // (the units of a head one after the other: narrow ones, of neighbouring waves, read the same
        // keys)
        const int row_tiles = (p.rows + unit_rows(NARROW) - 1) / unit_rows(NARROW);
        p.hk = uniform(divide(unit, row_tiles));
        p.row0 = (unit - p.hk * row_tiles) * unit_rows(NARROW);
        p.first = x == unit_at;
        if (st.whole) {
            p.next = x + st.span;
            p.parts = uniform(divide(cost, st.span));
            const int part = uniform(divide(x - unit_at, st.span));
            const int each = uniform(divide(p.tiles, p.parts)), more = p.tiles - each * p.parts;
            p.t0 = part * each + min(part, more);
            p.t1 = p.t0 + each + (part < more ? 1 : 0);
        } else {
            const int end = min(unit_at + cost, st.end);
            p.next = end;
            p.t0 = uniform(tiles_before(x - unit_at, p.tiles));
            p.t1 = end == unit_at + cost ? p.tiles : uniform(tiles_before(end - unit_at, p.tiles));
            // the last tile's piece: where it begins
            const int last = p.tiles > 1 ? unit_at + cost - kTileCost : unit_at;
            p.parts = uniform(divide(last, st.span)) - st.worker + 1;
        }
        // (Sums past 31 bits, which no q_start as it has to be leads to: nothing is done.)
        if (__builtin_expect(p.rows <= 0 || unit < 0 || unit >= units_of(p.rows) || p.next <= x ||
                                 p.t0 < 0 || p.t0 > p.t1 || p.t1 > p.tiles,
                             0)) {
            p.first = false;
            p.t0 = p.t1 = 0;
            p.next = st.end;
        }
        return p;
    }

    // The unit's rows from p.row0 on, as this lane's row `at` sees it. lists: LDS of a word for each of
    // the unit's rows, free before and after.
    __device__ __forceinline__ void rows_of(const Piece &p, int at, int *lists, int *lists2,
                                            TileRows *r) const {
        const int G = s.heads, lane = threadIdx.x & (kWave - 1);
        const int row = p.row0 + at, last_row = min(p.row0 + unit_rows(NARROW), p.rows) - 1;
        const auto barrier = [] {  // of the workers
            if (NARROW) {
                asm volatile("" ::: "memory");
                __builtin_amdgcn_wave_barrier();
            } else {
                __syncthreads();
            }
        };
        const int safe = min(row, last_row), tok = divide(safe, G);
        const int tok0 = uniform(divide(p.row0, G)), tok1 = uniform(divide(last_row, G));
        r->hk = p.hk;
        r->part = p.t0;
        r->part_end = p.t1;
        r->parts = max(p.tiles, 1);
        r->head = p.hk * G + safe - tok * G;
        r->live = row <= last_row;
        r->of_prefix = p.of_prefix;
        r->first_piece = p.first;
        r->pieces = p.parts;
        r->next = p.next;
        if (p.of_prefix) {
            // the tokens of the sequences that share the prefix, one sequence after the other
            int oldest = kNewest, newest = -kRowsMost, count = 0;
            const int cut = uniform(line.cut[p.group]);
#pragma unroll 1
            for (int base = 0; base < s.c.n_seqs && count <= tok1; base += kWave) {
                const int b = base + lane;
                int n = 0, q0 = 0, pos0 = 0;
                if (b < s.c.n_seqs) {
                    const Sequence q = sequence_at(b);
                    n = q.prefix() == p.group && shares(q, cut) ? q.tokens() : 0;
                    q0 = q.q0;
                    pos0 = first_position(q);
                }
                const int upto = wave_scan_dpp(n), start = count + upto - n;
                const int lo = max(tok0 - start, 0), hi = min(tok1 - start, n - 1);
                if (lo <= hi && pos0 + hi >= 0) {  // (a position below 0 sees no key)
                    oldest = min(oldest, max(pos0 + lo, 0));
                    newest = max(newest, pos0 + hi);
                }
                if (NARROW || threadIdx.x < kWave)
#pragma unroll 1
                    for (int j = lo; j <= hi; ++j) {
                        lists[start + j - tok0] = q0 + j;
                        lists2[start + j - tok0] = pos0 + j;
                    }
                count += __builtin_amdgcn_readlane(upto, kWave - 1);
            }
            barrier();
            r->token = lists[tok - tok0];
            r->pos = lists2[tok - tok0];
            barrier();
            r->tile_first = wave_oldest(oldest);
            r->tile_last = wave_newest(newest);
            r->first = wave_oldest(r->pos);
            r->last = wave_newest(r->pos);
            r->cut = cut;
            r->first_table = s.x.table + p.group * s.x.ld_table;
            r->table = r->first_table;
            r->from_cut = false;
            r->to_cut = true;
            r->direct = false;
        } else {
            Sequence q = sequence_at(p.group);
            q.q0 = uniform(q.q0);
            q.n_keys = uniform(q.n_keys);
            q.packed = uniform(q.packed);
            const int last = q.n_keys - 1, pos0 = q.n_keys - q.tokens();
            r->token = q.q0 + tok;
            r->pos = s.every ? last : pos0 + tok;
            r->tile_first = s.every ? last : pos0 + tok0;
            r->tile_last = s.every ? last : pos0 + tok1;
            r->first = uniform(__builtin_amdgcn_readlane(r->pos, 0));
            r->last = uniform(__builtin_amdgcn_readlane(r->pos, kWave - 1));
            r->cut = uniform(cut_of(q));
            r->table = s.c.table + p.group * s.c.ld_table;
            r->first_table = r->cut > 0 ? s.x.table + q.prefix() * s.x.ld_table : r->table;
            r->from_cut = shares(q, r->cut);
            r->to_cut = false;
            r->direct = !r->from_cut && p.first && p.parts == 1;
        }
    }

    // What the join has to know of the row in `place` of the unit, by the unit's first piece.
    __device__ __forceinline__ void write_record(const TileRows &r, int place) const {
        if (!r.first_piece) return;
        const Workspace w = workspace(s);
        const int64_t pair = r.token * static_cast<int64_t>(s.a.n_heads) + r.head;
        const int rest = this->place().slot + (NARROW ? kWaveRows : kTileRows) + place;
        const int parts = r.direct ? -1 : r.pieces + (NARROW ? kNarrowRecord : 0);
        (r.of_prefix ? w.prefix : w.own)[pair] = {parts, rest};
        if (!r.of_prefix && !r.from_cut) w.prefix[pair] = {0, 0};
    }
    // The partial sums of that row; where `lead`, its maximum and sum of weights are written, and its
    // record.
    __device__ __forceinline__ float *write_sums(const TileRows &r, int place, float m, float l,
                                                 bool lead) const {
        const Workspace w = workspace(s);
        const int64_t pair = r.token * static_cast<int64_t>(s.a.n_heads) + r.head;
        const int64_t row = r.first_piece ? pair + (r.of_prefix ? w.pairs : 0)
                                          : 2 * w.pairs + this->place().slot + place;
        if (lead) {
            write_record(r, place);
            w.ml[2 * row] = m;
            w.ml[2 * row + 1] = l;
        }
        return w.o + row * s.c.head_dim;
    }
};

// What the wide body asks for (attn_tile.h).
template <int DP>
struct UnitRows {
    using Args = UnitArgs;
    struct State {
        Line *line;
    };
    static constexpr bool kTwoTables = true;
    template <int, int>
    __device__ __forceinline__ static bool find(const Args &s, const State &state, int wid, int lane,
                                                uint16_t *lists, uint16_t *lists2, TileRows *r) {
        const Units<DP, false> units = {s, *state.line};
        const Piece p = units.piece();
        __syncthreads();  // (the LDS is free)
        r->next = p.next;
        if (!p.first && p.t0 == p.t1) return false;
        units.rows_of(p, wid * 32 + (lane & 31), reinterpret_cast<int *>(lists),
                      reinterpret_cast<int *>(lists2), r);
        return true;
    }
    __device__ __forceinline__ static float *write_sums(const Args &s, const State &state,
                                                        const TileRows &r, float m, float l,
                                                        bool lead) {
        return Units<DP, false>{s, *state.line}.write_sums(r, row_place(), m, l, lead);
    }
    __device__ __forceinline__ static void write_record(const Args &s, const State &state,
                                                        const TileRows &r) {
        Units<DP, false>{s, *state.line}.write_record(r, row_place());
    }
    __device__ __forceinline__ static bool is_partial(const Args &, const TileRows &r) {
        return !r.direct;
    }
    __device__ __forceinline__ static int row_place() {
        return (threadIdx.x >> 6) * 32 + (threadIdx.x & 31);
    }
};

// A narrow unit (attn_narrow.h).
struct NarrowUnit {
    KeyTiles<kNarrowTile, true> tiles;
    const int32_t *table;
    const uint16_t *q;
    int head;
    int begin, end, lo, sinks_end;  // keys that some row sees: begin .. end, from lo on or sinks
    int pos, before;                // the lane's row: newest key, newest one out of its window
    __device__ __forceinline__ const uint16_t *query() const { return q; }
    __device__ __forceinline__ int start(int t) const { return tiles.key(t); }
    __device__ __forceinline__ bool visible(int p) const {
        return (p >= begin) & (p <= end) & ((p >= lo) | (p < sinks_end));
    }
    __device__ __forceinline__ bool sees(int p) const {
        return (p >= begin) & (p <= pos) & ((p > before) | (p < sinks_end));
    }
    __device__ __forceinline__ int safe_key(int s0) const {
        const int p = min(max(s0, begin), end);
        if (p < sinks_end || p >= lo) return p;
        return lo <= end ? lo : max(min(sinks_end - 1, end), begin);
    }
};

// The piece at the wave's place; returns where the next one begins.
template <int DP, bool PAGE16>
__device__ __forceinline__ int narrow_piece(const UnitArgs &s, Line &line, uint16_t *lds) {
    const Units<DP, true> units = {s, line};
    const AttnArgs &a = s.a;
    const int lane = unknown(threadIdx.x) & (kWave - 1), at = lane & (kNarrowRows - 1), g = lane >> 4;
    const int D = s.c.head_dim;
    const Piece p = units.piece();
    if (!p.first && p.t0 == p.t1) return p.next;
    TileRows r;
    int *lists = reinterpret_cast<int *>(lds);
    units.rows_of(p, at, lists, lists + kNarrowRows, &r);
    const int lo = a.window > 0 ? max(r.tile_first - a.window + 1, 0) : 0;
    const int sinks_end = a.window > 0 ? a.sinks : 0;
    const int end = r.to_cut ? min(r.tile_last, r.cut - 1) : r.tile_last;
    const NarrowUnit unit = {KeyTiles<kNarrowTile, true>(r, lo, sinks_end),
                             r.table,
                             a.q + r.token * a.ldq + static_cast<int64_t>(r.head) * D,
                             p.hk,
                             r.from_cut ? r.cut : 0,
                             end,
                             lo,
                             sinks_end,
                             min(r.pos, end),
                             a.window > 0 ? r.pos - a.window : -1};
    const int t0 = unit.tiles.share(r.part, r.parts), t1 = unit.tiles.share(r.part_end, r.parts);
    floatx4_t o[DP / 16];
    float m, l;
    narrow_wave<DP, PAGE16, 1>(a, s.c, unit, t0, t1, lds, o, &m, &l);
    if (!r.live) return p.next;
    if (!r.direct) {
        float *to = units.write_sums(r, at, m, l, g == 0) + 4 * g;
#pragma unroll
        for (int d = 0; d < DP / 16; ++d)
            if (16 * d + 4 * g < D) *reinterpret_cast<floatx4_t *>(to + 16 * d) = o[d];
        return p.next;
    }
    if (g == 0) units.write_record(r, at);
    if (a.lse && g == 0) a.lse[r.token * static_cast<int64_t>(a.n_heads) + r.head] = log_sum(m, l);
    const float inv = inverse_sum(l);
    const bool wide = wide_rows(a);
    const int64_t to = r.token * a.ldy + static_cast<int64_t>(r.head) * D;
#pragma unroll
    for (int d = 0; d < DP / 16; ++d)
        if (16 * d + 4 * g < D)
            store_out4(a.y, to + 16 * d + 4 * g, o[d] * inv, a.out_f32, wide);
    return p.next;
}

template <int DP, int PAGES>
__global__ void __launch_bounds__(kThreads)
__attribute__((amdgpu_waves_per_eu(2, 2))) attn_units_kernel(UnitArgs args) {
    using L = TileLayout<DP>;
    constexpr int KT = tile_keys(DP);
    constexpr bool kNarrow = kNarrowMost<DP> > 0;
    constexpr int kKeys = KT / L::kSpan * L::kKeyBlock, kValues = KT / L::kSpan * L::kValueBlock;
    constexpr int kLeast = kNarrow ? kNarrowElements<DP> : 0;
    __shared__ __attribute__((aligned(16))) uint16_t sk0[kKeys > kLeast ? kKeys : kLeast];
    __shared__ __attribute__((aligned(16))) uint16_t sk1[kKeys > kLeast ? kKeys : kLeast];
    __shared__ __attribute__((aligned(16))) uint16_t sv0[kValues > kLeast ? kValues : kLeast];
    __shared__ __attribute__((aligned(16))) uint16_t sv1[kValues > kLeast ? kValues : kLeast];
    __shared__ int votes[kTileWaves];
    __shared__ Line line;

    const int wid = uniform(threadIdx.x / kWave);
    Place &place = line.place[wid];
    const bool narrow = Units<DP, false>{args, line}.plan(reinterpret_cast<int *>(sk0));
    // (arguments read anew for each piece: kept in registers across the pieces, they were spilled to
    // lanes of vector registers, and those to memory, within the loops over keys)
    if constexpr (kNarrow) {
        if (narrow) {
            uint16_t *lds = wid == 0 ? sk0 : wid == 1 ? sk1 : wid == 2 ? sv0 : sv1;
            while (uniform(place.x) < uniform(place.end))
                place.x =
                    narrow_piece<DP, PAGES != kAnyPages>(args_again<UnitArgs>(), line, lds);
            return;
        }
    }
    while (uniform(place.x) < uniform(place.end))
        place.x = attn_tile<UnitRows<DP>, DP, KT, PAGES, false>(args_again<UnitArgs>(), {&line}, sk0,
                                                                sk1, sv0, sv1, votes);
}

// Joins the partial results of a (token row, head), one wave each: groups of LANES lanes, 4 dims a
// lane, take every (64 / LANES)th of them and meet at the end, all in a fixed order.
template <int LANES>
__global__ void __launch_bounds__(256) attn_units_join_kernel(UnitArgs s) {
    const AttnArgs &a = s.a;
    const Workspace w = workspace(s);
    const int64_t pair = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, D = s.c.head_dim;
    const int64_t token = pair / a.n_heads;
    if (pair >= w.pairs) return;
    // (rows that q_start gives to no sequence have no record)
    if (a.q_start && (token < a.q_start[0] || token >= a.q_start[s.c.n_seqs])) return;
    const Record own = w.own[pair], prefix = w.prefix[pair];
    if (own.parts < 0) return;
    // (whatever q_start holds: rows of the workspace)
    const int most = s.grid * kTileRows - 1, workers = s.grid * kTileWaves;
    const int own_parts = min(own.parts & (kNarrowRecord - 1), workers);
    const int total = own_parts + min(prefix.parts & (kNarrowRecord - 1), workers);
    const int col = 4 * (lane % LANES), d = min(col, D - 4);
    float m = kNoMax, l = 0.0f;
    floatx4_t v = floatx4_t(0.0f);
    const auto add = [&](float m1, float l1, floatx4_t v1) {
        const float m2 = fmaxf(m, m1);
        const float f = __builtin_amdgcn_exp2f(m - m2), f1 = __builtin_amdgcn_exp2f(m1 - m2);
        m = m2;
        l = l * f + l1 * f1;
        v = v * f + v1 * f1;
    };
    // (Eight at once: 4 sequences over 1000 keys 17.5 us for 16.4; two: 16 over 16384 32.5 for 31.3.)
#pragma unroll 4
    for (int i = lane / LANES; i < total; i += kWave / LANES) {
        const bool second = i >= own_parts;
        const int part = second ? i - own_parts : i;
        const Record rec = second ? prefix : own;
        const int rest = rec.rest + (part - 1) * (rec.parts & kNarrowRecord ? kWaveRows : kTileRows);
        const int64_t row = part == 0 ? pair + (second ? w.pairs : 0)
                                      : 2 * w.pairs + min(max(rest, 0), most);
        const float m1 = w.ml[2 * row], l1 = w.ml[2 * row + 1];
        const floatx4_t v1 = *reinterpret_cast<const floatx4_t *>(w.o + row * D + d);
        // (a piece without keys has written no weighted sums)
        add(m1, l1, l1 == 0.0f ? floatx4_t(0.0f) : v1);
    }
#pragma unroll
    for (int o = LANES; o < kWave; o <<= 1) {
        floatx4_t v1;
#pragma unroll
        for (int i = 0; i < 4; ++i) v1[i] = __shfl_xor(v[i], o, kWave);
        add(__shfl_xor(m, o, kWave), __shfl_xor(l, o, kWave), v1);
    }
    if (lane >= LANES) return;
    if (a.lse && lane == 0) a.lse[pair] = log_sum(m, l);
    if (col < D)
        store_out4(a.y, token * a.ldy + (pair - token * a.n_heads) * D + col, v * inverse_sum(l),
                   a.out_f32, wide_rows(a));
}

template <int DP>
void launch(const UnitArgs &s, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(s.grid)), block(kThreads);
    if (s.c.page_mask >= tile_keys(DP) - 1)
        hipLaunchKernelGGL((attn_units_kernel<DP, kTilePages>), grid, block, 0, stream, s);
    else if (s.c.page_mask >= 15)
        hipLaunchKernelGGL((attn_units_kernel<DP, kSpanPages>), grid, block, 0, stream, s);
    else
        hipLaunchKernelGGL((attn_units_kernel<DP, kAnyPages>), grid, block, 0, stream, s);
}

// The workgroups that run at once: two on a compute unit, by LDS.
int grid_of() { return 2 * device_cu_count(); }

// The line's length: units, times the tiles that a unit can have, at the highest cost: in 31 bits.
bool supported(int64_t T, int n_heads, const KvView &c, int n_prefixes, int prefix_capacity) {
    const int64_t G = n_heads / c.n_kv;
    if (T > kMostTokens || c.n_seqs > kMostSequences ||
        T * n_heads > static_cast<int64_t>(kMaxThreads) / kWave - 4)
        return false;  // (the join's waves)
    const int64_t wide = 2 * (T * G / kTileRows), groups = c.n_seqs + std::min(c.n_seqs, n_prefixes);
    const int64_t keys = std::max(c.capacity, prefix_capacity);
    if (keys > 1 << 26) return false;  // (divide, of tiles)
    const int64_t most = (keys / kNarrowTile + 3) * kTileCost + kWideStart;
    return (wide + groups) * c.n_kv <= (1 << 30) / most;
}

hipError_t launch_units(const AttnArgs &a, const KvView &c, const Prefixes &x, bool every,
                        hipStream_t stream) {
    const int bucket = (c.n_seqs + kBuckets - 1) / kBuckets;
    const UnitArgs s = {a, c, x, every, grid_of(), bucket, (c.n_seqs + bucket - 1) / bucket,
                        a.n_heads / c.n_kv};
    if (c.head_dim <= 64)
        launch<64>(s, stream);
    else if (c.head_dim <= 128)
        launch<128>(s, stream);
    else
        launch<256>(s, stream);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const dim3 grid(static_cast<unsigned>((a.T * a.n_heads + 3) / 4)), block(256);
    const auto join = c.head_dim <= 64    ? attn_units_join_kernel<16>
                      : c.head_dim <= 128 ? attn_units_join_kernel<32>
                                          : attn_units_join_kernel<64>;
    hipLaunchKernelGGL(join, grid, block, 0, stream, s);
    return hipGetLastError();
}

}  // namespace

size_t attn_shared_work_bytes(int64_t T, int n_heads, const KvView &c) {
    const int64_t pairs = T * n_heads;
    return sizeof(float) * work_rows(pairs, grid_of()) * (c.head_dim + 2) +
           sizeof(Record) * 2 * pairs;
}

bool attn_shared_supported(int64_t T, int n_heads, const KvView &c, const Prefixes &x) {
    return supported(T, n_heads, c, x.n, x.capacity);
}
hipError_t launch_attn_shared(const AttnArgs &a, const KvView &c, const Prefixes &x,
                              hipStream_t stream) {
    return launch_units(a, c, x, false, stream);
}

// Cross attention: single rows as a decode step, sequences of up to 16 rows as units, of more as prompts
// (which have most pieces' sums nowhere to write: 2 x 2000 rows over 6000 states, 28 heads over 4 of 128,
// 336 us for 385 as units; 16 x 5 rows over up to 1500, 20 heads of 64, 28 us as units for 36).
enum CrossForm { kSingle, kUnits, kPrompts };
CrossForm cross_form(int64_t T, int n_heads, const KvView &c, bool single) {
    if (single) return kSingle;
    const bool few = T * (n_heads / c.n_kv) <= c.n_seqs * int64_t{kNarrowRows};
    return few && supported(T, n_heads, c, 0, 0) ? kUnits : kPrompts;
}
bool attn_cross_supported(int64_t T, int n_heads, const KvView &c, bool single) {
    switch (cross_form(T, n_heads, c, single)) {
        case kSingle: return attn_decode_supported(n_heads, c, 0, 0);
        case kUnits: return true;
        default: return attn_prefill_supported(T, n_heads, c, 0, 0);
    }
}
size_t attn_cross_work_bytes(int64_t T, int n_heads, const KvView &c, bool single) {
    switch (cross_form(T, n_heads, c, single)) {
        case kSingle: return attn_decode_work_bytes(n_heads, c, 0, 0);
        case kUnits: return attn_shared_work_bytes(T, n_heads, c);
        default: return attn_prefill_work_bytes(T, n_heads, c, 0, 0);
    }
}
hipError_t launch_attn_cross(const AttnArgs &a, const KvView &c, hipStream_t stream) {
    switch (cross_form(a.T, a.n_heads, c, !a.q_start)) {
        case kSingle: return launch_attn_decode(a, c, stream);
        case kUnits: return launch_units(a, c, Prefixes{}, true, stream);
        default: return launch_attn_prefill_cross(a, c, stream);
    }
}

}  // namespace w4
