// attn_shared.hip -- attention of sequences that share prefixes (w4_attn_shared).
//
// The softmax of a row over prefix and own keys is the join of two partial ones, and the rows of all
// sequences over one prefix can be stacked: its keys are then read and multiplied once per 128 rows,
// not once per sequence. Work is cut into units of up to 128 stacked rows of one key-value head:
//   prefix units: rows of all sequences over prefix g, its keys
//   own units:    rows of one sequence, its own keys; of a sequence that fills a unit by itself (or has
//                 no prefix) all of its keys, by both tables: nothing is gained by sharing there
// and each unit's keys into equal shares of at most `per` tiles, a workgroup each, `per` being such
// that the shares of all units together fill the card once. One launch runs them (attn_tile.h); every
// workgroup finds its share by itself, from the lengths. Rows of one share are written as they are, the
// others leave weighted sums, maximum and sum of weights in the workspace, which a second kernel
// joins in order.
#include <algorithm>

#include "attn_tile.h"

namespace w4 {

namespace {

// Shares are cut for `aim` workgroups. A unit has one share at least.
struct Plan {
    int aim;
    int64_t grid;
};

struct SharedArgs {
    AttnArgs a;
    KvView c;
    Prefixes x;
    Plan plan;
};

// Least tiles of a share: what a workgroup costs besides (plan, queries, partial sums) is about as
// long as four tiles of 64 keys.
template <int KT>
constexpr int kLeast = 256 / KT;

// A sequence in this call: its rows, its keys, and the part of them that a prefix holds.
struct Sequence {
    int q0, tokens, n_keys, prefix, cut;
    bool shares;  // its rows go with a prefix unit's
};
__device__ __forceinline__ Sequence sequence(const SharedArgs &s, int b) {
    const AttnArgs &a = s.a;
    Sequence r;
    r.n_keys = kv_length(s.c, b);
    r.q0 = b;
    r.tokens = 1;
    if (a.q_start) {
        r.q0 = max(read_const(a.q_start + b), 0);
        r.tokens = max(min(read_const(a.q_start + b + 1), static_cast<int>(a.T)) - r.q0, 0);
    }
    r.prefix = read_const(s.x.of + b);
    const bool has = r.prefix >= 0 && r.prefix < s.x.n;
    r.prefix = has ? r.prefix : 0;
    r.cut = has ? prefix_length(s.x, r.prefix) : 0;
    r.shares = r.cut > 0 && r.tokens > 0 && r.tokens * (a.n_heads / s.c.n_kv) < kTileRows;
    return r;
}

// Oldest and newest of 64 positions, -kRowsMost .. kNewest.
constexpr int kRowsMost = 1 << 24, kNewest = 1 << 30;
__device__ __forceinline__ int wave_oldest(int v) { return kNewest - wave_max_dpp(kNewest - v); }
__device__ __forceinline__ int wave_newest(int v) {
    return wave_max_dpp(v + kRowsMost) - kRowsMost;
}

// The workspace. Each (token row, head) pair has a record of its partial results, of the own unit's
// and of the prefix unit's shares: how many there are, and the row of partial sums of the second one.
// The first share's is the pair's own.
struct Record {
    int parts, rest;
};
struct Workspace {
    float *o, *ml;        // [rows][D], [rows][2]
    Record *own, *prefix; // [pairs]; own[pair].parts < 0: written, nothing to join
    int64_t pairs, rows;
};
__host__ __device__ __forceinline__ int64_t work_rows(int64_t pairs, const Plan &p) {
    return 2 * pairs + static_cast<int64_t>(p.aim) * kTileRows;
}
__device__ __forceinline__ Workspace workspace(const AttnArgs &a, const KvView &c, const Plan &p) {
    Workspace w;
    w.pairs = a.T * a.n_heads;
    w.rows = work_rows(w.pairs, p);
    w.o = static_cast<float *>(a.work);
    w.ml = w.o + w.rows * c.head_dim;
    w.own = reinterpret_cast<Record *>(w.ml + w.rows * 2);
    w.prefix = w.own + w.pairs;
    return w;
}

struct SharedRows {
    using Args = SharedArgs;
    static constexpr bool kTwoTables = true;

    // Key tiles of a unit whose rows stand at first .. last.
    template <int KT>
    __device__ __forceinline__ static int key_tiles(const SharedArgs &s, int first, int last, int cut,
                                                    bool from_cut, bool to_cut) {
        const AttnArgs &a = s.a;
        TileRows t;
        t.tile_first = first;
        t.tile_last = last;
        t.cut = cut;
        t.from_cut = from_cut;
        t.to_cut = to_cut;
        return KeyTiles<KT, true>(t, a.window > 0 ? max(first - a.window + 1, 0) : 0,
                                  a.window > 0 ? a.sinks : 0)
            .n;
    }

    template <int DP, int KT>
    __device__ __forceinline__ static bool find(const Args &s, int wid, int lane, uint16_t *scratch,
                                                uint16_t *scratch2, int *sums, TileRows *r) {
        const AttnArgs &a = s.a;
        const KvView &c = s.c;
        const int G = a.n_heads / c.n_kv, n_prefixes = s.x.n;
        int *tokens = reinterpret_cast<int *>(scratch);   // of each prefix
        int *oldest = reinterpret_cast<int *>(scratch2);  // position among its rows
        const int tid = wid * kWave + lane;
        const auto row_tiles = [&](int tokens) { return (tokens * G + kTileRows - 1) / kTileRows; };
        const auto own_tiles = [&](const Sequence &q) {
            return key_tiles<KT>(s, q.n_keys - q.tokens, q.n_keys - 1, q.cut, q.shares, false);
        };
        for (int g = tid; g < n_prefixes; g += kTileWaves * kWave) {
            tokens[g] = 0;
            oldest[g] = INT32_MAX;
        }
        __syncthreads();
        int cost = 0;
        for (int b = tid; b < c.n_seqs; b += kTileWaves * kWave) {
            const Sequence q = sequence(s, b);
            if (q.shares) {
                atomicAdd(&tokens[q.prefix], q.tokens);
                if (a.window > 0) atomicMin(&oldest[q.prefix], q.n_keys - q.tokens);
            }
            cost += row_tiles(q.tokens) * own_tiles(q);
        }
        cost = wave_sum_dpp(cost);
        if (lane == 0) sums[wid] = cost;
        __syncthreads();
        cost = 0;
#pragma unroll
        for (int w = 0; w < kTileWaves; ++w) cost += sums[w];
        const auto prefix_tiles = [&](int g) {
            const int cut = prefix_length(s.x, g);
            return key_tiles<KT>(s, oldest[g], INT32_MAX, cut, false, true);
        };
        int mine = 0;
        for (int g = lane; g < n_prefixes; g += kWave)
            if (tokens[g] > 0) mine += row_tiles(tokens[g]) * prefix_tiles(g);
        cost += wave_sum_dpp(mine);
        const int64_t all = static_cast<int64_t>(cost) * c.n_kv;
        const int per = max(static_cast<int>((all + s.plan.aim - 1) / s.plan.aim), kLeast<KT>);
        const auto shares_of = [&](int tiles) { return max((tiles + per - 1) / per, 1); };

        // this workgroup's unit: prefixes first, then sequences
        const int block = blockIdx.x;
        int before = 0, units_before = 0;  // workgroups, units
        int at = -1, shares = 0;
        const auto scan = [&](int base, int n_units, int n_shares) {
            const int blocks = n_units * n_shares;
            const int upto = wave_scan_dpp(blocks), upto_units = wave_scan_dpp(n_units);
            const uint64_t hit = __ballot(block < before + upto);
            if (hit) {
                const int w = __builtin_ctzll(hit);
                at = base + w;
                shares = __builtin_amdgcn_readlane(n_shares, w);
                before += __builtin_amdgcn_readlane(upto - blocks, w);
                units_before += __builtin_amdgcn_readlane(upto_units - n_units, w);
                return true;
            }
            before += __builtin_amdgcn_readlane(upto, kWave - 1);
            units_before += __builtin_amdgcn_readlane(upto_units, kWave - 1);
            return false;
        };
        bool found = false, of_prefix = true;
        for (int base = 0; base < n_prefixes && !found; base += kWave) {
            const int g = base + lane;
            const int n = g < n_prefixes ? tokens[g] : 0;
            found = scan(base, n > 0 ? row_tiles(n) * c.n_kv : 0, n > 0 ? shares_of(prefix_tiles(g)) : 0);
        }
        if (!found) {
            of_prefix = false;
            for (int base = 0; base < c.n_seqs && !found; base += kWave) {
                const int b = base + lane;
                int n_units = 0, n_shares = 0;
                if (b < c.n_seqs) {
                    const Sequence q = sequence(s, b);
                    n_units = row_tiles(q.tokens) * c.n_kv;
                    n_shares = shares_of(own_tiles(q));
                }
                found = scan(base, n_units, n_shares);
            }
        }
        if (!found) return false;
        at = uniform(at);
        shares = uniform(shares);
        // the heads of a share one after the other, then its parts, then the row tiles
        const int i = uniform(block - before);
        const int hk = i % c.n_kv, part = i / c.n_kv % shares, row_tile = i / c.n_kv / shares;
        const int unit = row_tile * c.n_kv + hk;
        r->hk = hk;
        r->part = part;
        r->parts = shares;
        // (places of partial sums behind the pairs': one for each share after the first)
        r->extra = before + unit * shares - units_before - unit;
        r->of_prefix = of_prefix;
        // (never so where q_start is as it has to be)
        if (r->extra + shares - 1 > s.plan.aim) return false;

        const int row0 = row_tile * kTileRows, row = row0 + wid * 32 + (lane & 31);
        if (of_prefix) {
            const int rows = uniform(tokens[at]) * G;
            __syncthreads();  // (the counts are read no more)
            // the tokens of the unit's rows: token row and position
            const int t0 = row0 / G, t1 = min(row0 + kTileRows, rows) - 1;
            const int last = t1 / G;
            int *token_row = tokens, *position = oldest;
            int first_pos = kNewest, last_pos = -kRowsMost;
            int count = 0;
            for (int base = 0; base < c.n_seqs && count <= last; base += kWave) {
                const int b = base + lane;
                int n = 0, q0 = 0, pos0 = 0;
                if (b < c.n_seqs) {
                    const Sequence q = sequence(s, b);
                    n = q.shares && q.prefix == at ? q.tokens : 0;
                    q0 = q.q0;
                    pos0 = q.n_keys - q.tokens;
                }
                const int upto = wave_scan_dpp(n), start = count + upto - n;
                const int lo = max(t0 - start, 0), hi = min(last - start, n - 1);
                if (lo <= hi) {
                    first_pos = min(first_pos, pos0 + lo);
                    last_pos = max(last_pos, pos0 + hi);
                }
                if (wid == 0)
                    for (int j = lo; j <= hi; ++j) {
                        token_row[start + j - t0] = q0 + j;
                        position[start + j - t0] = pos0 + j;
                    }
                count += __builtin_amdgcn_readlane(upto, kWave - 1);
            }
            __syncthreads();
            const int safe_row = min(row, rows - 1), tok = safe_row / G;
            r->token = token_row[tok - t0];
            r->pos = position[tok - t0];
            r->head = hk * G + safe_row - tok * G;
            r->live = row < rows;
            r->tile_first = wave_oldest(first_pos);
            r->tile_last = wave_newest(last_pos);
            r->first = wave_oldest(r->pos);
            r->last = wave_newest(r->pos);
            r->cut = uniform(prefix_length(s.x, at));
            r->first_table = s.x.table + at * s.x.ld_table;
            r->table = r->first_table;
            r->from_cut = false;
            r->to_cut = true;
            r->direct = false;
            __syncthreads();  // (the tiles come where the lists are)
            return true;
        }
        __syncthreads();  // (the counts are read no more)
        const Sequence q = sequence(s, at);
        const int rows = q.tokens * G, pos0 = q.n_keys - q.tokens;
        const int safe_row = min(row, rows - 1), tok = safe_row / G;
        const auto position = [&](int row) { return pos0 + min(row, rows - 1) / G; };
        r->token = q.q0 + tok;
        r->pos = pos0 + tok;
        r->head = hk * G + safe_row - tok * G;
        r->live = row < rows;
        r->tile_first = position(row0);
        r->tile_last = position(row0 + kTileRows - 1);
        r->first = position(row0 + wid * 32);
        r->last = position(row0 + wid * 32 + 31);
        r->cut = q.cut;
        r->table = c.table + at * c.ld_table;
        r->first_table = s.x.table + q.prefix * s.x.ld_table;
        r->from_cut = q.shares;
        r->to_cut = false;
        r->direct = !q.shares && shares == 1;
        return true;
    }

    __device__ __forceinline__ static bool is_partial(const Args &, const TileRows &r) {
        return !r.direct;
    }
    // The row of partial sums of the lane's row.
    __device__ __forceinline__ static int64_t sums_row(const Args &s, const TileRows &r,
                                                       const Workspace &w) {
        if (r.part == 0)
            return (r.of_prefix ? w.pairs : 0) +
                   r.token * static_cast<int64_t>(s.a.n_heads) + r.head;
        return 2 * w.pairs + (r.extra + r.part - 1) * static_cast<int64_t>(kTileRows) +
               (threadIdx.x >> 6) * 32 + (threadIdx.x & 31);
    }
    __device__ __forceinline__ static void write_record(const Args &s, const TileRows &r) {
        if (r.part != 0) return;
        const Workspace w = workspace(s.a, s.c, s.plan);
        const int rest = r.extra * kTileRows + (threadIdx.x >> 6) * 32 + (threadIdx.x & 31);
        Record *to = r.of_prefix ? w.prefix : w.own;
        to[r.token * static_cast<int64_t>(s.a.n_heads) + r.head] = {r.direct ? -1 : r.parts, rest};
    }
    __device__ __forceinline__ static void write_sums(const Args &s, const TileRows &r, float m,
                                                      float l) {
        const Workspace w = workspace(s.a, s.c, s.plan);
        const int64_t row = sums_row(s, r, w);
        w.ml[2 * row] = m;
        w.ml[2 * row + 1] = l;
    }
    __device__ __forceinline__ static float *sums(const Args &s, const TileRows &r) {
        const Workspace w = workspace(s.a, s.c, s.plan);
        return w.o + sums_row(s, r, w) * s.c.head_dim;
    }
};

// Joins the partial results of a (token row, head), one wave each: groups of LANES lanes, 4 dims a
// lane, take every (64 / LANES)th of them and meet at the end, all in a fixed order.
template <int LANES>
__global__ void __launch_bounds__(256) attn_shared_join_kernel(SharedArgs s) {
    const AttnArgs &a = s.a;
    const KvView &c = s.c;
    const Workspace w = workspace(a, c, s.plan);
    const int64_t pair = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63, D = c.head_dim;
    if (pair >= w.pairs) return;
    const int token = static_cast<int>(pair / a.n_heads);
    RowPlace at;
    if (!place_of_row(c, a.q_start, token, &at)) return;
    const Sequence q = sequence(s, at.seq);
    Record own = w.own[pair], prefix = w.prefix[pair];
    if (own.parts < 0) return;
    if (!q.shares) prefix.parts = 0;
    // (whatever q_start holds: rows of the workspace)
    const int most = static_cast<int>(min(w.rows - 2 * w.pairs, int64_t{INT32_MAX}));
    const int total = min(own.parts, s.plan.aim + 1) + min(max(prefix.parts, 0), s.plan.aim + 1);
    own.parts = min(own.parts, s.plan.aim + 1);
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
#pragma unroll 4
    for (int i = lane / LANES; i < total; i += kWave / LANES) {
        const bool second = i >= own.parts;
        const int part = second ? i - own.parts : i;
        const int rest = (second ? prefix.rest : own.rest) + (part - 1) * kTileRows;
        const int64_t row = part == 0 ? pair + (second ? w.pairs : 0)
                                      : 2 * w.pairs + min(max(rest, 0), most - 1);
        const float m1 = w.ml[2 * row], l1 = w.ml[2 * row + 1];
        const floatx4_t v1 = *reinterpret_cast<const floatx4_t *>(w.o + row * D + d);
        // (a share without keys has written no weighted sums)
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
        store_out4(a.y, token * a.ldy + (pair - static_cast<int64_t>(token) * a.n_heads) * D + col,
                   v * inverse_sum(l), a.out_f32, wide_rows(a));
}

Plan plan_of(int64_t T, int n_heads, const KvView &c, const Prefixes &x) {
    const int64_t G = n_heads / c.n_kv;
    Plan p;
    p.aim = 2 * device_cu_count();
    // every sequence and every prefix in use rounds up once
    const int64_t units = 2 * (T * G / kTileRows) + c.n_seqs + std::min(c.n_seqs, x.n);
    p.grid = units * c.n_kv + p.aim;
    return p;
}

}  // namespace

bool attn_shared_supported(int64_t T, int n_heads, const KvView &c, const Prefixes &x, int, int) {
    const Plan p = plan_of(T, n_heads, c, x);
    // the key tiles of all units of one head: in 31 bits
    const int64_t keys = std::max(c.capacity, x.capacity);
    if ((p.grid - p.aim) / c.n_kv > INT32_MAX / (keys / tile_keys(c.head_dim) + 3)) return false;
    return p.grid <= static_cast<int64_t>(kMaxThreads) / (kTileWaves * 64);
}

size_t attn_shared_work_bytes(int64_t T, int n_heads, const KvView &c, const Prefixes &x, int, int) {
    const int64_t pairs = T * n_heads;
    return sizeof(float) * work_rows(pairs, plan_of(T, n_heads, c, x)) * (c.head_dim + 2) +
           sizeof(Record) * 2 * pairs;
}

hipError_t launch_attn_shared(const AttnArgs &a, const KvView &c, const Prefixes &x,
                              hipStream_t stream) {
    const SharedArgs s = {a, c, x, plan_of(a.T, a.n_heads, c, x)};
    launch_tiles<SharedRows>(s, s.plan.grid, stream);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
    const dim3 grid(static_cast<unsigned>((a.T * a.n_heads + 3) / 4)), block(256);
    const auto join = c.head_dim <= 64    ? attn_shared_join_kernel<16>
                      : c.head_dim <= 128 ? attn_shared_join_kernel<32>
                                          : attn_shared_join_kernel<64>;
    hipLaunchKernelGGL(join, grid, block, 0, stream, s);
    return hipGetLastError();
}

}  // namespace w4
