// attn_prefill.hip -- attention of prompts and chunks of prompts over the paged cache.
//
// y = softmax(scale Q K^T) V in one pass over the keys (w4_attn_prefill), for the rows of one
// sequence and one key-value head: the G = n_heads / n_kv query heads that share a key-value head
// are stacked, row r being token r / G, head r % G, so that a tile of rows reads each key once for
// all of them, whatever G is.
//
// A workgroup takes 128 of these rows (attn_tile.h). Bound by the sum of products and softmax: three
// prompts of up to 4096 tokens, 28 heads over 4 of 128, take 296 to 313 us over runs, 915 to 968
// TFLOP/s of the 1350 that a large matrix product reaches here, with the matrix cores busy 44 to 46
// % and the vector units 46 to 48 % of the time (32 exponentials, multiply-adds and sums, 16
// roundings and 16 maxima a lane for every 32 products). Exponentials between the products'
// instructions of the same wave left the time as it was (320 us for 321 in one run), as did two
// groups of waves in turns.
//
// Cross attention of more than 16 rows a sequence and key-value head runs here too, its rows all at the
// last position: 2 x 2000 rows over 6000 keys 336 us (905 TFLOP/s).
#include <algorithm>

#include "attn_tile.h"

namespace w4 {

namespace {

// A block's rows: of sequence `seq`, stacked rows row0 .. row0 + BM - 1 of `rows`; token row q0 and
// position pos0 of stacked row 0.
struct Tile {
    int seq, row0, rows, q0, pos0;
};

// Tiles of BM rows of all sequences in the order in which they are given out: the tiles that see
// most keys first (by their level: the tile's number in its sequence plus the tiles its earlier
// keys would make), so that the last ones to run are short. With CROSS every tile of a sequence sees
// all of its keys, which are its level (2 x 2000 rows over 6000 states 336 us for 350, 28 heads over 4
// of 128). Up to 64 sequences, a lane each; more are taken in order, the last rows of each first. Every
// lane of every wave takes part.
template <int BM, bool CROSS>
__device__ __forceinline__ bool find_tile(const KvView &c, const int32_t *q_start, int64_t T,
                                          int G, int tile, Tile *out) {
    const int lane = threadIdx.x & (kWave - 1);
    int before = 0;
    for (int base = 0; base < c.n_seqs; base += kWave) {
        const int b = base + lane;
        int begin = 0, nq = 0, n_keys = 0;
        if (b < c.n_seqs) {
            begin = max(read_const(q_start + b), 0);
            nq = max(min(read_const(q_start + b + 1), static_cast<int>(T)) - begin, 0);
            n_keys = kv_length(c, b);
        }
        const int mine = (nq * G + BM - 1) / BM;
        const int sum = wave_scan_dpp(mine);
        const int all = __builtin_amdgcn_readlane(sum, kWave - 1);
        if (tile >= before + all) {
            before += all;
            continue;
        }
        int w, row_tile;  // the lane of the sequence, the tile's number in it
        if (c.n_seqs <= kWave) {
            // levels first .. first + mine - 1 are this sequence's (CROSS: `first`, of 64 keys each);
            // the largest level with more than `tile` tiles at it or above
            const int first =
                CROSS ? n_keys >> 6
                      : static_cast<int>(min(static_cast<int64_t>(max(n_keys - nq, 0)) * G / BM,
                                             int64_t{1} << 29));
            const auto from_level = [&](int level) {  // this sequence's tiles at it or above
                return CROSS ? (first >= level ? mine : 0) : max(min(first + mine - level, mine), 0);
            };
            int lo = 0, hi = wave_max_dpp(CROSS ? first : first + mine);
            while (lo < hi) {
                const int mid = lo + (hi - lo + 1) / 2;
                if (wave_sum_dpp(from_level(mid)) > tile)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int above = wave_sum_dpp(from_level(lo + 1));
            const int here = from_level(lo) - from_level(lo + 1);
            const int upto = wave_scan_dpp(here);  // (with every lane: outside of any condition)
            const uint64_t hit = __ballot((here != 0) & (above + upto > tile));
            if (!hit) return false;
            w = __builtin_ctzll(hit);
            row_tile = CROSS ? tile - above - __builtin_amdgcn_readlane(upto - here, w)
                             : lo - __builtin_amdgcn_readlane(first, w);
        } else {
            const uint64_t hit = __ballot(before + sum > tile);
            if (!hit) return false;
            w = __builtin_ctzll(hit);
            row_tile = before + __builtin_amdgcn_readlane(sum, w) - tile - 1;
        }
        const int tokens = __builtin_amdgcn_readlane(nq, w);
        out->seq = base + w;
        out->rows = tokens * G;
        out->row0 = row_tile * BM;
        out->q0 = __builtin_amdgcn_readlane(begin, w);
        out->pos0 = __builtin_amdgcn_readlane(n_keys, w) - tokens;
        return true;
    }
    return false;
}

// Partial results of split `part`: per (token row, head) D weighted sums, and the pair (maximum in
// log2 units, sum of weights).
struct Partials {
    float *o, *ml;
};
__device__ __forceinline__ Partials partials(void *work, int64_t pairs, int splits, int part,
                                             int D) {
    float *base = static_cast<float *>(work);
    return {base + part * pairs * D, base + splits * pairs * D + part * pairs * 2};
}

// What the tile kernel asks of a call: CROSS, where every row sees all keys of its sequence.
template <bool CROSS>
struct PrefillRows {
    struct Args {
        AttnArgs a;
        KvView c;
        int splits;
    };
    struct State {};
    static constexpr bool kTwoTables = false;

    template <int DP, int KT>
    __device__ __forceinline__ static bool find(const Args &args, const State &, int wid, int lane,
                                                uint16_t *, uint16_t *, TileRows *r) {
        const AttnArgs &a = args.a;
        const KvView &c = args.c;
        const int G = a.n_heads / c.n_kv;
        r->hk = blockIdx.x % c.n_kv;
        r->part = blockIdx.x / c.n_kv % args.splits;
        r->part_end = r->part + 1;
        r->parts = args.splits;
        Tile t;
        if (!find_tile<kTileRows, CROSS>(c, a.q_start, a.T, G, blockIdx.x / c.n_kv / args.splits, &t))
            return false;
        const int row = t.row0 + wid * 32 + (lane & 31);
        const int safe_row = min(row, t.rows - 1);
        const int tok = safe_row / G;
        r->token = t.q0 + tok;
        r->head = r->hk * G + (safe_row - tok * G);
        r->live = row < t.rows;
        const auto position = [&](int row) {
            const int last = t.rows - 1;
            return t.pos0 + (CROSS ? last : min(row, last)) / G;
        };
        r->pos = position(row);
        r->tile_first = position(t.row0);
        r->tile_last = position(t.row0 + kTileRows - 1);
        r->first = position(t.row0 + wid * 32);
        r->last = position(t.row0 + wid * 32 + 31);
        r->table = c.table + t.seq * c.ld_table;
        return true;
    }
    __device__ __forceinline__ static bool is_partial(const Args &args, const TileRows &) {
        return args.splits > 1;
    }
    // The lane's row of partial sums; its maximum and sum of weights are written where `lead`.
    __device__ __forceinline__ static float *write_sums(const Args &args, const State &,
                                                        const TileRows &r, float m, float l,
                                                        bool lead) {
        const AttnArgs &a = args.a;
        const int D = args.c.head_dim;
        const Partials p = partials(a.work, a.T * a.n_heads, args.splits, r.part, D);
        const int64_t pair = r.token * static_cast<int64_t>(a.n_heads) + r.head;
        if (lead) {
            p.ml[2 * pair] = m;
            p.ml[2 * pair + 1] = l;
        }
        return p.o + pair * D;
    }
};

// Joins the splits of a (token row, head), one wave each: groups of LANES lanes, 4 dims a lane,
// take every (64 / LANES)th split and meet at the end, all in a fixed order.
template <int LANES>
__global__ void __launch_bounds__(256) attn_prefill_join_kernel(AttnArgs a, int D, int n_seqs,
                                                                int splits) {
    const int64_t pairs = a.T * a.n_heads;
    const int64_t pair = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    const int64_t token = pair / a.n_heads;
    // (rows that q_start gives to no sequence have no partial results)
    if (pair >= pairs || token < a.q_start[0] || token >= a.q_start[n_seqs]) return;
    const int col = 4 * (lane % LANES), at = min(col, D - 4);
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
    for (int i = lane / LANES; i < splits; i += kWave / LANES) {
        const Partials p = partials(a.work, pairs, splits, i, D);
        const float m1 = p.ml[2 * pair], l1 = p.ml[2 * pair + 1];
        const floatx4_t v1 = *reinterpret_cast<const floatx4_t *>(p.o + pair * D + at);
        // (a split without keys has written no weighted sums)
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
    const float inv = inverse_sum(l);
    if (a.lse && lane == 0) a.lse[pair] = log_sum(m, l);
    if (col < D)
        store_out4(a.y, token * a.ldy + (pair - token * a.n_heads) * D + col, v * inv, a.out_f32,
                   wide_rows(a));
}

struct Plan {
    int splits;
    int64_t tiles;  // at most this many tiles of rows: every sequence rounds up once
};
Plan plan_of(int64_t T, int n_heads, const KvView &c, int window, int sinks) {
    const int64_t G = n_heads / c.n_kv, cus = device_cu_count();
    Plan p;
    p.tiles = T * G / kTileRows + c.n_seqs;
    const int64_t blocks = p.tiles * c.n_kv;
    int64_t keys = c.capacity;
    if (window > 0 && int64_t(window) + sinks + kTileRows < keys)
        keys = int64_t(window) + sinks + kTileRows;
    const int64_t key_tiles = (keys + 63) / 64;
    p.splits = 1;
    // Few rows over many keys: the keys split over workgroups, four tiles each at least. (28 / 4
    // heads of 128: 16 tokens of 2 sequences after 16000 keys 457 us unsplit, 30 split; at least 2
    // or 8 tiles each: 16 tokens after 2000 keys 22 and 19 us for 15.)
    if (blocks < cus && key_tiles >= 8)
        p.splits = static_cast<int>(std::min({2 * cus / blocks, key_tiles / 4, int64_t{64}}));
    return p;
}

template <bool CROSS>
hipError_t launch(const AttnArgs &a, const KvView &c, hipStream_t stream) {
    const Plan p = plan_of(a.T, a.n_heads, c, a.window, a.sinks);
    launch_tiles<PrefillRows<CROSS>>({a, c, p.splits}, p.tiles * c.n_kv * p.splits, stream);
    if (p.splits > 1) {
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
        const dim3 grid(static_cast<unsigned>((a.T * a.n_heads + 3) / 4)), block(256);
        const auto join = c.head_dim <= 64    ? attn_prefill_join_kernel<16>
                          : c.head_dim <= 128 ? attn_prefill_join_kernel<32>
                                              : attn_prefill_join_kernel<64>;
        hipLaunchKernelGGL(join, grid, block, 0, stream, a, c.head_dim, c.n_seqs, p.splits);
    }
    return hipGetLastError();
}

}  // namespace

bool attn_prefill_supported(int64_t T, int n_heads, const KvView &c, int window, int sinks) {
    // (so T G, which the kernel rounds up to tiles, stays below 2^31 too)
    const Plan p = plan_of(T, n_heads, c, window, sinks);
    return p.tiles * c.n_kv * p.splits <= static_cast<int64_t>(kMaxThreads) / (kTileWaves * 64);
}

size_t attn_prefill_work_bytes(int64_t T, int n_heads, const KvView &c, int window, int sinks) {
    const Plan p = plan_of(T, n_heads, c, window, sinks);
    if (p.splits == 1) return 0;
    return sizeof(float) * p.splits * T * n_heads * (c.head_dim + 2);
}

hipError_t launch_attn_prefill(const AttnArgs &a, const KvView &c, hipStream_t stream) {
    return launch<false>(a, c, stream);
}
hipError_t launch_attn_prefill_cross(const AttnArgs &a, const KvView &c, hipStream_t stream) {
    return launch<true>(a, c, stream);
}

}  // namespace w4
