// attn_decode.hip -- attention of one new token per sequence over the paged cache.
//
// One pass over the keys and values of a sequence (w4_attn_decode), by attn_narrow.h: a unit's rows
// are the G = n_heads / n_kv query heads of a key-value head, up to 16 of them (more heads read the
// keys once per 16: 32 heads over 1, 32 x 4096 keys, 26 us).
//
// A sequence's visible keys (its sinks, then its window; all without a window) are cut into tiles
// of 32 keys. Every unit (sequence, key-value head, 16 query heads) is cut into equal shares of at
// most `per` tiles, a workgroup each, `per` being such that the shares of all sequences together
// fill the card once: ragged lengths leave no compute unit idle. In a workgroup each of the four
// waves takes every fourth tile, and the waves join in LDS. The shares of a unit that was cut meet
// in the caller's workspace, and a second kernel joins them in order.
//
// 28 heads over 4 of 128: 4 sequences of up to 131072 keys 185 us (5.5 TB/s of keys and values; a
// large copy reaches 5.0 to 5.5, an elementwise pass 6.3), 32 of up to 8192 63 us (4.4 TB/s). One
// sequence of 4097 keys takes 11.3 us: nothing but waits for memory, one after the other (page,
// keys, partial results), and two launches (7.2 and 4.2 us).
#include "attn_narrow.h"

namespace w4 {

namespace {

constexpr int kTile = kNarrowTile, kWaves = kNarrowWaves, kRows = kNarrowRows;

// The visible keys of a sequence, as tiles.
struct Keys {
    int last, lo;          // newest key; oldest key inside the window
    int n_sink, lo_tile;   // tiles of sinks; first tile after them
    int n_tiles;
    __device__ __forceinline__ int start(int t) const {
        return (t < n_sink ? t : lo_tile + t - n_sink) * kTile;
    }
};

__device__ __forceinline__ Keys visible_keys(const AttnArgs &a, int n) {  // of n keys
    Keys k;
    k.last = n - 1;
    k.lo = a.window > 0 ? max(n - a.window, 0) : 0;
    k.n_sink = (min(a.sinks, k.lo) + kTile - 1) / kTile;
    k.lo_tile = max(k.lo / kTile, k.n_sink);
    k.n_tiles = n == 0 ? 0 : k.n_sink + k.last / kTile + 1 - k.lo_tile;
    return k;
}
__device__ __forceinline__ Keys visible_keys(const AttnArgs &a, const KvView &c, int b) {
    return visible_keys(a, kv_length(c, b));
}

// How the tiles are shared out. whole_units: one share per unit (caches so short that cutting them
// costs more than it gives). Otherwise shares of at most ceil(tiles of all units / aim) tiles, and
// of one tile for each wave at least.
struct Plan {
    int units_per_seq, units, aim, grid;
    bool whole_units;
};

// The shares of one unit of sequence `seq`, which is group `first` of the launch plus `units before
// it in the sequence` times `shares`.
struct Shares {
    int seq, n_tiles, shares, first;
};

__device__ __forceinline__ int shares_of(int n_tiles, int per) {
    return (n_tiles + per - 1) / per;
}
__device__ __forceinline__ int most_tiles(const Plan &p, int all_tiles) {
    return max((all_tiles * p.units_per_seq + p.aim - 1) / p.aim, kWaves);
}

// The sequence for which stop(groups before it, groups of it, sequence) holds: every lane of a wave
// takes part, a lane per sequence. seq = n_seqs if there is none. (The entry point bounds the tiles
// of all units by 2^31.)
template <typename Stop>
__device__ __forceinline__ Shares find_shares(const AttnArgs &a, const KvView &c, const Plan &p,
                                              Stop stop) {
    const int lane = threadIdx.x & (kWave - 1);
    int n = lane < c.n_seqs ? visible_keys(a, c, lane).n_tiles : 0;
    int all = n;
    for (int b = lane + kWave; b < c.n_seqs; b += kWave) all += visible_keys(a, c, b).n_tiles;
    const int per = most_tiles(p, wave_sum_dpp(all));
    Shares s;
    for (int b0 = 0, base = 0;;) {
        const int mine = shares_of(n, per) * p.units_per_seq;
        const int sum = wave_scan_dpp(mine);
        const uint64_t hit = __ballot(stop(base + sum - mine, mine, b0 + lane));
        if (hit) {
            const int w = __builtin_ctzll(hit);
            s.seq = b0 + w;
            s.n_tiles = __builtin_amdgcn_readlane(n, w);
            s.shares = shares_of(s.n_tiles, per);
            s.first = base + __builtin_amdgcn_readlane(sum - mine, w);
            return s;
        }
        base += __builtin_amdgcn_readlane(sum, kWave - 1);
        b0 += kWave;
        if (b0 >= c.n_seqs) break;
        n = b0 + lane < c.n_seqs ? visible_keys(a, c, b0 + lane).n_tiles : 0;
    }
    s.seq = c.n_seqs;
    s.n_tiles = s.shares = s.first = 0;
    return s;
}

// A share's partial result: rows x D weighted sums (16-byte rows: D is a multiple of 8), and after
// those of all shares its `rows` maxima (log2 units) and `rows` sums of weights.
struct Partial {
    float *o, *m, *l;
};
__device__ __forceinline__ Partial partial(void *work, const Plan &p, int64_t group, int rows,
                                           int D) {
    float *base = static_cast<float *>(work);
    float *m = base + static_cast<int64_t>(p.grid) * rows * D + group * 2 * rows;
    return {base + group * rows * D, m, m + rows};
}

// The rows of a sequence without keys: zeros.
__device__ __forceinline__ void write_empty(const AttnArgs &a, const KvView &c, int b) {
    const int width = a.n_heads * c.head_dim;
    for (int i = threadIdx.x; i < width; i += kWaves * 64)
        store_out(a.y, b * a.ldy + i, 0.0f, a.out_f32);
    if (a.lse)
        for (int h = threadIdx.x; h < a.n_heads; h += kWaves * 64)
            a.lse[static_cast<int64_t>(b) * a.n_heads + h] = -INFINITY;
}

// A unit as a wave goes through it (narrow_wave).
struct DecodeUnit {
    const AttnArgs &a;
    Keys keys;
    const int32_t *table;
    int b, head, head0, n_rows, D;
    __device__ __forceinline__ const uint16_t *query() const {
        const int r = min(static_cast<int>(threadIdx.x & 15), n_rows - 1);
        return a.q + b * a.ldq + static_cast<int64_t>(head0 + r) * D;
    }
    __device__ __forceinline__ int start(int t) const { return keys.start(t); }
    __device__ __forceinline__ bool visible(int p) const {
        return (p <= keys.last) & ((p >= keys.lo) | (p < a.sinks));
    }
    __device__ __forceinline__ bool sees(int p) const { return visible(p); }
    __device__ __forceinline__ int safe_key(int s0) const {  // (the newest key if there is none)
        if (s0 < a.sinks && s0 < keys.lo) return s0;
        return s0 > keys.last || s0 + 15 < keys.lo ? keys.last : max(s0, keys.lo);
    }
};

// Registers: sums, queries and a tile of keys and values take 112 of them at 128 dims (3 waves a
// SIMD; 4 spill: decode of 4 x 131072 keys 292 us for 188) and 224 at 256 dims (one wave a SIMD; 2
// spill: 32 x 8192 keys, window 1024, 54 us for 34).
template <int DP, bool PAGE16>
__global__ void __launch_bounds__(kWaves * 64)
__attribute__((amdgpu_waves_per_eu(DP > 128 ? 1 : DP > 64 ? 3 : 4))) attn_decode_kernel(
    AttnArgs a, KvView c, Plan plan) {
    // per wave: the value tile, 32 rows of bf16; after the loop its sums, 16 rows of fp32
    __shared__ __attribute__((aligned(16))) uint16_t sv[kWaves][kNarrowElements<DP>];
    __shared__ float sm[kWaves][kRows], sl[kWaves][kRows];

    const int G = a.n_heads / c.n_kv, D = c.head_dim;
    const int row_tiles = (G + kRows - 1) / kRows;

    // A sequence without keys has no share: its rows are written by the group of its number.
    for (int e = blockIdx.x; e < c.n_seqs; e += gridDim.x)
        if (kv_length(c, e) == 0) write_empty(a, c, e);

    // this workgroup's share: tiles t0 .. t1 of a unit
    int b, unit, t0, t1;
    bool whole;
    if (plan.whole_units) {
        b = blockIdx.x / plan.units_per_seq;
        unit = blockIdx.x % plan.units_per_seq;
        t0 = 0;
        t1 = visible_keys(a, c, b).n_tiles;
        whole = true;
    } else {
        const int group = blockIdx.x;
        const Shares s = find_shares(a, c, plan, [&](int before, int mine, int) {
            return before <= group && group < before + mine;
        });
        if (s.seq == c.n_seqs) return;
        b = s.seq;
        unit = (group - s.first) / s.shares;
        const int i = group - s.first - unit * s.shares;
        t0 = static_cast<int>(static_cast<int64_t>(s.n_tiles) * i / s.shares);
        t1 = static_cast<int>(static_cast<int64_t>(s.n_tiles) * (i + 1) / s.shares);
        whole = s.shares == 1;
    }
    if (t0 == t1) return;
    b = uniform(b);
    unit = uniform(unit);
    t0 = uniform(t0);
    t1 = uniform(t1);
    const int rt = unit % row_tiles, hk = unit / row_tiles;
    const int head0 = hk * G + rt * kRows, n_rows = min(G - rt * kRows, kRows);
    const DecodeUnit u = {a, visible_keys(a, c, b), c.table + b * c.ld_table, b, hk, head0, n_rows, D};
    const bool wide = wide_rows(a);
    const int tid = threadIdx.x, lane = tid & 63, wid = uniform(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    floatx4_t o[DP / 16];
    float M, l;
    narrow_wave<DP, PAGE16, kWaves>(a, c, u, t0 + wid, t1, sv[wid], o, &M, &l);

    // Join the waves.
    constexpr int kRow = kNarrowRow<DP>;
    if (g == 0) {
        sm[wid][r] = M;
        sl[wid][r] = l;
    }
    float *my_o = reinterpret_cast<float *>(sv[wid]);
#pragma unroll
    for (int d = 0; d < DP / 16; ++d)
        *reinterpret_cast<floatx4_t *>(&my_o[r * kRow + 16 * d + 4 * g]) = o[d];
    __syncthreads();
    const Partial part = partial(a.work, plan, blockIdx.x, min(G, kRows), D);
    for (int e = tid; e < n_rows * (DP / 4); e += kWaves * 64) {
        const int row = e / (DP / 4), d = e % (DP / 4) * 4;
        if (d >= D) continue;
        float m = sm[0][row], sum = 0.0f;
#pragma unroll
        for (int w = 1; w < kWaves; ++w) m = fmaxf(m, sm[w][row]);
        floatx4_t v = floatx4_t(0.0f);
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
            const float f = __builtin_amdgcn_exp2f(sm[w][row] - m);
            sum += f * sl[w][row];
            v += f * *reinterpret_cast<const floatx4_t *>(reinterpret_cast<const float *>(sv[w]) +
                                                          row * kRow + d);
        }
        if (whole) {
            v *= inverse_sum(sum);
            store_out4(a.y, b * a.ldy + static_cast<int64_t>(head0 + row) * D + d, v, a.out_f32,
                       wide);
            if (a.lse && d == 0)
                a.lse[static_cast<int64_t>(b) * a.n_heads + head0 + row] = log_sum(m, sum);
        } else {
            *reinterpret_cast<floatx4_t *>(part.o + row * D + d) = v;
            if (d == 0) {
                part.m[row] = m;
                part.l[row] = sum;
            }
        }
    }
}

// Joins the partial results of a (sequence, head): one workgroup each, its threads over groups of
// partials and the head's dims, the groups' sums through LDS in order.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(AttnArgs a, KvView c, Plan plan) {
    __shared__ floatx4_t so[kJoinThreads];
    __shared__ float sm[kJoinThreads], sl[kJoinThreads];
    const int64_t pair = blockIdx.x;
    const int b = static_cast<int>(pair / a.n_heads), head = static_cast<int>(pair % a.n_heads);
    const int G = a.n_heads / c.n_kv, D = c.head_dim, rows = min(G, kRows);
    const Shares s = find_shares(a, c, plan, [&](int, int, int seq) { return seq == b; });
    if (s.shares <= 1) return;  // written by the first kernel
    const int row_tiles = (G + kRows - 1) / kRows, in_group = head % G;
    const int unit = head / G * row_tiles + in_group / kRows, row = in_group % kRows;
    const int n = s.shares;
    const auto part = [&](int i) {
        return partial(a.work, plan, s.first + unit * n + i, rows, D);
    };
    const int tid = threadIdx.x;
    const int lanes = D / 4;                  // threads over the dims, 4 each
    const int groups = kJoinThreads / lanes;  // (threads past groups * lanes idle)
    const int grp = tid / lanes, d = tid % lanes * 4;
    float m = kNoMax, l = 0.0f;
    floatx4_t v = floatx4_t(0.0f);
    const auto add = [&](float m1, float l1, floatx4_t v1) {
        const float m2 = fmaxf(m, m1);
        const float f = __builtin_amdgcn_exp2f(m - m2), f1 = __builtin_amdgcn_exp2f(m1 - m2);
        m = m2;
        l = l * f + l1 * f1;
        v = v * f + v1 * f1;
    };
    if (grp < groups) {
#pragma unroll 4
        for (int i = grp; i < n; i += groups) {
            const Partial p = part(i);
            add(p.m[row], p.l[row], *reinterpret_cast<const floatx4_t *>(p.o + row * D + d));
        }
        so[tid] = v;
        sm[tid] = m;
        sl[tid] = l;
    }
    __syncthreads();
    if (tid >= lanes) return;
    for (int q = 1; q < groups; ++q)
        add(sm[q * lanes + tid], sl[q * lanes + tid], so[q * lanes + tid]);
    v *= inverse_sum(l);
    store_out4(a.y, b * a.ldy + static_cast<int64_t>(head) * D + d, v, a.out_f32, wide_rows(a));
    if (a.lse && d == 0) a.lse[pair] = log_sum(m, l);
}

Plan plan_of(int n_heads, const KvView &c, int window, int sinks) {
    const int G = n_heads / c.n_kv;
    Plan p;
    p.units_per_seq = c.n_kv * ((G + kRows - 1) / kRows);
    p.units = c.n_seqs * p.units_per_seq;
    // tiles a sequence can have: its window and its sinks touch at most two partial tiles each
    int64_t keys = c.capacity;
    if (window > 0 && int64_t(window) + sinks + 4 * kTile < keys)
        keys = int64_t(window) + sinks + 4 * kTile;
    const int64_t tiles = (keys + kTile - 1) / kTile;
    const int cus = device_cu_count();
    // One launch instead of two, the longest unit's pass instead of a share's. Measured at 28 / 4
    // heads of 128, us whole / cut: one sequence of 500 keys 10.1 / 10.4, of 1000 16.0 / 10.4; 64
    // sequences (a unit for every compute unit) of 1000 keys 28 / 35, of 2000 50 / 58.
    p.whole_units = tiles <= (p.units >= cus ? 64 : 16);
    // Workgroups that run at once (by registers; 6 at 64 dims measured better than the 4 that fit:
    // 64 x 3000 keys, 8 heads, 76 us for 85). Few units: shares that fill the card once, where
    // every unit rounds up by half a share. Many: about two rounds, which even out by themselves.
    // (32 ragged sequences of up to 8192 keys, 128 units, us at 1 / 2 / 3 / 4 times the compute
    // units: 78 / 73 / 65 / 64; 100 of up to 6000, 400 units: 164 / 144 / 144 / 144, at 6 times
    // 141.)
    const int resident = cus * (c.head_dim > 128 ? 1 : c.head_dim > 64 ? 3 : 6);
    p.aim = p.units <= resident / 2 ? resident - p.units / 2 : 2 * resident;
    const int64_t most = p.units * ((tiles + kWaves - 1) / kWaves);  // shares of kWaves tiles
    const int64_t grid = static_cast<int64_t>(p.units) + p.aim;
    p.grid = p.whole_units ? p.units : static_cast<int>(grid < most ? grid : most);
    return p;
}

template <int DP>
void launch(const Plan &p, const AttnArgs &a, const KvView &c, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(p.grid));
    if (c.page_mask >= 15)
        hipLaunchKernelGGL((attn_decode_kernel<DP, true>), grid, dim3(kWaves * 64), 0, stream, a,
                           c, p);
    else
        hipLaunchKernelGGL((attn_decode_kernel<DP, false>), grid, dim3(kWaves * 64), 0, stream, a,
                           c, p);
}

}  // namespace

bool attn_decode_supported(int n_heads, const KvView &c, int window, int sinks) {
    // the tiles of all units, and their division into shares (most_tiles): in 31 bits
    const int64_t pairs = static_cast<int64_t>(c.n_seqs) * n_heads;  // units at most
    if (pairs > (INT32_MAX - (1 << 16)) / (c.capacity / kTile + 1)) return false;
    const Plan p = plan_of(n_heads, c, window, sinks);
    return p.grid <= static_cast<int64_t>(kMaxThreads) / (kWaves * 64) &&
           (p.whole_units || pairs <= static_cast<int64_t>(kMaxThreads) / kJoinThreads);
}

size_t attn_decode_work_bytes(int n_heads, const KvView &c, int window, int sinks) {
    const Plan p = plan_of(n_heads, c, window, sinks);
    const int G = n_heads / c.n_kv;
    if (p.whole_units) return 0;
    return sizeof(float) * p.grid * (G < kRows ? G : kRows) * (c.head_dim + 2);
}

hipError_t launch_attn_decode(const AttnArgs &a, const KvView &c, hipStream_t stream) {
    const Plan p = plan_of(a.n_heads, c, a.window, a.sinks);
    if (c.head_dim <= 64)
        launch<64>(p, a, c, stream);
    else if (c.head_dim <= 128)
        launch<128>(p, a, c, stream);
    else
        launch<256>(p, a, c, stream);
    if (!p.whole_units) {
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
        hipLaunchKernelGGL(attn_join_kernel,
                           dim3(static_cast<unsigned>(c.n_seqs) * static_cast<unsigned>(a.n_heads)),
                           dim3(kJoinThreads), 0, stream, a, c, p);
    }
    return hipGetLastError();
}

}  // namespace w4
