// attn_prefill.hip -- attention of prompts and chunks of prompts over the paged cache.
//
// y = softmax(scale Q K^T) V in one pass over the keys (w4_attn_prefill), for the rows of one
// sequence and one key-value head: the G = n_heads / n_kv query heads that share a key-value head
// are stacked, row r being token r / G, head r % G, so that a tile of rows reads each key once for
// all of them, whatever G is.
//
// Both products run transposed on v_mfma_f32_32x32x16_bf16, 32 rows per wave:
//   S^T[key][row] = K Q^T:   K from LDS, Q^T held in registers for the whole pass
//   O^T[d][row]  += V^T P^T: V from LDS through the transposed read
// A lane then holds scores of ONE row (its column), 16 of every 32 keys, the lane 32 further the
// others: the maximum needs one exchange, the rescale of O^T none, and P^T in bf16 is, register
// for register, the operand of the second product -- with the keys of a 16-key step in the order
// the first product left them, which V's rows follow.
//
// The running maximum M (in units of log2) is only raised when a tile exceeds it by more than 2^8:
// the weights then stay below 2^8 and keep their relative precision, and the accumulators are
// rarely rescaled. The weights enter the second product as bf16 (each within 2^-8 of itself, like
// the keys and values; a second product for what is cut off, as the decode kernel has it, would
// cost half as much again); their sum takes them before that rounding.
//
// A workgroup is four waves, 128 stacked rows; tiles of 64 keys (32 at 256 dims) go from memory
// straight to LDS, double buffered, one barrier a tile. Two workgroups run on a compute unit, so
// that one can multiply while the other turns scores into weights. Bound by the sum of both: three
// prompts of up to 4096 tokens, 28 heads over 4 of 128, take 296 to 313 us over runs, 915 to 968
// TFLOP/s of the 1350 that a large matrix product reaches here, with the matrix cores busy 44 to 46
// % and the vector units 46 to 48 % of the time (32 exponentials, multiply-adds and sums, 16
// roundings and 16 maxima a lane for every 32 products). Exponentials between the products'
// instructions of the same wave left the time as it was (320 us for 321 in one run), as did two
// groups of waves in turns.
#include <algorithm>

#include "attn_device.h"

namespace w4 {

namespace {

constexpr int kWaves = 4, kTileRows = 32 * kWaves;
constexpr int kSlack = 8;
constexpr float kFar = 1 << 20;

// A block's rows: of sequence `seq`, stacked rows row0 .. row0 + BM - 1 of `rows`; token row q0 and
// position pos0 of stacked row 0.
struct Tile {
    int seq, row0, rows, q0, pos0;
};

// Tiles of BM rows of all sequences in the order in which they are given out: the tiles that see
// most keys first (by their level: the tile's number in its sequence plus the tiles its earlier
// keys would make), so that the last ones to run are short. Up to 64 sequences, a lane each; more
// are taken in order, the last rows of each first. Every lane of every wave takes part.
template <int BM>
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
            // levels first .. first + mine - 1 are this sequence's; the largest level with more
            // than `tile` tiles at it or above
            const int first = static_cast<int>(
                min(static_cast<int64_t>(max(n_keys - nq, 0)) * G / BM, int64_t{1} << 29));
            int lo = 0, hi = wave_max_dpp(first + mine);
            while (lo < hi) {
                const int mid = lo + (hi - lo + 1) / 2;
                const int above = max(min(first + mine - mid, mine), 0);
                if (wave_sum_dpp(above) > tile)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int above = wave_sum_dpp(max(min(first + mine - (lo + 1), mine), 0));
            const int here = (first <= lo) & (lo < first + mine);
            const int rank = wave_scan_dpp(here);  // (with every lane: outside of any condition)
            const uint64_t hit = __ballot((here != 0) & (rank == tile - above + 1));
            if (!hit) return false;
            w = __builtin_ctzll(hit);
            row_tile = lo - __builtin_amdgcn_readlane(first, w);
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

// Orders a run of N products, each with READS LDS reads for its fragment, every fragment read AHEAD
// products before its use. (Left to itself the scheduler keeps two fragments in flight, where a
// product waits for most of an LDS read. At 256 dims registers are short: 4 key fragments ahead
// instead of 2 cost 10 %.)
template <int N, int READS, int AHEAD>
__device__ __forceinline__ void order_products() {
    constexpr int kMatrix = 0x008, kLdsRead = 0x100;
    __builtin_amdgcn_sched_group_barrier(kLdsRead, READS * AHEAD, 0);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        __builtin_amdgcn_sched_group_barrier(kMatrix, 1, 0);
        if (i + AHEAD < N) __builtin_amdgcn_sched_group_barrier(kLdsRead, READS, 0);
    }
}

// s_waitcnt immediate: vmcnt(N), the other counters not waited for.
template <int N>
constexpr int wait_vm() {
    return (N & 0xF) | (N >> 4) << 14 | 0x7 << 4 | 0xF << 8;
}

// Barrier after a tile: this wave's LDS reads are done, what it sent for has landed.
__device__ __forceinline__ void tile_barrier() {
    phase_fence();
    __builtin_amdgcn_s_waitcnt(wait_vm<0>() & 0xF0FF);  // vmcnt(0) and lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    phase_fence();
}

// The same value, as if unknown: nothing computed from it is taken for what was computed before.
__device__ __forceinline__ int unknown(int v) {
    asm volatile("" : "+v"(v));
    return v;
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

// A tile in LDS: direct loads from memory, which lay 64 lanes of 16 bytes down in a row, put kSpan
// consecutive rows of DP elements into a block of 1 KiB; blocks follow each other with a gap.
// Inside a row the 16-byte chunks are permuted (by the choice of what each lane loads), so that
// neither the key fragments (one chunk of 16 or 32 consecutive rows) nor the transposed value reads
// (32 bytes of 4 consecutive rows) meet in the same of the 64 banks: chunk c of row r is at place
//   c ^ key_swap(r) for keys,   c ^ 4 value_swap(r) for values,
// rows of 128, 256 and 512 bytes covering 1/2, 1 and 2 rows of banks.
template <int DP>
struct TileLayout {
    static constexpr int kSpan = 512 / DP;
    static constexpr int kKeyBlock = 512 + (DP > 128 ? 16 : 32);   // elements from block to block
    static constexpr int kValueBlock = 512 + (DP > 128 ? 64 : 0);
    static constexpr int kValueSwaps = DP == 128 ? 4 : 2;  // values that value_swap takes
    __device__ static int key_swap(int r) {
        return DP > 128 ? r & 1 : DP > 64 ? r & 3 : r >> 1 & 3;
    }
    __device__ static int value_swap(int r) {
        return DP > 128 ? r & 1 : DP > 64 ? r & 3 : r >> 1 & 1;
    }
    // Element offset of chunk c of row r.
    __device__ static int key_at(int r, int c) {
        return r / kSpan * kKeyBlock + r % kSpan * DP + 8 * (c ^ key_swap(r));
    }
    __device__ static int value_at(int r, int c) {
        return r / kSpan * kValueBlock + r % kSpan * DP + 8 * (c ^ 4 * value_swap(r));
    }
};

// 16 bytes per lane from memory to LDS, lane l's at lds + 16 l.
__device__ __forceinline__ void load_to_lds(const void *from, uint16_t *lds) {
    typedef const __attribute__((address_space(1))) void *global_t;
    typedef __attribute__((address_space(3))) void *lds_t;
    __builtin_amdgcn_global_load_lds((global_t)from, (lds_t)lds, 16, 0, 0);
}

// What lies in one page: a tile (pages of KT slots and more), the rows a wave stages in one
// instruction (8 at most, aligned: pages of 8 slots and more), or a row. (4 prompts of up to 2048
// tokens, 28 heads over 4 of 128: pages of 64 121 us, of 32 by spans 133. 2 chunks of up to 4096
// tokens, 16 heads over 4 of 256, window 1024, pages of 16: by spans 197 us, by rows 218.)
enum { kAnyPages = 0, kSpanPages = 1, kTilePages = 2 };

struct Args {
    AttnArgs a;
    KvView c;
    int splits;
};
// The kernel's arguments, read once more: its only parameter is at the start of their segment.
__device__ __forceinline__ Args args_again() {
    typedef const __attribute__((address_space(4))) uint32_t *const_ptr;
    uint64_t p = reinterpret_cast<uint64_t>(__builtin_amdgcn_kernarg_segment_ptr());
    asm volatile("" : "+s"(p));
    static_assert(sizeof(Args) % 4 == 0, "words");
    uint32_t words[sizeof(Args) / 4];
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(Args) / 4); ++i)
        words[i] = reinterpret_cast<const_ptr>(p)[i];
    Args args;
    __builtin_memcpy(&args, words, sizeof(Args));
    return args;
}

// One tile of rows over the keys of one split.
//
// A weight of 0 hides only a finite value from a row: 0 times infinity is NaN. So a block in which
// any sum is not finite at the end goes through its keys again with ANY set: one tile at a time, 64
// dims at a time, and values that are not finite reach only the rows that see them. Rows that see
// none come out the same, bit for bit. So does a block with a row whose scores are so large that
// their rounding matters (see `weights`). (3 prompts of up to 4096 tokens, 28 heads over 4 of 128:
// 0.30 ms, with one infinity in the longest 0.91, all values NaN 2.5. The check itself costs a call
// of 77 tokens 0.3 us.) The second pass reads its arguments anew and takes its lane number as if
// unknown: whatever the two passes shared would occupy registers throughout, and the first pass'
// loop lost its order of reads or spilled (one prompt of 2048 tokens: 54 us for 49; 2 chunks of up
// to 4096, 256 dims, window 1024: 201 us for 176).
template <int DP, int KT, int PAGES, bool ANY>
__device__ __forceinline__ void prefill_tile(const AttnArgs &a, const KvView &c, int splits,
                                             uint16_t *sk0, uint16_t *sk1, uint16_t *sv0,
                                             uint16_t *sv1, int *votes) {
    constexpr int BM = kTileRows, NW = kWaves;
    constexpr int kChunks = DP / 8;                    // 16-byte chunks of a row
    constexpr int kSpan = 64 / kChunks;                // rows a wave stages in one instruction
    constexpr int kLoads = KT / (NW * kSpan);          // instructions a wave stages a tile with
    static_assert(kLoads * NW * kSpan == KT, "every wave stages the same number of rows");
    using L = TileLayout<DP>;
    constexpr int DT = DP / 32, KS = DP / 16, SUB = KT / 32;
    const int tid = ANY ? unknown(threadIdx.x) : threadIdx.x;
    const int lane = tid & 63;
    const int wid = uniform(tid >> 6);
    const int G = a.n_heads / c.n_kv, D = c.head_dim;
    const int hk = blockIdx.x % c.n_kv, part = blockIdx.x / c.n_kv % splits;
    Tile t;
    if (!find_tile<BM>(c, a.q_start, a.T, G, blockIdx.x / c.n_kv / splits, &t)) return;

    const int half = lane >> 5;
    const int row = t.row0 + wid * 32 + (lane & 31);
    const int safe_row = min(row, t.rows - 1);
    const int tok = safe_row / G;
    const int head = hk * G + (safe_row - tok * G);
    const int pos = t.pos0 + tok;

    // positions of the block's rows (tile_first .. tile_last) and of the wave's (first .. last)
    const int tile_first = t.pos0 + t.row0 / G;
    const int tile_last = t.pos0 + min(t.row0 + BM - 1, t.rows - 1) / G;
    const int first = t.pos0 + min(t.row0 + wid * 32, t.rows - 1) / G;
    const int last = t.pos0 + min(t.row0 + wid * 32 + 31, t.rows - 1) / G;

    // Key tiles: those of the sinks, then those from the oldest key in a row's window on; of them
    // this split's.
    const int lo = a.window > 0 ? max(tile_first - a.window + 1, 0) : 0;
    const int sinks_end = a.window > 0 ? a.sinks : 0;
    const int n_sink = (min(sinks_end, lo) + KT - 1) / KT;
    const int lo_tile = max(lo / KT, n_sink);
    const int n_all = tile_last < 0 ? 0 : n_sink + tile_last / KT + 1 - lo_tile;
    const int it0 = static_cast<int>(static_cast<int64_t>(n_all) * part / splits);
    const int n_iter = static_cast<int>(static_cast<int64_t>(n_all) * (part + 1) / splits) - it0;
    const auto tile_key = [&](int it) {
        it += it0;
        return (it < n_sink ? it : lo_tile + it - n_sink) * KT;
    };

    // Q^T: lane holds dims 16 s + 8 half .. + 7 of its row
    bf16x8_t qf[KS];
    {
        const uint16_t *src = a.q + (t.q0 + tok) * a.ldq + static_cast<int64_t>(head) * D;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int d = 16 * s + 8 * half;
            const uintx4_t v = *reinterpret_cast<const uintx4_t *>(src + min(d, D - 8));
            qf[s] = __builtin_bit_cast(bf16x8_t, d < D ? v : uintx4_t{0, 0, 0, 0});
        }
    }

    floatx16_t o[DT];
#pragma unroll
    for (int i = 0; i < DT; ++i) o[i] = floatx16_t(0.0f);
    // (a scale of 0 as the smallest number, which moves no weight, so that hidden scores of -inf
    // stay -inf)
    const float cs = fmaxf(a.scale * kLog2e, 0x1p-149f);
    const int before = a.window > 0 ? pos - a.window : -1;  // newest position out of the window
    float M = kNoMax, l = 0.0f;

    // Staging: in each of kLoads instructions a wave moves kSpan consecutive rows of the tile. A
    // row whose key no row of the block sees is read from one that some row sees (finite; its
    // weights are 0; of the same rows, if there is any); dims past D from the row's last chunk
    // (they meet zeros of q, or outputs that are not kept).
    const int my_row = lane / kChunks;
    const int k_col = min(8 * (lane % kChunks ^ L::key_swap(my_row)), D - 8);
    const int v_col = min(8 * (lane % kChunks ^ 4 * L::value_swap(my_row)), D - 8);
    const int32_t *table = c.table + t.seq * c.ld_table;
    const uint16_t *head_k = c.k + static_cast<int64_t>(hk) * c.head_stride;
    const uint16_t *head_v = c.v + static_cast<int64_t>(hk) * c.head_stride;
    const auto span_at = [&](int i) { return (i * NW + wid) * kSpan; };
    const auto all_seen = [&](int k0) {  // each key of the tile by some row of the block
        return (k0 + KT - 1 <= tile_last) & ((k0 >= lo) | (k0 + KT - 1 < sinks_end));
    };
    const auto visible = [&](int p) {
        return (p <= tile_last) & ((p >= lo) | (p < sinks_end));
    };
    // a key that is seen, among the n from s0 on if any is
    const auto safe_of = [&](int s0, int n) {
        if (s0 > tile_last) return tile_last;
        if (s0 < sinks_end) return s0;
        return s0 + n - 1 < lo ? lo : max(s0, lo);
    };
    const auto page_offset = [&](int page) {
        return static_cast<int64_t>(min(max(page, 0), c.n_pages - 1)) * c.page_stride;
    };
    // A tile's rows for this lane: a base (uniform but for PAGES == kAnyPages) and an offset.
    constexpr int kBases = PAGES == kTilePages ? 1 : kLoads;
    struct Where {
        int64_t base[kBases];
        uint32_t off[kLoads];
    };
    // The offsets in a tile whose rows are all seen. At 256 dims, where registers are short, the
    // part that is uniform is added at the use. (2 chunks of up to 4096 tokens, window 1024: 170 us
    // so, 188 with a register each; at 128 dims one prompt of 2048: 51.5 so, 49.9 with registers.)
    constexpr bool kAddUniform = DP > 128 && PAGES == kTilePages;
    uint32_t row_off[kAddUniform ? 1 : kLoads];
#pragma unroll
    for (int i = 0; i < (kAddUniform ? 1 : kLoads); ++i)
        row_off[i] = ((PAGES == kTilePages && !kAddUniform ? span_at(i) : 0) + my_row) *
                     c.slot_stride;
    const auto seen_off = [&](int i) {
        return kAddUniform ? row_off[0] + uniform(span_at(i) * c.slot_stride) : row_off[i];
    };
    int entry[kBases];
    const auto look_up = [&](int it) {  // the page table entries of a tile
        const int k0 = tile_key(it);
        if constexpr (PAGES == kTilePages) {
            // (the page of the tile's first key, which is seen or a later one is)
            entry[0] = read_const(table + (k0 >> c.page_shift));
        } else if constexpr (PAGES == kSpanPages) {
            const bool all = all_seen(k0);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int s0 = k0 + span_at(i);
                entry[i] = read_const(table + ((all ? s0 : safe_of(s0, kSpan)) >> c.page_shift));
            }
        }
    };
    const auto locate = [&](int it, Where &w) {
        const int k0 = tile_key(it);
        if constexpr (PAGES == kTilePages) {
            w.base[0] = page_offset(entry[0]) +
                        static_cast<int64_t>((k0 & c.page_mask) * c.slot_stride);
            const int safe = k0 < sinks_end ? k0 : max(k0, lo);
            const uint32_t other = (safe - k0) * c.slot_stride;
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                // (uniform, to be added here: else each sum has a register of its own throughout)
                w.off[i] = visible(uniform(k0 + span_at(i)) + my_row) ? seen_off(i) : other;
        } else {
            const bool all = all_seen(k0);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int s0 = k0 + span_at(i), p = s0 + my_row;
                const int safe = all ? s0 : safe_of(s0, kSpan);
                const bool vis = all | visible(p);
                if constexpr (PAGES == kSpanPages) {
                    // the span's first row if the span has a row that is seen, else the row instead
                    const int first_row = safe >= s0 && safe < s0 + kSpan ? s0 : safe;
                    w.base[i] = page_offset(entry[i]) +
                                static_cast<int64_t>((first_row & c.page_mask) * c.slot_stride);
                    w.off[i] = vis ? seen_off(i) : (safe - first_row) * c.slot_stride;
                } else {
                    const int from = vis ? p : safe;
                    w.base[i] = page_offset(read_const(table + (from >> c.page_shift)));
                    w.off[i] = (from & c.page_mask) * c.slot_stride;
                }
            }
        }
    };
    const auto fetch = [&](const uint16_t *kv, const Where &w, int col, uint16_t *dst, int block)
                           __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            load_to_lds(reinterpret_cast<const char *>(kv + w.base[PAGES == kTilePages ? 0 : i]) +
                            2u * (w.off[i] + col),
                        dst + (i * NW + wid) * block);
    };
    // Sends for the keys of tile it + 2 and the values of tile it + 1, whose rows were found for
    // its keys. (Past the last tile both repeat it, into buffers that nothing reads any more.)
    Where newest;  // of tile it + 1
    const auto tile_at = [&](int it) { return min(it, n_iter - 1); };
    const auto send = [&](int it, uint16_t *k, uint16_t *v) __attribute__((always_inline)) {
        fetch(head_v, newest, v_col, v, L::kValueBlock);
        locate(tile_at(it + 2), newest);
        fetch(head_k, newest, k_col, k, L::kKeyBlock);
        look_up(tile_at(it + 3));
    };

    // An iteration multiplies the keys of tile i + 1 and the values of tile i, then turns the
    // scores of tile i + 1 into weights, while the other workgroup of the compute unit multiplies.
    // send(i) overwrites the buffers of keys i and values i - 1, read in the iteration before, and
    // has the iteration to land: one barrier a tile.
    floatx16_t s[SUB];
    bf16x8_t pf[SUB][2];  // the weights of the tile whose values come next

    const auto scores = [&](const uint16_t *k) __attribute__((always_inline)) {
        // (chunks 2 ks + half, swapped: even and odd steps each at constant offsets)
        const uint16_t *kp[2] = {k + L::key_at(lane & 31, half),
                                 k + L::key_at(lane & 31, 2 + half)};
#pragma unroll
        for (int u = 0; u < SUB; ++u) s[u] = floatx16_t(0.0f);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int u = 0; u < SUB; ++u)
                s[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                    *reinterpret_cast<const bf16x8_t *>(kp[ks & 1] + 32 * u / kSpan * L::kKeyBlock +
                                                        ks / 2 * 32),
                    qf[ks], s[u], 0, 0, 0);
    };
    // O^T += V^T P^T, 16 keys a step: slots 8 half + 0..3 are keys 4 half + 0..3 of the step, slots
    // 8 half + 4..7 keys 8 + 4 half + 0..3
    const auto weigh = [&](const uint16_t *v) __attribute__((always_inline)) {
        // (chunk 4 d + 2 (lane / 16 % 2) + (lane & 3) / 2 of a row, swapped: an address for each d
        // modulo the swaps, constant offsets beyond)
        constexpr int N = L::kValueSwaps;
        const int r = 4 * half + (lane & 15) / 4, c = 2 * (lane >> 4 & 1) + (lane & 3) / 2;
        const uint16_t *vp[N];
#pragma unroll
        for (int d = 0; d < N; ++d) vp[d] = v + L::value_at(r, 4 * d + c) + 4 * (lane & 1);
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int st = 0; st < 2; ++st)
#pragma unroll
                for (int d = 0; d < DT; ++d) {
                    const uint16_t *p =
                        vp[d % N] + (32 * u + 16 * st) / kSpan * L::kValueBlock + d / N * N * 32;
                    const uintx2_t v0 = lds_read_transposed(p);
                    const uintx2_t v1 = lds_read_transposed(p + 8 / kSpan * L::kValueBlock);
                    const uintx4_t vv = {v0[0], v0[1], v1[0], v1[1]};
                    o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        __builtin_bit_cast(bf16x8_t, vv), pf[u][st], o[d], 0, 0, 0);
                }
    };
    // The same for kAnyDims times 32 dims from 32 d0 on, where values may be infinite or NaN. The
    // finite ones go through the product above; the others, counted by kind for each row that sees
    // them (1 for infinity, 32 for minus infinity, 1024 for NaN; 16 keys a step), are added as what
    // they are.
    constexpr int kAnyDims = 2;
    const auto weigh_any = [&](const uint16_t *v, int d0) __attribute__((always_inline)) {
        const int r = 4 * half + (lane & 15) / 4, c = 2 * (lane >> 4 & 1) + (lane & 3) / 2;
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                uintx4_t seen;  // bf16 ones where weights are
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    seen[i] = (s[u][8 * st + 2 * i] != -INFINITY ? 0x3F80u : 0) |
                              (s[u][8 * st + 2 * i + 1] != -INFINITY ? 0x3F800000u : 0);
#pragma unroll
                for (int d = 0; d < kAnyDims; ++d) {
                    const uint16_t *p = v + (32 * u + 16 * st) / kSpan * L::kValueBlock +
                                        L::value_at(r, 4 * (d0 + d) + c) + 4 * (lane & 1);
                    const uintx2_t v0 = lds_read_transposed(p);
                    const uintx2_t v1 = lds_read_transposed(p + 8 / kSpan * L::kValueBlock);
                    const uintx4_t all = {v0[0], v0[1], v1[0], v1[1]};
                    uintx4_t kind;
                    const uintx4_t fin = split_values<0x4200u, 0x4480u>(all, &kind);
                    o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                        __builtin_bit_cast(bf16x8_t, fin), pf[u][st], o[d], 0, 0, 0);
                    if (__any((kind[0] | kind[1] | kind[2] | kind[3]) != 0)) {
                        const floatx16_t n = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                            __builtin_bit_cast(bf16x8_t, kind), __builtin_bit_cast(bf16x8_t, seen),
                            floatx16_t(0.0f), 0, 0, 0);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            o[d][i] = add_kinds<32, 1024>(o[d][i], static_cast<int>(n[i]));
                    }
                    phase_fence();
                }
            }
    };
    // Hides the scores of the keys that a row does not see, and raises M; returns the factor that
    // the sums so far have to take if it rose for any row (`rose`).
    const auto raise = [&](int it, bool *rose) __attribute__((always_inline)) {
        const int k0 = tile_key(it);
        // every key of the tile seen by every row of the wave?
        const bool whole = k0 + KT - 1 <= first &&
                           (a.window == 0 || k0 > last - a.window || k0 + KT - 1 < a.sinks);
        if (!whole) {
            // key i of the lane's is at place 32 u + 8 (i / 4) + i % 4 of those from k0 + 4 half on
            const int base = k0 + 4 * half;
            const int newest_at = pos - base, before_at = before - base;
            const int sinks_at = sinks_end - base;
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int at = 32 * u + 8 * (i / 4) + i % 4;
                    const bool ok = (at <= newest_at) & ((at > before_at) | (at < sinks_at));
                    s[u][i] = ok ? s[u][i] : -INFINITY;
                }
        }
        float mx = s[0][0];
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[u][i]);
        mx = max_of_halves(mx) * cs;
        float f = 1.0f;
        *rose = __any(mx > M + kSlack);
        if (*rose) {
            const float M2 = fmaxf(M, mx);
            f = __builtin_amdgcn_exp2f(M - M2);
            M = M2;
            l *= f;
        }
        return f;
    };
    // A weight's exponent comes from one multiply-add, while M is rounded: by as much as the
    // exponent may be off (2^-4 at kFar; 2^16 at 2^40, which overflows). With ANY, the scores of
    // rows whose M is beyond kFar are scaled, and so rounded, as M was.
    const auto is_far = [&] { return fabsf(M) > kFar && M != kNoMax; };
    const auto weights = [&]() __attribute__((always_inline)) {
        const float k = ANY && is_far() ? 1.0f : cs;
        if (ANY) {
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float scaled = s[u][i] * cs;
                    asm volatile("" : "+v"(scaled));  // (rounded, not fused with what follows)
                    s[u][i] = is_far() ? scaled : s[u][i];
                }
        }
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
            uintx4_t x[2];
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                const float p0 = __builtin_amdgcn_exp2f(fmaf(s[u][i], k, -M));
                const float p1 = __builtin_amdgcn_exp2f(fmaf(s[u][i + 1], k, -M));
                l += p0 + p1;
                x[i / 8][i % 8 / 2] = pack_bf16(p0, p1);
            }
            pf[u][0] = __builtin_bit_cast(bf16x8_t, x[0]);
            pf[u][1] = __builtin_bit_cast(bf16x8_t, x[1]);
        }
    };

    // k and v: the buffers of tile it, k1 and v1: of tile it + 1
    const auto step = [&](int it, uint16_t *k, uint16_t *v, uint16_t *k1, uint16_t *v1)
                          __attribute__((always_inline)) {
        send(it, k, v1);
        scores(k1);
        order_products<SUB * KS, 1, (DP > 128 ? 2 : 4)>();
        bool rose;
        const float f = raise(it + 1, &rose);
        weigh(v);
        order_products<SUB * 2 * DT, 2, 3>();
        phase_fence();
        if (rose) {
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d] *= f;
        }
        weights();
        tile_barrier();
    };

    const auto block_any = [&](bool v) {  // (called once)
        const bool mine = __any(v);
        if (lane == 0) votes[wid] = mine;
        __syncthreads();
        bool any = false;
#pragma unroll
        for (int w = 0; w < NW; ++w) any |= votes[w] != 0;
        return any;
    };
    // What is written of a row: its maximum and sum of weights (or its lse), and 32 of its dims.
    const auto pair_of_row = [&] { return (t.q0 + tok) * static_cast<int64_t>(a.n_heads) + head; };
    const auto write_row = [&]() __attribute__((always_inline)) {
        l += other_half(l);
        if (row >= t.rows || half != 0) return;
        const int64_t pair = pair_of_row();
        if (splits > 1) {
            const Partials p = partials(a.work, a.T * a.n_heads, splits, part, D);
            p.ml[2 * pair] = M;
            p.ml[2 * pair + 1] = l;
        } else if (a.lse) {
            a.lse[pair] = log_sum(M, l);
        }
    };
    const auto write_dims = [&](int d, const floatx16_t &o) __attribute__((always_inline)) {
        // (splits without keys: their sum is 0, the weighted sums are not read)
        if (row >= t.rows || (splits > 1 && n_iter == 0)) return;
        const Partials p = partials(a.work, a.T * a.n_heads, splits, part, D);
        const int64_t token = t.q0 + tok;
        const int64_t base = token * a.ldy + static_cast<int64_t>(head) * D;
        const float inv = inverse_sum(l);
        const bool wide = wide_rows(a);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int col = 32 * d + 8 * g + 4 * half;
            if (col >= D) continue;
            floatx4_t v = {o[4 * g], o[4 * g + 1], o[4 * g + 2], o[4 * g + 3]};
            if (splits > 1)
                *reinterpret_cast<floatx4_t *>(p.o + pair_of_row() * D + col) = v;
            else
                store_out4(a.y, base + col, v * inv, a.out_f32, wide);
        }
    };

    if constexpr (ANY) {
        for (int d0 = 0; 32 * d0 < D; d0 += kAnyDims) {
            M = kNoMax;
            l = 0.0f;
#pragma unroll
            for (int d = 0; d < kAnyDims; ++d) o[d] = floatx16_t(0.0f);
            for (int i = 0; i < n_iter; ++i) {
                look_up(i);
                locate(i, newest);
                fetch(head_k, newest, k_col, sk0, L::kKeyBlock);
                fetch(head_v, newest, v_col, sv0, L::kValueBlock);
                tile_barrier();
                scores(sk0);
                bool rose;
                const float f = raise(i, &rose);
                if (rose) {
#pragma unroll
                    for (int d = 0; d < kAnyDims; ++d) o[d] *= f;
                }
                weights();
                weigh_any(sv0, d0);
                tile_barrier();
            }
            if (d0 == 0)
                write_row();
            else
                l += other_half(l);
#pragma unroll
            for (int d = 0; d < kAnyDims; ++d) write_dims(d0 + d, o[d]);
        }
        return;
    }
    if (n_iter > 0) {
        look_up(0);
        locate(0, newest);
        fetch(head_k, newest, k_col, sk0, L::kKeyBlock);
        phase_fence();
        look_up(tile_at(1));
        send(-1, sk1, sv0);
        // (every wave's keys 0 have landed; the rest has time until the first iteration)
        phase_fence();
        __builtin_amdgcn_s_waitcnt(wait_vm<2 * kLoads>());
        __builtin_amdgcn_s_barrier();
        phase_fence();
        scores(sk0);
        bool rose;
        raise(0, &rose);
        weights();
        tile_barrier();
        int it = 0;
        if (n_iter > 2) {
            do {
                step(it, sk0, sv0, sk1, sv1);
                step(it + 1, sk1, sv1, sk0, sv0);
                it += 2;
            } while (it + 2 < n_iter);
        }
        if (it + 1 < n_iter) {
            step(it, sk0, sv0, sk1, sv1);
            ++it;
        }
        weigh(it & 1 ? sv1 : sv0);

        float odd[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) odd[i % 4] = fmaf(o[d][i], 0.0f, odd[i % 4]);
        const bool again = odd[0] + odd[1] + (odd[2] + odd[3]) != 0.0f || is_far();
        if (__builtin_expect(block_any(again), 0)) {
            const Args args = args_again();
            prefill_tile<DP, KT, PAGES, true>(args.a, args.c, args.splits, sk0, sk0, sv0, sv0,
                                              votes);
            return;
        }
    }

    write_row();
#pragma unroll
    for (int d = 0; d < DT; ++d) write_dims(d, o[d]);
}

template <int DP, int KT, int PAGES>
__global__ void __launch_bounds__(kWaves * 64)
__attribute__((amdgpu_waves_per_eu(2, 2))) attn_prefill_kernel(Args args) {
    using L = TileLayout<DP>;
    // (arrays of their own: the compiler then sees that a direct load on its way into one does not
    // touch the others, and does not wait for it before it reads them)
    __shared__ __attribute__((aligned(16))) uint16_t sk0[KT / L::kSpan * L::kKeyBlock];
    __shared__ __attribute__((aligned(16))) uint16_t sk1[KT / L::kSpan * L::kKeyBlock];
    __shared__ __attribute__((aligned(16))) uint16_t sv0[KT / L::kSpan * L::kValueBlock];
    __shared__ __attribute__((aligned(16))) uint16_t sv1[KT / L::kSpan * L::kValueBlock];
    __shared__ int votes[kWaves];
    prefill_tile<DP, KT, PAGES, false>(args.a, args.c, args.splits, sk0, sk1, sv0, sv1, votes);
}

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

template <int DP, int KT>
void launch(const Plan &p, const AttnArgs &a, const KvView &c, hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(p.tiles * c.n_kv * p.splits)), block(kWaves * 64);
    const Args args = {a, c, p.splits};
    if (c.page_mask >= KT - 1)
        hipLaunchKernelGGL((attn_prefill_kernel<DP, KT, kTilePages>), grid, block, 0, stream, args);
    else if (c.page_mask >= 7)
        hipLaunchKernelGGL((attn_prefill_kernel<DP, KT, kSpanPages>), grid, block, 0, stream, args);
    else
        hipLaunchKernelGGL((attn_prefill_kernel<DP, KT, kAnyPages>), grid, block, 0, stream, args);
}

}  // namespace

bool attn_prefill_supported(int64_t T, int n_heads, const KvView &c, int window, int sinks) {
    // (so T G, which the kernel rounds up to tiles, stays below 2^31 too)
    const Plan p = plan_of(T, n_heads, c, window, sinks);
    return p.tiles * c.n_kv * p.splits <= static_cast<int64_t>(kMaxThreads) / (kWaves * 64);
}

size_t attn_prefill_work_bytes(int64_t T, int n_heads, const KvView &c, int window, int sinks) {
    const Plan p = plan_of(T, n_heads, c, window, sinks);
    if (p.splits == 1) return 0;
    return sizeof(float) * p.splits * T * n_heads * (c.head_dim + 2);
}

hipError_t launch_attn_prefill(const AttnArgs &a, const KvView &c, hipStream_t stream) {
    const Plan p = plan_of(a.T, a.n_heads, c, a.window, a.sinks);
    if (c.head_dim <= 64)
        launch<64, 64>(p, a, c, stream);
    else if (c.head_dim <= 128)
        launch<128, 64>(p, a, c, stream);
    else
        launch<256, 32>(p, a, c, stream);
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

}  // namespace w4
