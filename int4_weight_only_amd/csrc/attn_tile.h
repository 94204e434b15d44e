// attn_tile.h -- the body shared by the attention kernels of many rows (prompts, cross attention,
// shared prefixes): 128 rows of one key-value head over a share of the keys, on the matrix cores.
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
// that one can multiply while the other turns scores into weights.
//
// Rows says which rows these are, which keys they see and where their results go: of one sequence over
// its keys (attn_prefill.hip), or of many over keys that lie by one or two page tables (attn_units.hip).
#pragma once

#include <type_traits>

#include "attn_device.h"

namespace w4 {

constexpr int kTileWaves = 4, kTileRows = 32 * kTileWaves;
constexpr float kFar = 1 << 20;

// What a workgroup computes. Rows::find fills it; every wave of the workgroup finds the same but for
// what belongs to a lane's row and a wave's rows.
struct TileRows {
    int hk;           // key-value head
    int part, part_end, parts;  // the share of the key tiles: from part to part_end of `parts`
    // of the lane's row, or of a row that exists where there is none: token row, query head, position
    int token, head, pos;
    bool live;
    int tile_first, tile_last;  // oldest and newest position of the workgroup's rows
    int first, last;            // of the wave's rows
    const int32_t *table;       // pages of the keys
    // Two tables (Rows::kTwoTables): keys before `cut` have their pages in first_table. Seen are the
    // keys of the first table only, of the second only, or of both.
    const int32_t *first_table;
    int cut;
    bool from_cut, to_cut;
    // (of Rows that cut units into pieces: rows of a prefix; rows written as they are; the first of the
    // unit's pieces, how many there are, and where the piece after this one begins)
    bool of_prefix, direct, first_piece;
    int pieces, next;
};

// The key tiles that the rows of a workgroup see: those of the sinks, then those from `lo` on. Where
// the second table begins inside a tile, that tile comes twice, once with the keys of each table.
template <int KT, bool TABLES>
struct KeyTiles {
    int n, n_sink, lo_tile;
    int from, cut_tiles, twice;
    __device__ __forceinline__ KeyTiles(const TileRows &t, int lo, int sinks_end) {
        int last = t.tile_last, begin = 0;
        from = cut_tiles = twice = 0;
        if constexpr (TABLES) {
            begin = t.from_cut ? t.cut : 0;
            last = t.to_cut ? min(last, t.cut - 1) : last;
            twice = t.cut % KT != 0;
            cut_tiles = t.cut / KT + twice;
            from = number(begin, t.cut);
        }
        if constexpr (TABLES) {
            const int early = min(min(sinks_end, lo), last + 1);
            n_sink = early > begin ? number(early - 1, t.cut) + 1 - from : 0;
            lo_tile = max(number(max(lo, begin), t.cut), from + n_sink);
            n = n_sink + (last < begin ? 0 : max(number(last, t.cut) + 1 - lo_tile, 0));
        } else {
            n_sink = (min(sinks_end, lo) + KT - 1) / KT;
            lo_tile = max(lo / KT, n_sink);
            n = last < 0 ? 0 : n_sink + last / KT + 1 - lo_tile;
        }
    }
    // Where share `part` of `parts` begins. (As many shares as tiles: a plan's own numbers.)
    __device__ __forceinline__ int share(int part, int parts) const {
        if (TABLES && parts == n) return part;
        return static_cast<int>(static_cast<int64_t>(n) * part / parts);
    }
    __device__ __forceinline__ int number(int p, int cut) const {
        return p / KT + (p < cut ? 0 : twice);
    }
    __device__ __forceinline__ int tile(int it) const {
        return it < n_sink ? from + it : lo_tile + it - n_sink;
    }
    __device__ __forceinline__ bool first_table(int it) const {
        return TABLES && tile(it) < cut_tiles;
    }
    __device__ __forceinline__ int key(int it) const {  // first key
        const int i = tile(it);
        return (TABLES && i >= cut_tiles ? i - twice : i) * KT;
    }
};

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

// The kernel's arguments, read once more: its only parameter is at the start of their segment.
template <class Args>
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

// One tile of rows over one share of its keys, as Rows says (see TileRows).
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
// Returns what find left in `next`.
template <class Rows, int DP, int KT, int PAGES, bool ANY>
__device__ __forceinline__ int attn_tile(const typename Rows::Args &args,
                                          const typename Rows::State &state, uint16_t *sk0,
                                         uint16_t *sk1, uint16_t *sv0, uint16_t *sv1, int *votes) {
    constexpr bool TABLES = Rows::kTwoTables;
    const AttnArgs &a = args.a;
    const KvView &c = args.c;
    constexpr int NW = kTileWaves;
    constexpr int kChunks = DP / 8;                    // 16-byte chunks of a row
    constexpr int kSpan = 64 / kChunks;                // rows a wave stages in one instruction
    constexpr int kLoads = KT / (NW * kSpan);          // instructions a wave stages a tile with
    static_assert(kLoads * NW * kSpan == KT, "every wave stages the same number of rows");
    using L = TileLayout<DP>;
    constexpr int DT = DP / 32, KS = DP / 16, SUB = KT / 32;
    // (TABLES: called in a loop over units, out of which nothing that takes registers is to move)
    const int tid = ANY || TABLES ? unknown(threadIdx.x) : threadIdx.x;
    const int lane = tid & 63;
    const int wid = uniform(tid >> 6);
    const int D = c.head_dim;
    const int half = lane >> 5;
    TileRows t;
    t.next = 0;
    if (!Rows::template find<DP, KT>(args, state, wid, lane, sk0, sv0, &t)) return t.next;
    const int hk = t.hk, pos = t.pos, tile_last = t.tile_last;

    // Key tiles: those of the sinks, then those from the oldest key in a row's window on; of them
    // this share's.
    const int lo = a.window > 0 ? max(t.tile_first - a.window + 1, 0) : 0;
    const int sinks_end = a.window > 0 ? a.sinks : 0;
    const KeyTiles<KT, TABLES> tiles(t, lo, sinks_end);
    const int it0 = tiles.share(t.part, t.parts);
    const int n_iter = tiles.share(t.part_end, t.parts) - it0;
    const auto tile_key = [&](int it) { return tiles.key(it + it0); };
    // With two tables: where the keys of a tile end that its table holds, and where they begin.
    const auto tile_end = [&](int it) {
        return !TABLES || !tiles.first_table(it + it0) ? tile_last : min(tile_last, t.cut - 1);
    };
    const auto tile_begin = [&](int it) {
        return !TABLES || tiles.first_table(it + it0) ? 0 : t.cut;
    };

    // Q^T: lane holds dims 16 s + 8 half .. + 7 of its row
    bf16x8_t qf[KS];
    {
        const uint16_t *src = a.q + t.token * a.ldq + static_cast<int64_t>(t.head) * D;
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
    const uint16_t *head_k = c.k + static_cast<int64_t>(hk) * c.head_stride;
    const uint16_t *head_v = c.v + static_cast<int64_t>(hk) * c.head_stride;
    const auto span_at = [&](int i) { return (i * NW + wid) * kSpan; };
    // (of a tile whose table holds the keys begin .. end)
    const auto all_seen = [&](int k0, int begin, int end) {  // each key by some row of the block
        return (!TABLES | (k0 >= begin)) & (k0 + KT - 1 <= end) &
               ((k0 >= lo) | (k0 + KT - 1 < sinks_end));
    };
    const auto visible = [&](int p, int begin, int end) {
        return (!TABLES | (p >= begin)) & (p <= end) & ((p >= lo) | (p < sinks_end));
    };
    // a key that is seen, among the n from s0 on if any is
    const auto safe_of = [&](int s0, int n, int begin, int end) {
        if constexpr (TABLES) {
            const int p = min(max(s0, begin), end);
            if (p < sinks_end || p >= lo) return p;
            return lo <= end ? lo : max(min(sinks_end - 1, end), begin);
        }
        if (s0 > end) return end;
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
        const int k0 = tile_key(it), begin = tile_begin(it), end = tile_end(it);
        const int32_t *table = TABLES && tiles.first_table(it + it0) ? t.first_table : t.table;
        if constexpr (PAGES == kTilePages) {
            // (the page of the tile's first key, which is seen or a later one is)
            entry[0] = read_const(table + (k0 >> c.page_shift));
        } else if constexpr (PAGES == kSpanPages) {
            const bool all = all_seen(k0, begin, end);
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int s0 = k0 + span_at(i);
                entry[i] = read_const(
                    table + ((all ? s0 : safe_of(s0, kSpan, begin, end)) >> c.page_shift));
            }
        }
    };
    const auto locate = [&](int it, Where &w) {
        const int k0 = tile_key(it), begin = tile_begin(it), end = tile_end(it);
        if constexpr (PAGES == kTilePages) {
            w.base[0] = page_offset(entry[0]) +
                        static_cast<int64_t>((k0 & c.page_mask) * c.slot_stride);
            const int first = TABLES ? max(k0, begin) : k0;
            const int safe = first < sinks_end ? first : max(first, lo);
            const uint32_t other = (safe - k0) * c.slot_stride;
#pragma unroll
            for (int i = 0; i < kLoads; ++i)
                // (uniform, to be added here: else each sum has a register of its own throughout)
                w.off[i] = visible(uniform(k0 + span_at(i)) + my_row, begin, end) ? seen_off(i) : other;
        } else {
            const bool all = all_seen(k0, begin, end);
            const int32_t *table = TABLES && tiles.first_table(it + it0) ? t.first_table : t.table;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int s0 = k0 + span_at(i), p = s0 + my_row;
                const int safe = all ? s0 : safe_of(s0, kSpan, begin, end);
                const bool vis = all | visible(p, begin, end);
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
        const int begin = tile_begin(it), end = tile_end(it);
        const bool whole = k0 + KT - 1 <= (TABLES ? min(t.first, end) : t.first) &&
                           (!TABLES || k0 >= begin) &&
                           (a.window == 0 || k0 > t.last - a.window || k0 + KT - 1 < a.sinks);
        if (!whole) {
            // key i of the lane's is at place 32 u + 8 (i / 4) + i % 4 of those from k0 + 4 half on
            const int base = k0 + 4 * half;
            const int newest_at = (TABLES ? min(pos, end) : pos) - base, before_at = before - base;
            const int sinks_at = sinks_end - base, begin_at = begin - base;
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int at = 32 * u + 8 * (i / 4) + i % 4;
                    const bool ok = (at <= newest_at) & (!TABLES | (at >= begin_at)) &
                                    ((at > before_at) | (at < sinks_at));
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
        *rose = __any(mx > M + kScoreSlack);
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
    // What is written of a row: its maximum and sum of weights (or its lse) where `lead`, and N times
    // 32 of its dims, from 32 d0 on.
    const auto write = [&](bool lead, int d0, auto n, const floatx16_t *o)
                           __attribute__((always_inline)) {
        constexpr int N = decltype(n)::value;
        l += other_half(l);
        if (!t.live) return;
        lead &= half == 0;
        if (Rows::is_partial(args, t)) {
            // (shares without keys: their sum is 0, the weighted sums are not read)
            float *to = Rows::write_sums(args, state, t, M, l, lead) + 4 * half;
            if (n_iter == 0) return;
#pragma unroll
            for (int d = 0; d < N; ++d)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int col = 32 * (d0 + d) + 8 * g;  // (D is a multiple of 8)
                    if (col < D)
                        *reinterpret_cast<floatx4_t *>(to + col) = floatx4_t{
                            o[d][4 * g], o[d][4 * g + 1], o[d][4 * g + 2], o[d][4 * g + 3]};
                }
            return;
        }
        if constexpr (TABLES) {
            if (lead) Rows::write_record(args, state, t);
        }
        if (lead && a.lse) a.lse[t.token * static_cast<int64_t>(a.n_heads) + t.head] = log_sum(M, l);
        const int64_t base = t.token * a.ldy + static_cast<int64_t>(t.head) * D + 4 * half;
        const float inv = inverse_sum(l);
        const bool wide = wide_rows(a);
#pragma unroll
        for (int d = 0; d < N; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int col = 32 * (d0 + d) + 8 * g;
                if (col >= D) continue;
                const floatx4_t v = {o[d][4 * g], o[d][4 * g + 1], o[d][4 * g + 2], o[d][4 * g + 3]};
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
            write(d0 == 0, d0, std::integral_constant<int, kAnyDims>{}, o);
        }
        return t.next;
    }
    bool again = false;
    // (with few rows in a unit, waves without any only move keys and values, at the same barriers: a loop
    // of its own, as conditions inside the other one spilled its registers. 24 sequences of 5 tokens, 16
    // heads over 4 of 256, 20 rows each: 45 us, all waves multiplying 50.)
    const bool idle = TABLES && !__any(t.live);
    if (idle && n_iter > 0) {
        look_up(0);
        locate(0, newest);
        fetch(head_k, newest, k_col, sk0, L::kKeyBlock);
        phase_fence();
        look_up(tile_at(1));
        send(-1, sk1, sv0);
        phase_fence();
        __builtin_amdgcn_s_waitcnt(wait_vm<2 * kLoads>());
        __builtin_amdgcn_s_barrier();
        phase_fence();
        tile_barrier();
        for (int it = 0; it + 1 < n_iter; ++it) {
            if (it & 1)
                send(it, sk1, sv0);
            else
                send(it, sk0, sv1);
            tile_barrier();
        }
    }
    if (!idle && n_iter > 0) {
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
        again = odd[0] + odd[1] + (odd[2] + odd[3]) != 0.0f || is_far();
    }
    if (n_iter > 0 && __builtin_expect(block_any(again), 0)) {
        attn_tile<Rows, DP, KT, PAGES, true>(args_again<typename Rows::Args>(), state, sk0, sk0, sv0,
                                             sv0, votes);
        return t.next;
    }

    if (!idle) write(true, 0, std::integral_constant<int, DT>{}, o);
    return t.next;
}

// PER_CU: workgroups on a compute unit.
template <class Rows, int DP, int KT, int PAGES, int PER_CU>
__global__ void __launch_bounds__(kTileWaves * 64)
__attribute__((amdgpu_waves_per_eu(PER_CU, PER_CU))) attn_tile_kernel(typename Rows::Args args) {
    using L = TileLayout<DP>;
    // (arrays of their own: the compiler then sees that a direct load on its way into one does not
    // touch the others, and does not wait for it before it reads them)
    __shared__ __attribute__((aligned(16))) uint16_t sk0[KT / L::kSpan * L::kKeyBlock];
    __shared__ __attribute__((aligned(16))) uint16_t sk1[KT / L::kSpan * L::kKeyBlock];
    __shared__ __attribute__((aligned(16))) uint16_t sv0[KT / L::kSpan * L::kValueBlock];
    __shared__ __attribute__((aligned(16))) uint16_t sv1[KT / L::kSpan * L::kValueBlock];
    __shared__ int votes[kTileWaves];
    attn_tile<Rows, DP, KT, PAGES, false>(args, {}, sk0, sk1, sv0, sv1, votes);
}

// Keys of a tile, by head size.
constexpr int tile_keys(int head_dim) { return head_dim > 128 ? 32 : 64; }

template <class Rows, int DP, int PER_CU>
void launch_tiles(const typename Rows::Args &args, int64_t blocks, hipStream_t stream) {
    constexpr int KT = tile_keys(DP);
    const auto kernel = args.c.page_mask >= KT - 1 ? attn_tile_kernel<Rows, DP, KT, kTilePages, PER_CU>
                        : args.c.page_mask >= 7 ? attn_tile_kernel<Rows, DP, KT, kSpanPages, PER_CU>
                                                : attn_tile_kernel<Rows, DP, KT, kAnyPages, PER_CU>;
    hipLaunchKernelGGL(kernel, dim3(static_cast<unsigned>(blocks)), dim3(kTileWaves * 64), 0, stream,
                       args);
}
template <class Rows>
void launch_tiles(const typename Rows::Args &args, int64_t blocks, hipStream_t stream) {
    // At 64 dims registers do for three workgroups on a compute unit (those of the second pass are
    // spilled: with one infinity in the values 3 x 4096, 28 heads over 4, 523 us for 467, 8 x 1024, 20
    // heads, 104 for 81): prompts of 3 x 4096 179 to 186 us for 194 to 199; 8 x 448 rows over 1500 states,
    // 20 heads, 49 for 55, as 580 workgroups then run at once. Where two on each hold all, three only
    // share them out unevenly: 4 x 200 after 3000 keys 28.3 us for 27.3.
    // Pages under 8 slots, whose rows each have an address, take longer side by side: where most rows see
    // all keys before them, three gain with more than four for each only (pages of 4, 8 heads, us for
    // three / two: one prompt of 11000, 688 workgroups, 230 / 200, of 12500, 784, 266 / 228, of 16000,
    // 1008, 350 / 382; 8 x 1024, 20 heads, 1280, 43.5 / 47.7; window 4096, one of 9000, 568, 105 / 98),
    // within windows as elsewhere (2 x 5000, 576, window 512, 26.8 / 32.9; one of 9000, window 1024, 38.7
    // / 46.0).
    const bool by_rows = args.c.page_mask < 7 && !(args.a.window > 0 && args.a.window <= 1024);
    if (args.c.head_dim <= 64 && blocks > (by_rows ? 4 : 2) * int64_t{device_cu_count()})
        launch_tiles<Rows, 64, 3>(args, blocks, stream);
    else if (args.c.head_dim <= 64)
        launch_tiles<Rows, 64, 2>(args, blocks, stream);
    else if (args.c.head_dim <= 128)
        launch_tiles<Rows, 128, 2>(args, blocks, stream);
    else
        launch_tiles<Rows, 256, 2>(args, blocks, stream);
}

}  // namespace w4
