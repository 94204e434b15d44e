// attn_narrow.h -- the body shared by the attention kernels of few rows (single tokens, and units of
// up to 16 rows of a batch): rows of one key-value head over a range of its keys, bound by reading
// them: 1 flop per byte and row (1.5 with the weights in two parts, below).
//
// The rows (query heads that share the key-value head, of one token or of several) are the columns of
// one 16-wide matrix-core tile, so that a key is read once for up to 16 of them.
//
//   S^T[key][row] = K Q^T    on v_mfma_f32_16x16x32_bf16; a lane's 16 bytes of a key row are the
//                            operand as they come from memory
//   O^T[d][row]  += V^T P^T  V through LDS and its transposed read; P^T is, register for register,
//                            the operand: V's rows follow the key order the first product left
// P enters the second product as the sum of two bf16 values (16 bits of each weight): the matrix
// cores have time to spare here.
//
// Tiles are of 32 keys. A wave goes through its tiles on its own (no barrier in the loop, the next
// tile's loads in flight); what it leaves are weighted sums in registers.
#pragma once

#include <type_traits>

#include "attn_device.h"

namespace w4 {

constexpr int kNarrowTile = 32;  // keys of a tile
constexpr int kNarrowWaves = 4;
constexpr int kNarrowRows = 16;  // rows of a workgroup
// Values that are not finite, counted over a tile's keys: bf16 64 for minus infinity, 4096 for NaN.
constexpr uint32_t kMinus = 0x4280u, kNan = 0x4580u;

// Elements from row to row of a value tile: a transposed read takes 32 bytes of 4 consecutive rows at
// once, which the gap puts 32 bytes further each in the 64 banks.
template <int DP>
constexpr int kNarrowRow = DP + 16;
// A wave's LDS: the value tile, 32 rows of bf16; after the loop its sums, 16 rows of fp32.
template <int DP>
constexpr int kNarrowElements = kNarrowTile * kNarrowRow<DP>;

// Every STEPth tile of a unit from t0 on, below t1:
//   unit.head, unit.table
//   unit.query()      the query of the lane's row (of one that exists where there is none)
//   unit.start(t)     first key of a tile, a multiple of 32
//   unit.sees(p)      does the lane's row see key p;  unit.visible(p): does any row of the unit
//   unit.safe_key(s)  a visible key, among the 16 from s on if any is
// my_v: the wave's LDS. Leaves in lane (g, r) = (lane / 16, lane % 16) dims 16 i + 4 g .. + 3 of row r's
// weighted sums in o[i], the row's maximum (log2 units) in *row_max, and sum of weights in *row_sum.
//
// PAGE16: pages of 16 slots and more, so that 16 aligned keys lie in one page, whose address is
// looked up a tile ahead, once for all lanes. (Else each row looks up its own: 32 x 8192 keys,
// 16 heads over 4 of 256, window 1024, 62 us for 33; one of 4097, 28 over 4 of 128, 11.8 for 11.0.)
template <int DP, bool PAGE16, int STEP, class Unit>
__device__ __forceinline__ void narrow_wave(const AttnArgs &a, const KvView &c, const Unit &unit,
                                            int t0, int t1, uint16_t *my_v, floatx4_t (&o)[DP / 16],
                                            float *row_max, float *row_sum) {
    constexpr int KS = DP / 32;      // steps of the first product
    constexpr int DT = DP / 16;      // tiles of the second
    constexpr int kChunks = DP / 8;  // 16-byte chunks of a row
    constexpr int kVRows = 64 / kChunks;       // rows a wave's load instruction covers
    constexpr int kVLoads = kNarrowTile / kVRows;
    constexpr int kRow = kNarrowRow<DP>;
    const int D = c.head_dim, lane = threadIdx.x & 63;
    const int r = lane & 15, g = lane >> 4;  // column (row of the unit), group of 16 lanes
    const float cs = a.scale * kLog2e;

    bf16x8_t qf[KS];
    {
        const uint16_t *src = unit.query();
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int d = 32 * s + 8 * g;
            const uintx4_t v = *reinterpret_cast<const uintx4_t *>(src + min(d, D - 8));
            qf[s] = __builtin_bit_cast(bf16x8_t, d < D ? v : uintx4_t{0, 0, 0, 0});
        }
    }

    const int64_t head_off = static_cast<int64_t>(unit.head) * c.head_stride;
    // 16 keys as they are read: the page offset of a visible key among them (of another one if
    // there is none), and that key. Keys that are not visible are read from it: finite values,
    // whose weight is 0.
    struct Span {
        int start, safe;
        int64_t page;
    };
    const auto page_offset = [&](int page) {
        page = page < 0 ? 0 : (page >= c.n_pages ? c.n_pages - 1 : page);
        return static_cast<int64_t>(page) * c.page_stride + head_off;
    };
    // Eight elements from element `col` on of row i (0..15) of a span. (The page's address is
    // uniform where the span lies in one page: a scalar base and a 32-bit offset in bytes.)
    const auto load_row = [&](const uint16_t *kv, const Span &sp, int i, int col) {
        const int p = sp.start + i;
        const int from = unit.visible(p) ? p : sp.safe;
        const int64_t page =
            PAGE16 ? sp.page : page_offset(read_const(unit.table + (from >> c.page_shift)));
        const uint32_t off = (from & c.page_mask) * c.slot_stride + col;
        return *reinterpret_cast<const uintx4_t *>(
            reinterpret_cast<const char *>(kv + page) + 2u * off);
    };

    // The next tile to be fetched, and the one after it: their spans' keys, and the table
    // entries on their way.
    Span next[2];
    int entry[2] = {0, 0};
    const auto look_up = [&](int t) {
        if (!PAGE16) return;
#pragma unroll
        for (int u = 0; u < 2; ++u)
            entry[u] = read_const(unit.table + (unit.safe_key(unit.start(t) + 16 * u) >> c.page_shift));
    };
    const auto locate = [&](int t) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            next[u].start = unit.start(t) + 16 * u;
            next[u].safe = unit.safe_key(next[u].start);
            next[u].page = page_offset(entry[u]);
        }
    };
    // Dims past D repeat the row's last chunk: they meet zeros of q, or outputs that are not
    // kept.
    const int v_row = lane / kChunks, v_chunk = min(8 * (lane % kChunks), D - 8);
    uintx4_t rk[2][KS], rv[kVLoads];
    const auto fetch_k = [&] {
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int s = 0; s < KS; ++s)
                rk[u][s] = load_row(c.k, next[u], r, min(32 * s + 8 * g, D - 8));
    };
    const auto fetch_v = [&] {
#pragma unroll
        for (int i = 0; i < kVLoads; ++i)
            rv[i] = load_row(c.v, next[i * kVRows / 16], i * kVRows % 16 + v_row, v_chunk);
    };

#pragma unroll
    for (int i = 0; i < DT; ++i) o[i] = floatx4_t(0.0f);
    float M = kNoMax, l = 0.0f;

    // One tile; with MORE, the wave's next tile is fetched on the way, and the one after that
    // looked up; with ANY, values may be infinite or NaN.
    const auto step = [&](auto more, auto any, int t) {
        constexpr bool MORE = decltype(more)::value, ANY = decltype(any)::value;
        const int k0 = unit.start(t), after = min(t + 2 * STEP, t1 - 1);
        if constexpr (MORE) look_up(after);
        floatx4_t s[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            s[u] = floatx4_t(0.0f);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
                s[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8_t, rk[u][ks]), qf[ks], s[u], 0, 0, 0);
        }
        phase_fence();
        if constexpr (MORE) fetch_k();
        phase_fence();
#pragma unroll
        for (int i = 0; i < kVLoads; ++i) {
            uintx4_t kind, *to = reinterpret_cast<uintx4_t *>(
                               &my_v[(i * kVRows + v_row) * kRow + 8 * (lane % kChunks)]);
            *to = ANY ? split_values<kMinus, kNan>(rv[i], &kind) : rv[i];
        }
        phase_fence();
        __builtin_amdgcn_wave_barrier();
        if constexpr (MORE) {
            fetch_v();
            locate(after);
        }
        phase_fence();

        float mx = -INFINITY;
        bool ok[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ok[u][i] = unit.sees(k0 + 16 * u + 4 * g + i);
                s[u][i] = s[u][i] * cs;
                mx = ok[u][i] ? fmaxf(mx, s[u][i]) : mx;
            }
        mx = fmaxf(mx, __shfl_xor(mx, 16, kWave));
        mx = fmaxf(mx, __shfl_xor(mx, 32, kWave));
        if (__any(mx > M + kScoreSlack)) {
            const float M2 = fmaxf(M, mx);
            const float f = __builtin_amdgcn_exp2f(M - M2);
            M = M2;
            l *= f;
#pragma unroll
            for (int d = 0; d < DT; ++d) o[d] *= f;
        }
        uintx4_t hi, lo;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const float p0 = ok[u][i] ? __builtin_amdgcn_exp2f(s[u][i] - M) : 0.0f;
                const float p1 = ok[u][i + 1] ? __builtin_amdgcn_exp2f(s[u][i + 1] - M) : 0.0f;
                l += p0 + p1;
                const uint32_t w = pack_bf16(p0, p1);
                hi[2 * u + i / 2] = w;
                lo[2 * u + i / 2] = pack_bf16(p0 - __uint_as_float(w << 16),
                                              p1 - __uint_as_float(w & 0xFFFF0000u));
            }
        // slots 8 g + 0..3 are keys 4 g + 0..3, slots 8 g + 4..7 keys 16 + 4 g + 0..3
        const uint16_t *vp = &my_v[(4 * g + r / 4) * kRow + 4 * (r & 3)];
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            const uintx2_t v0 = lds_read_transposed(vp + 16 * d);
            const uintx2_t v1 = lds_read_transposed(vp + 16 * kRow + 16 * d);
            const uintx4_t vv = {v0[0], v0[1], v1[0], v1[1]};
            const bf16x8_t vf = __builtin_bit_cast(bf16x8_t, vv);
            o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, __builtin_bit_cast(bf16x8_t, hi),
                                                           o[d], 0, 0, 0);
            o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, __builtin_bit_cast(bf16x8_t, lo),
                                                           o[d], 0, 0, 0);
        }
        asm volatile("" ::: "memory");
        __builtin_amdgcn_wave_barrier();
        if constexpr (ANY) {
            // the values that are not finite, counted by kind for the keys that are seen
            uintx4_t seen;  // bf16 ones where weights are
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int i = 0; i < 4; i += 2)
                    seen[2 * u + i / 2] =
                        (ok[u][i] && s[u][i] != -INFINITY ? 0x3F80u : 0) |
                        (ok[u][i + 1] && s[u][i + 1] != -INFINITY ? 0x3F800000u : 0);
#pragma unroll
            for (int i = 0; i < kVLoads; ++i) {
                uintx4_t kind;
                split_values<kMinus, kNan>(rv[i], &kind);
                *reinterpret_cast<uintx4_t *>(
                    &my_v[(i * kVRows + v_row) * kRow + 8 * (lane % kChunks)]) = kind;
            }
            asm volatile("" ::: "memory");
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int d = 0; d < DT; ++d) {
                const uintx2_t v0 = lds_read_transposed(vp + 16 * d);
                const uintx2_t v1 = lds_read_transposed(vp + 16 * kRow + 16 * d);
                const uintx4_t vv = {v0[0], v0[1], v1[0], v1[1]};
                const floatx4_t n = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8_t, vv), __builtin_bit_cast(bf16x8_t, seen),
                    floatx4_t(0.0f), 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    o[d][i] = add_kinds<64, 4096>(o[d][i], static_cast<int>(n[i]));
            }
            asm volatile("" ::: "memory");
            __builtin_amdgcn_wave_barrier();
        }
    };
    int t = t0;
    if (t < t1) {
        look_up(t);
        locate(t);
        fetch_k();
        fetch_v();
        look_up(min(t + STEP, t1 - 1));
        locate(min(t + STEP, t1 - 1));
        if (t + STEP < t1) {
            do {
                step(std::true_type{}, std::false_type{}, t);
                t += STEP;
            } while (t + STEP < t1);
        }
        step(std::false_type{}, std::false_type{}, t);
    }
    // An infinite value times the lower part of its weight, or a weight of 0 (where the row
    // that stands in for a hidden one holds it), is not that infinity. So a wave whose sums are
    // not finite goes through its tiles again, its values split into finite ones and others.
    float odd[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) odd[i] = fmaf(o[d][i], 0.0f, odd[i]);
    if (__builtin_expect(__any(odd[0] + odd[1] + (odd[2] + odd[3]) != 0.0f), 0)) {
        M = kNoMax;
        l = 0.0f;
#pragma unroll
        for (int d = 0; d < DT; ++d) o[d] = floatx4_t(0.0f);
        for (t = t0; t < t1; t += STEP) {
            look_up(t);
            locate(t);
            fetch_k();
            fetch_v();
            step(std::false_type{}, std::true_type{}, t);
        }
    }

    *row_max = M;
    *row_sum = l + __shfl_xor(l, 16, kWave);
    *row_sum += __shfl_xor(*row_sum, 32, kWave);
}

}  // namespace w4
