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
// rarely rescaled.
#include "attn_device.h"

namespace w4 {

namespace {

constexpr int kSlack = 8;

struct Tile {  // the rows of a block
    int seq, row0, rows;      // rows of the sequence's G * nq stacked rows; rows = those in all
    int q0, pos0;             // token row of stacked row 0, its position
};

// The tile'th tile of BM rows, counted through the sequences in order, the last rows of a sequence
// (which see the most keys) first. Every lane of every wave takes part.
template <int BM>
__device__ __forceinline__ bool find_tile(const KvView &c, const int32_t *q_start, int64_t T,
                                          int G, int tile, Tile *out) {
    const int lane = threadIdx.x & (kWave - 1);
    int before = 0;
    for (int base = 0; base < c.n_seqs; base += kWave) {
        const int b = base + lane;
        int begin = 0, end = 0;
        if (b < c.n_seqs) {
            begin = max(read_const(q_start + b), 0);
            end = min(read_const(q_start + b + 1), static_cast<int>(T));
        }
        const int nq = max(end - begin, 0);
        const int mine = static_cast<int>((static_cast<int64_t>(nq) * G + BM - 1) / BM);
        const int sum = wave_scan_dpp(mine);
        const uint64_t hit = __ballot(before + sum > tile);
        if (hit) {
            const int w = __builtin_ctzll(hit);
            const int tokens = __builtin_amdgcn_readlane(nq, w);
            const int tiles = __builtin_amdgcn_readlane(mine, w);
            const int left = tile - before - (__builtin_amdgcn_readlane(sum, w) - tiles);
            out->seq = base + w;
            out->rows = tokens * G;
            out->row0 = (tiles - 1 - left) * BM;
            out->q0 = __builtin_amdgcn_readlane(begin, w);
            out->pos0 = kv_length(c, base + w) - tokens;
            return true;
        }
        before += __builtin_amdgcn_readlane(sum, kWave - 1);
    }
    return false;
}

template <int DP, int NW, int KT>
__global__ void __launch_bounds__(NW * 64)
__attribute__((amdgpu_waves_per_eu(2))) attn_prefill_kernel(AttnArgs a, KvView c, int n_tiles) {
    constexpr int BM = NW * 32;
    constexpr int kChunks = DP / 8;
    constexpr int kThreads = NW * 64;
    constexpr int kLoads = KT * kChunks / kThreads;  // 16-byte chunks a thread stages of K, of V
    static_assert(KT * kChunks % kThreads == 0, "every thread stages the same number of chunks");
    constexpr int kRowStep = kThreads / kChunks;  // rows between a thread's chunks
    constexpr int kKeyRow = Rows<DP>::kKey, kValueRow = Rows<DP>::kValue;
    constexpr int DT = DP / 32, KS = DP / 16, SUB = KT / 32;
    __shared__ __attribute__((aligned(16))) uint16_t sk[2][KT * kKeyRow];
    __shared__ __attribute__((aligned(16))) uint16_t sv[2][KT * kValueRow];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wid = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int hk = blockIdx.x % c.n_kv;
    const int G = a.n_heads / c.n_kv, D = c.head_dim;
    Tile t;
    if (!find_tile<BM>(c, a.q_start, a.T, G, blockIdx.x / c.n_kv, &t)) return;

    const int half = lane >> 5;
    const int row = t.row0 + wid * 32 + (lane & 31);
    const int safe_row = min(row, t.rows - 1);
    const int tok = safe_row / G;
    const int head = hk * G + (safe_row - tok * G);
    const int pos = t.pos0 + tok;

    // the wave's rows: positions first .. last; the block's: tile_first .. tile_last
    const int tile_first = t.pos0 + t.row0 / G;
    const int tile_last = t.pos0 + min(t.row0 + BM - 1, t.rows - 1) / G;
    const int wave_row = min(t.row0 + wid * 32, t.rows - 1);
    const int first = t.pos0 + wave_row / G;
    const int last = t.pos0 + min(t.row0 + wid * 32 + 31, t.rows - 1) / G;

    // Key tiles: those of the sinks, then those from the oldest key in a row's window on.
    const int lo = a.window > 0 ? max(tile_first - a.window + 1, 0) : 0;
    const int n_sink = a.window > 0 ? (min(a.sinks, max(lo, 0)) + KT - 1) / KT : 0;
    const int sinks_end = a.window > 0 ? a.sinks : 0;  // (lo is 0 without a window)
    const int lo_tile = max(lo / KT, n_sink);
    const int n_iter = tile_last < 0 ? 0 : n_sink + tile_last / KT + 1 - lo_tile;

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
    // (a scale of 0 as one that moves no weight, so that hidden scores of -inf stay -inf)
    const float cs = fmaxf(a.scale * kLog2e, 1e-37f);
    const int before = a.window > 0 ? pos - a.window : -1;  // newest position out of the window
    float M = kNoMax, l = 0.0f;

    // Staging: this thread's chunk of rows r0, r0 + kRowStep, ... of each tile. A row whose key no
    // row of the block sees is read from one that some row sees (finite; its weights are 0), dims
    // past D from the row's last chunk (they meet zeros of q, or outputs that are not kept). The
    // page table entries are read a tile ahead of the rows, the rows a tile ahead of their use.
    const int my_chunk = tid % kChunks, r0 = tid / kChunks;
    const int my_col = hk * c.head_stride + min(8 * my_chunk, D - 8);
    const int32_t *table = c.table + t.seq * c.ld_table;
    const auto tile_key = [&](int it) { return (it < n_sink ? it : lo_tile + it - n_sink) * KT; };
    const auto key_of = [&](int it, int i) {
        const int p = min(tile_key(it) + r0 + i * kRowStep, tile_last);
        return p >= sinks_end && p < lo ? lo : p;
    };
    int entry[kLoads];
    const auto look_up = [&](int it) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            entry[i] = read_const(table + (key_of(it, i) >> c.page_shift));
    };
    uintx4_t rk[kLoads], rv[kLoads];
    const auto fetch = [&](int it) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int page = min(max(entry[i], 0), c.n_pages - 1);
            const int64_t at = static_cast<int64_t>(page) * c.page_stride +
                               ((key_of(it, i) & c.page_mask) * c.slot_stride + my_col);
            rk[i] = *reinterpret_cast<const uintx4_t *>(c.k + at);
            rv[i] = *reinterpret_cast<const uintx4_t *>(c.v + at);
        }
    };
    const auto stage = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int r = r0 + i * kRowStep;
            *reinterpret_cast<uintx4_t *>(&sk[buf][r * kKeyRow + 8 * my_chunk]) = rk[i];
            *reinterpret_cast<uintx4_t *>(&sv[buf][r * kValueRow + 8 * my_chunk]) = rv[i];
        }
    };
    if (n_iter > 0) {
        look_up(0);
        fetch(0);
        look_up(min(1, n_iter - 1));
        stage(0);
    }
    __syncthreads();

    if (n_iter > 0) {
    int it = 0;
    do {
        const int buf = it & 1;
        if (it + 1 < n_iter) {
            fetch(it + 1);
            look_up(min(it + 2, n_iter - 1));
        }
        const int k0 = tile_key(it);
        // any key of the tile that some row of the wave sees?
        const bool seen = k0 <= last && (a.window == 0 || k0 < a.sinks ||
                                         k0 + KT - 1 > first - a.window);
        if (seen) {
            floatx16_t s[SUB];
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                s[u] = floatx16_t(0.0f);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const bf16x8_t kf = *reinterpret_cast<const bf16x8_t *>(
                        &sk[buf][(32 * u + (lane & 31)) * kKeyRow + 16 * ks + 8 * half]);
                    s[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf, qf[ks], s[u], 0, 0, 0);
                }
            }
            // every key of the tile seen by every row of the wave?
            const bool whole =
                k0 + KT - 1 <= first &&
                (a.window == 0 || k0 > last - a.window || k0 + KT - 1 < a.sinks);
            if (!whole) {
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int j = k0 + 32 * u + 8 * (i / 4) + 4 * half + i % 4;
                        const bool ok = (j <= pos) & ((j > before) | (j < a.sinks));
                        s[u][i] = ok ? s[u][i] : -INFINITY;
                    }
            }
            float mx = s[0][0];
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int i = 0; i < 16; ++i) mx = fmaxf(mx, s[u][i]);
            mx = fmaxf(mx, other_half(mx)) * cs;
            if (__any(mx > M + kSlack)) {
                const float M2 = fmaxf(M, mx);
                const float f = __builtin_amdgcn_exp2f(M - M2);
                M = M2;
                l *= f;
#pragma unroll
                for (int d = 0; d < DT; ++d) o[d] *= f;
            }
            bf16x8_t pf[SUB][2];
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                uintx4_t w[2];
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const float p0 = __builtin_amdgcn_exp2f(fmaf(s[u][i], cs, -M));
                    const float p1 = __builtin_amdgcn_exp2f(fmaf(s[u][i + 1], cs, -M));
                    l += p0 + p1;
                    w[i / 8][i % 8 / 2] = pack_bf16(p0, p1);
                }
                pf[u][0] = __builtin_bit_cast(bf16x8_t, w[0]);
                pf[u][1] = __builtin_bit_cast(bf16x8_t, w[1]);
            }
            // O^T += V^T P^T, 16 keys a step: slots 8 half + 0..3 are keys 4 half + 0..3 of the
            // step, slots 8 half + 4..7 keys 8 + 4 half + 0..3
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int st = 0; st < 2; ++st) {
                    const uint16_t *vp =
                        &sv[buf][(32 * u + 16 * st + 4 * half + (lane & 15) / 4) * kValueRow +
                                 (lane & 16) + 4 * (lane & 3)];
#pragma unroll
                    for (int d = 0; d < DT; ++d) {
                        const uintx2_t v0 = lds_read_transposed(vp + 32 * d);
                        const uintx2_t v1 = lds_read_transposed(vp + 8 * kValueRow + 32 * d);
                        const uintx4_t vv = {v0[0], v0[1], v1[0], v1[1]};
                        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                            __builtin_bit_cast(bf16x8_t, vv), pf[u][st], o[d], 0, 0, 0);
                    }
                }
        }
        if (it + 1 < n_iter) stage(buf ^ 1);
        __syncthreads();
    } while (++it < n_iter);
    }

    l += other_half(l);
    if (row >= t.rows) return;
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    const int64_t token = t.q0 + tok;
    if (a.lse && half == 0)
        a.lse[token * a.n_heads + head] = l > 0.0f ? M * kLn2 + logf(l) : -INFINITY;
    const int64_t base = token * a.ldy + static_cast<int64_t>(head) * D;
    const bool wide = wide_rows(a);
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int col = 32 * d + 8 * g + 4 * half;
            if (col >= D) continue;
            floatx4_t v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = o[d][4 * g + i] * inv;
            store_out4(a.y, base + col, v, a.out_f32, wide);
        }
}

template <int DP, int NW, int KT>
void launch(const AttnArgs &a, const KvView &c, hipStream_t stream) {
    const int64_t G = a.n_heads / c.n_kv;
    // at most this many tiles: every sequence rounds up once
    const int64_t tiles = a.T * G / (NW * 32) + c.n_seqs;
    const dim3 grid(static_cast<unsigned>(tiles * c.n_kv));
    hipLaunchKernelGGL((attn_prefill_kernel<DP, NW, KT>), grid, dim3(NW * 64), 0, stream, a, c,
                       static_cast<int>(tiles));
}

}  // namespace

size_t attn_prefill_work_bytes(int64_t, int, const KvView &, int, int) { return 0; }

hipError_t launch_attn_prefill(const AttnArgs &a, const KvView &c, hipStream_t stream) {
    if (c.head_dim <= 64)
        launch<64, 8, 64>(a, c, stream);
    else if (c.head_dim <= 128)
        launch<128, 8, 64>(a, c, stream);
    else
        launch<256, 8, 32>(a, c, stream);
    return hipGetLastError();
}

}  // namespace w4
