// attn_decode.hip -- attention of one new token per sequence over the paged cache.
//
// One pass over the keys and values of a sequence (w4_attn_decode), bound by reading them: 4 flop
// per byte and query head. The G = n_heads / n_kv query heads of a key-value head are the columns
// of one 16-wide matrix-core tile, so that a key is read once for all of them (16 at a time).
//
//   S^T[key][head] = K Q^T   on v_mfma_f32_16x16x32_bf16; a lane's 16 bytes of a key row are the
//                            operand as they come from memory
//   O^T[d][head]  += V^T P^T V through LDS and its transposed read; P^T is, register for register,
//                            the operand: V's rows follow the key order the first product left
// P enters the second product as the sum of two bf16 values (16 bits of each weight): the matrix
// cores have time to spare here.
//
// A sequence's visible keys (its sinks, then its window; all without a window) are cut into tiles
// of 32 keys and chunks of tiles; a workgroup takes a chunk, each of its four waves every fourth
// tile on its own (no barrier in the loop, the next tile's loads in flight), and joins the waves'
// results in LDS. Where a sequence has more than one chunk, the chunks' results meet in the caller's
// workspace and a second kernel joins them in order.
#include "attn_device.h"

namespace w4 {

namespace {

constexpr int kTile = 32;   // keys of a tile
constexpr int kWaves = 4;
constexpr int kRows = 16;   // query heads of a workgroup
constexpr int kSlack = 8;   // log2 of how far a weight may pass 1 before the sums are rescaled

// The visible keys of a sequence, as tiles.
struct Keys {
    int last, lo;          // newest key; oldest key inside the window
    int n_sink, lo_tile;   // tiles of sinks; first tile after them
    int n_tiles;
    __device__ __forceinline__ int start(int t) const {
        return (t < n_sink ? t : lo_tile + t - n_sink) * kTile;
    }
};

__device__ __forceinline__ Keys visible_keys(const AttnArgs &a, const KvView &c, int b) {
    Keys k;
    const int n = kv_length(c, b);
    k.last = n - 1;
    k.lo = a.window > 0 ? max(n - a.window, 0) : 0;
    k.n_sink = (min(a.sinks, k.lo) + kTile - 1) / kTile;
    k.lo_tile = max(k.lo / kTile, k.n_sink);
    k.n_tiles = n == 0 ? 0 : k.n_sink + k.last / kTile + 1 - k.lo_tile;
    return k;
}

// Partial results: per (sequence, head, chunk) D weighted sums, then per (sequence, head, chunk)
// the pair (maximum in log2 units, sum of weights).
struct Partials {
    float *o;
    float *ml;
    int chunks;
};

__host__ __device__ __forceinline__ Partials partials(void *work, int64_t pairs, int chunks,
                                                      int D) {
    Partials p;
    p.o = static_cast<float *>(work);
    p.ml = p.o + pairs * chunks * D;
    p.chunks = chunks;
    return p;
}

// PAGE16: pages of 16 slots and more, so that 16 aligned keys lie in one page.
template <int DP, bool PAGE16>
__global__ void __launch_bounds__(kWaves * 64)
__attribute__((amdgpu_waves_per_eu(DP > 128 ? 1 : DP > 64 ? 3 : 4))) attn_decode_kernel(
    AttnArgs a, KvView c, int chunk_tiles, Partials parts) {
    constexpr int KS = DP / 32;      // steps of the first product
    constexpr int DT = DP / 16;      // tiles of the second
    constexpr int kChunks = DP / 8;  // 16-byte chunks of a row
    constexpr int kVRows = 64 / kChunks;       // rows a wave's load instruction covers
    constexpr int kVLoads = kTile / kVRows;
    // per wave: the value tile [32][DP] bf16; after the loop its sums [16][DP] fp32 (the same size)
    __shared__ __attribute__((aligned(16))) uint16_t sv[kWaves][kTile * DP];
    __shared__ float sm[kWaves][kRows], sl[kWaves][kRows];

    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int G = a.n_heads / c.n_kv, D = c.head_dim;
    const int row_tiles = (G + kRows - 1) / kRows;
    int id = blockIdx.x;
    const int rt = id % row_tiles;
    id /= row_tiles;
    const int hk = id % c.n_kv;
    id /= c.n_kv;
    const int b = id % c.n_seqs, chunk = id / c.n_seqs;
    const Keys keys = visible_keys(a, c, b);
    const int t0 = chunk * chunk_tiles;
    const int t1 = min(keys.n_tiles, t0 + chunk_tiles);
    if (chunk > 0 && t0 >= t1) return;  // (chunk 0 of an empty sequence writes its zeros)

    const int r = lane & 15, g = lane >> 4;  // column (query head), group of 16 lanes
    const int head0 = hk * G + rt * kRows;
    const int n_rows = min(G - rt * kRows, kRows);

    bf16x8_t qf[KS];
    {
        const uint16_t *src = a.q + b * a.ldq + static_cast<int64_t>(head0 + min(r, n_rows - 1)) * D;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int d = 32 * s + 8 * g;
            uintx4_t v = {0, 0, 0, 0};
            if (d < D) v = *reinterpret_cast<const uintx4_t *>(src + d);
            qf[s] = __builtin_bit_cast(bf16x8_t, v);
        }
    }

    const int32_t *table = c.table + b * c.ld_table;
    const int64_t head_off = static_cast<int64_t>(hk) * c.head_stride;
    const auto visible = [&](int p) { return p <= keys.last && (p >= keys.lo || p < a.sinks); };
    // Where the 16 keys from s0 on are read: a key that is not visible is replaced by one that is
    // (finite values; its weight is 0), by one of the same 16 if there is any.
    const auto safe_key = [&](int s0) {
        if (s0 <= keys.last && (s0 < a.sinks || s0 + 15 >= keys.lo))
            return s0 < a.sinks && s0 < keys.lo ? s0 : max(s0, keys.lo);
        return keys.last;
    };
    // Element offset of key p of the 16 from s0 on (page_off: the offset of safe_key(s0)'s page).
    const auto page_off = [&](int safe) {
        return static_cast<int64_t>(kv_page(c, table, safe)) * c.page_stride + head_off;
    };
    const auto in_page = [&](int p, int safe) {
        return static_cast<uint32_t>(((visible(p) ? p : safe) & c.page_mask) * c.slot_stride);
    };

    uintx4_t rk[2][KS], rv[kVLoads];
    const auto fetch_k = [&](int k0) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int s0 = k0 + 16 * u, safe = safe_key(s0), p = s0 + r;
            const uint16_t *row = c.k + (PAGE16 ? page_off(safe)
                                                : page_off(visible(p) ? p : safe)) +
                                  in_page(p, safe);
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                const int d = 32 * s + 8 * g;
                rk[u][s] = uintx4_t{0, 0, 0, 0};
                if (d < D) rk[u][s] = *reinterpret_cast<const uintx4_t *>(row + d);
            }
        }
    };
    const int v_row = lane / kChunks, v_chunk = lane % kChunks;
    const auto fetch_v = [&](int k0) {
#pragma unroll
        for (int i = 0; i < kVLoads; ++i) {
            const int s0 = k0 + i * kVRows / 16 * 16, safe = safe_key(s0);
            const int p = k0 + i * kVRows + v_row;
            rv[i] = uintx4_t{0, 0, 0, 0};
            if (v_chunk * 8 < D)
                rv[i] = *reinterpret_cast<const uintx4_t *>(
                    c.v + (PAGE16 ? page_off(safe) : page_off(visible(p) ? p : safe)) +
                    in_page(p, safe) + v_chunk * 8);
        }
    };

    floatx4_t o[DT];
#pragma unroll
    for (int i = 0; i < DT; ++i) o[i] = floatx4_t(0.0f);
    const float cs = a.scale * kLog2e;
    float M = kNoMax, l = 0.0f;
    uint16_t *my_v = sv[wid];

    int t = t0 + wid;
    if (t < t1) {
        fetch_k(keys.start(t));
        fetch_v(keys.start(t));
    }
    for (; t < t1; t += kWaves) {
        const int k0 = keys.start(t);
        const int next = keys.start(min(t + kWaves, t1 - 1));  // (the last tile again at the end)
        floatx4_t s[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            s[u] = floatx4_t(0.0f);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
                s[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    __builtin_bit_cast(bf16x8_t, rk[u][ks]), qf[ks], s[u], 0, 0, 0);
        }
        fetch_k(next);
#pragma unroll
        for (int i = 0; i < kVLoads; ++i)
            *reinterpret_cast<uintx4_t *>(
                &my_v[8 * value_slot<DP>(i * kVRows + v_row, v_chunk)]) = rv[i];
        asm volatile("" ::: "memory");
        __builtin_amdgcn_wave_barrier();
        fetch_v(next);

        float mx = -INFINITY;
        bool ok[2][4];
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                ok[u][i] = visible(k0 + 16 * u + 4 * g + i);
                s[u][i] = s[u][i] * cs;
                mx = ok[u][i] ? fmaxf(mx, s[u][i]) : mx;
            }
        mx = fmaxf(mx, __shfl_xor(mx, 16, kWave));
        mx = fmaxf(mx, __shfl_xor(mx, 32, kWave));
        if (__any(mx > M + kSlack)) {
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
        const int vr = 4 * g + r / 4;
#pragma unroll
        for (int d = 0; d < DT; ++d) {
            const int col = 16 * d + 4 * (r & 3);
            const uintx2_t v0 = lds_read_transposed(&my_v[8 * value_slot<DP>(vr, col / 8) + col % 8]);
            const uintx2_t v1 =
                lds_read_transposed(&my_v[8 * value_slot<DP>(vr + 16, col / 8) + col % 8]);
            const uintx4_t vv = {v0[0], v0[1], v1[0], v1[1]};
            const bf16x8_t vf = __builtin_bit_cast(bf16x8_t, vv);
            o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, __builtin_bit_cast(bf16x8_t, hi),
                                                           o[d], 0, 0, 0);
            o[d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, __builtin_bit_cast(bf16x8_t, lo),
                                                           o[d], 0, 0, 0);
        }
        asm volatile("" ::: "memory");
        __builtin_amdgcn_wave_barrier();
    }

    // Join the waves: lane (g, r) holds dims 16 d + 4 g + 0..3 of head r.
    l += __shfl_xor(l, 16, kWave);
    l += __shfl_xor(l, 32, kWave);
    if (g == 0) {
        sm[wid][r] = M;
        sl[wid][r] = l;
    }
    float *my_o = reinterpret_cast<float *>(my_v);
#pragma unroll
    for (int d = 0; d < DT; ++d)
        *reinterpret_cast<floatx4_t *>(&my_o[r * DP + 16 * d + 4 * g]) = o[d];
    __syncthreads();
    const bool whole = keys.n_tiles <= chunk_tiles;  // this chunk is all there is
    const bool wide = wide_rows(a);
    for (int e = threadIdx.x; e < n_rows * (DP / 4); e += kWaves * 64) {
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
            v += f * *reinterpret_cast<const floatx4_t *>(
                         reinterpret_cast<const float *>(sv[w]) + row * DP + d);
        }
        const int64_t pair = static_cast<int64_t>(b) * a.n_heads + head0 + row;
        if (whole) {
            v *= sum > 0.0f ? 1.0f / sum : 0.0f;
            store_out4(a.y, b * a.ldy + static_cast<int64_t>(head0 + row) * D + d, v, a.out_f32,
                       wide);
            if (a.lse && d == 0) a.lse[pair] = sum > 0.0f ? m * kLn2 + logf(sum) : -INFINITY;
        } else {
            const int64_t at = pair * parts.chunks + chunk;
            *reinterpret_cast<floatx4_t *>(parts.o + at * D + d) = v;
            if (d == 0) {
                parts.ml[2 * at] = m;
                parts.ml[2 * at + 1] = sum;
            }
        }
    }
}

// Joins a (sequence, head)'s chunks: one workgroup each, its threads over groups of chunks and the
// head's dims, the groups' sums through LDS in order.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(AttnArgs a, KvView c,
                                                                 int chunk_tiles, Partials parts) {
    __shared__ floatx4_t so[kJoinThreads];
    __shared__ float red[kJoinThreads / 64], sw[kJoinThreads];
    const int64_t pair = blockIdx.x;
    const int b = static_cast<int>(pair / a.n_heads), head = static_cast<int>(pair % a.n_heads);
    const int n_tiles = visible_keys(a, c, b).n_tiles;
    if (n_tiles <= chunk_tiles) return;  // written by the first kernel
    const int n = (n_tiles + chunk_tiles - 1) / chunk_tiles;
    const float *ml = parts.ml + 2 * pair * parts.chunks;
    const float *o = parts.o + pair * parts.chunks * c.head_dim;
    const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;

    float m = kNoMax;
    for (int i = tid; i < n; i += kJoinThreads) m = fmaxf(m, ml[2 * i]);
    m = wave_max(m);
    if (lane == 0) red[wid] = m;
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int w = 1; w < kJoinThreads / 64; ++w) m = fmaxf(m, red[w]);

    const int lanes = c.head_dim / 4;          // threads over the dims, 4 each
    const int groups = kJoinThreads / lanes;   // (threads past groups * lanes idle)
    const int grp = tid / lanes, d = tid % lanes * 4;
    float l = 0.0f;
    floatx4_t v = floatx4_t(0.0f);
    if (grp < groups) {
        for (int i = grp; i < n; i += groups) {
            const float f = __builtin_amdgcn_exp2f(ml[2 * i] - m);
            l += f * ml[2 * i + 1];
            v += f * *reinterpret_cast<const floatx4_t *>(o + static_cast<int64_t>(i) * c.head_dim + d);
        }
        so[tid] = v;
        sw[tid] = l;
    }
    __syncthreads();
    if (tid >= lanes) return;
    for (int q = 1; q < groups; ++q) {
        v += so[q * lanes + tid];
        l += sw[q * lanes + tid];
    }
    v *= l > 0.0f ? 1.0f / l : 0.0f;
    store_out4(a.y, b * a.ldy + static_cast<int64_t>(head) * c.head_dim + d, v, a.out_f32,
               wide_rows(a));
    if (a.lse && d == 0) a.lse[pair] = l > 0.0f ? m * kLn2 + logf(l) : -INFINITY;
}

// How the keys are cut: chunks of at least one tile per wave, as few as give the card four
// workgroups per compute unit.
struct Plan {
    int chunk_tiles, chunks, units;
};
Plan plan_of(int n_heads, const KvView &c, int window, int sinks) {
    const int G = n_heads / c.n_kv;
    Plan p;
    p.units = c.n_seqs * c.n_kv * ((G + kRows - 1) / kRows);
    // tiles a sequence can have: its window and its sinks touch at most two partial tiles each
    int64_t keys = c.capacity;
    if (window > 0 && int64_t(window) + sinks + 4 * kTile < keys)
        keys = int64_t(window) + sinks + 4 * kTile;
    const int64_t tiles = (keys + kTile - 1) / kTile;
    const int64_t want = 4ll * device_cu_count();
    int64_t per = (tiles * p.units + want - 1) / want;
    per = (per + kWaves - 1) / kWaves * kWaves;
    p.chunk_tiles = static_cast<int>(per < kWaves ? kWaves : per);
    p.chunks = static_cast<int>((tiles + p.chunk_tiles - 1) / p.chunk_tiles);
    return p;
}

template <int DP>
void launch(const Plan &p, const AttnArgs &a, const KvView &c, const Partials &parts,
            hipStream_t stream) {
    const dim3 grid(static_cast<unsigned>(p.units) * static_cast<unsigned>(p.chunks));
    if (c.page_mask >= 15)
        hipLaunchKernelGGL((attn_decode_kernel<DP, true>), grid, dim3(kWaves * 64), 0, stream, a,
                           c, p.chunk_tiles, parts);
    else
        hipLaunchKernelGGL((attn_decode_kernel<DP, false>), grid, dim3(kWaves * 64), 0, stream, a,
                           c, p.chunk_tiles, parts);
}

}  // namespace

size_t attn_decode_work_bytes(int n_heads, const KvView &c, int window, int sinks) {
    const Plan p = plan_of(n_heads, c, window, sinks);
    if (p.chunks <= 1) return 0;
    return static_cast<size_t>(c.n_seqs) * n_heads * p.chunks * (c.head_dim + 2) * sizeof(float);
}

hipError_t launch_attn_decode(const AttnArgs &a, const KvView &c, hipStream_t stream) {
    const Plan p = plan_of(a.n_heads, c, a.window, a.sinks);
    const int64_t pairs = static_cast<int64_t>(c.n_seqs) * a.n_heads;
    const Partials parts = partials(a.work, pairs, p.chunks, c.head_dim);
    if (c.head_dim <= 64)
        launch<64>(p, a, c, parts, stream);
    else if (c.head_dim <= 128)
        launch<128>(p, a, c, parts, stream);
    else
        launch<256>(p, a, c, parts, stream);
    if (p.chunks > 1) {
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
        hipLaunchKernelGGL(attn_join_kernel, dim3(static_cast<unsigned>(pairs)),
                           dim3(kJoinThreads), 0, stream, a, c, p.chunk_tiles, parts);
    }
    return hipGetLastError();
}

}  // namespace w4
