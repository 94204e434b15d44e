// tables.hip -- the page tables, lengths and slots of a serving step from its requests' lengths
// (w4_batch_tables).
//
// Three sums run over the sequences: token rows before a sequence (q_start), pages given out before
// it, pages that came back before it. They are taken by every workgroup for itself, 1024 sequences
// at a time (up to four a thread), so that one launch does: what a workgroup then needs of a
// sequence lies in LDS. The rows, the new table entries and the pages that come back are numbered
// through, each thread finds the sequence of its number by bisection, and the workgroups share the
// numbers out.
//
// A page given out is named by its number alone (place head + number of the ring), so that no
// workgroup waits for an entry that another one writes: entries read lie below a span's end, entries
// written at it or after; ring places read hold pages before the call, places written none.
//
// Bound by waits one after the other, lengths, sums, table, stores: in a graph 7.4 us for a decode step of
// 48 sequences, three of which give back 1200 pages, in one workgroup; 11.3 us for 512 prompts of 1.05
// million tokens (20 MB written, 3.3 us at the rate of memory). Four items of a thread at once: 7.4 us for
// 7.7 and 11.3 for 12.1 with one.
#include "attn_device.h"

namespace w4 {

namespace {

constexpr int kThreads = 256, kPerThread = 4, kChunk = kThreads * kPerThread;
constexpr int kAtOnce = 4;  // items of a thread, their searches and loads in flight together
constexpr int kMostTokens = (1 << 30) - 1;

struct Sums {
    int rows, fresh, back;
};

// What a sequence asks for. rows: at most `T` (sums of rows stop there).
struct Request {
    int len, tokens, begin, end, want;
    bool over;
    __device__ __forceinline__ int fresh() const { return over ? 0 : max(want - end, 0); }
    __device__ __forceinline__ int back() const { return over ? end - begin : 0; }
};
__device__ __forceinline__ Request request(const TablesArgs &a, int b) {
    Request r;
    const int n = a.kv_len[b], m = a.n_new[b];
    r.over = m < 0;
    r.len = max(n, 0);  // (past the table's last column too: only what names pages ends there)
    r.tokens = min(max(m, 0), kMostTokens);
    r.begin = min(max(a.spans[2 * b], 0), a.table_cols);
    r.end = min(max(a.spans[2 * b + 1], r.begin), a.table_cols);
    const int64_t keys = static_cast<int64_t>(r.len) + r.tokens;
    r.want = static_cast<int>(
        min((keys + (1 << a.page_shift) - 1) >> a.page_shift, static_cast<int64_t>(a.table_cols)));
    return r;
}

__device__ __forceinline__ int upto_31_bits(uint32_t v) {
    return static_cast<int>(min(v, uint32_t{INT32_MAX}));
}

// Sums over lanes 0 .. own lane; `rows` stop at T (as good as a sum: all are >= 0).
__device__ __forceinline__ int wave_scan_upto(int v, int T) {
    v = min(v + dpp_i<0x111, 0xF, true>(v), T);
    v = min(v + dpp_i<0x112, 0xF, true>(v), T);
    v = min(v + dpp_i<0x114, 0xF, true>(v), T);
    v = min(v + dpp_i<0x118, 0xF, true>(v), T);
    v = min(v + dpp_i<0x142, 0xA, false>(v), T);
    v = min(v + dpp_i<0x143, 0xC, false>(v), T);
    return v;
}

// FILL: rows, table entries and ring places; LENGTHS: what a sequence and the ring have afterwards.
enum { kFill = 1, kLengths = 2 };

__global__ void __launch_bounds__(kThreads) batch_tables_kernel(TablesArgs a, int what) {
    __shared__ int s_row[kChunk], s_fresh[kChunk], s_back[kChunk];  // before each sequence
    __shared__ int s_len[kChunk], s_begin[kChunk], s_end[kChunk];
    __shared__ Sums s_wave[kThreads / kWave];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wid = tid / kWave;
    const int T = a.T, R = a.ring_size;
    const int count = min(max(a.ring_state[1], 0), R);
    const int head = a.ring_state[0] >= 0 && a.ring_state[0] < R ? a.ring_state[0] : 0;
    const bool lengths = (what & kLengths) && blockIdx.x == 0;
    const bool fill = (what & kFill) != 0;
    const int start = blockIdx.x * kThreads * kAtOnce + tid, step = gridDim.x * kThreads * kAtOnce;
    // the ring's place of number k from its head on
    const auto place_of = [&](int64_t k) { return head + k >= R ? head + k - R : head + k; };

    Sums before = {0, 0, 0};
    if (lengths && tid == 0) a.q_start[0] = 0;
    for (int base = 0; base < a.n_seqs; base += kChunk) {
        const int n = min(a.n_seqs - base, kChunk);
        // the sequences of a thread follow each other
        const int each = (n + kThreads - 1) / kThreads;
        Request r[kPerThread];
        Sums mine = {0, 0, 0};
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            const int b = base + tid * each + i;
            if (i < each && b < a.n_seqs) {
                r[i] = request(a, b);
                mine.rows = min(mine.rows + min(r[i].tokens, T), T);
                mine.fresh += r[i].fresh();
                mine.back += r[i].back();
            }
        }
        Sums upto = {wave_scan_upto(mine.rows, T), wave_scan_dpp(mine.fresh),
                     wave_scan_dpp(mine.back)};
        if (lane == kWave - 1) s_wave[wid] = upto;
        // (sums before this thread: rows by a lane shift, since their sums stop at T)
        Sums at = {__shfl_up(upto.rows, 1, kWave), upto.fresh - mine.fresh, upto.back - mine.back};
        if (lane == 0) at.rows = 0;
        __syncthreads();
        Sums all = before;
#pragma unroll
        for (int w = 0; w < kThreads / kWave; ++w) {
            if (w == wid) {
                at.rows = min(at.rows + all.rows, T);
                at.fresh += all.fresh;
                at.back += all.back;
            }
            all.rows = min(all.rows + s_wave[w].rows, T);
            all.fresh += s_wave[w].fresh;
            all.back += s_wave[w].back;
        }
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            const int place = tid * each + i, b = base + place;
            if (i < each && b < a.n_seqs) {
                s_row[place] = at.rows;
                s_fresh[place] = at.fresh;
                s_back[place] = at.back;
                s_len[place] = r[i].len;
                s_begin[place] = r[i].begin;
                s_end[place] = r[i].end;
                const int first = at.fresh;
                at.rows = min(at.rows + min(r[i].tokens, T), T);
                at.fresh += r[i].fresh();
                at.back += r[i].back();
                if (lengths) {
                    const int got = min(max(count - first, 0), r[i].fresh());
                    a.q_start[b + 1] = at.rows;
                    a.kv_len_out[b] =
                        r[i].over ? 0 : upto_31_bits(uint32_t(r[i].len) + uint32_t(r[i].tokens));
                    a.spans_out[2 * b] = r[i].over ? 0 : r[i].begin;
                    a.spans_out[2 * b + 1] = r[i].over ? 0 : r[i].end + got;
                }
            }
        }
        __syncthreads();
        if (fill) {
            // The items of these sequences: new table entries, pages that come back, rows; each takes
            // one page from the table or the ring.
            const int fresh = all.fresh - before.fresh;
            const int back = max(min(all.back, R - count) - before.back, 0);
            const int items = fresh + back + all.rows - before.rows;
            // the last sequence of p .. n - 1 with no more than k before it; steps: at least n - p
            const auto find = [&](const int *first, int p, int bit, int k) {
                const int at = min(p + bit, n - 1);
                return first[at] <= k ? at : p;
            };
            for (int j0 = start; j0 - tid < items; j0 += step) {
                // Where the workgroup's items are all rows, they belong to few sequences.
                int from = 0, bits = n;
                const int rows0 = fresh + back, c0 = j0 - tid;
                if (c0 >= rows0) {
                    const int k0 = before.rows + c0 - rows0;
                    const int k1 = min(k0 + kThreads * kAtOnce, all.rows) - 1;
                    int last = 0;
                    for (int bit = 1 << (31 - __builtin_clz(n)); bit > 0; bit >>= 1) {
                        from = find(s_row, from, bit, k0);
                        last = find(s_row, last, bit, k1);
                    }
                    bits = last - from;
                }
                int kind[kAtOnce], k[kAtOnce], p[kAtOnce], page[kAtOnce];
                const int *first[kAtOnce];
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) {
                    const int j = min(j0 + i * kThreads, items - 1);
                    kind[i] = j < fresh ? 0 : j < fresh + back ? 1 : 2;
                    k[i] = kind[i] == 0   ? before.fresh + j
                           : kind[i] == 1 ? before.back + j - fresh
                                          : before.rows + j - fresh - back;
                    first[i] = kind[i] == 0 ? s_fresh : kind[i] == 1 ? s_back : s_row;
                    p[i] = from;
                }
                for (int bit = bits > 0 ? 1 << (31 - __builtin_clz(bits)) : 0; bit > 0; bit >>= 1)
#pragma unroll
                    for (int i = 0; i < kAtOnce; ++i) p[i] = find(first[i], p[i], bit, k[i]);
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) {
                    const int b = base + p[i], end = s_end[p[i]], in = k[i] - first[i][p[i]];
                    // (positions need 32 bits; a column beyond the table is only compared)
                    const uint32_t pos = static_cast<uint32_t>(s_len[p[i]]) + in;
                    const int col = kind[i] == 1 ? s_begin[p[i]] + in
                                                 : upto_31_bits(pos >> a.page_shift);
                    const bool inside = col < a.table_cols;
                    // number among the pages given out, of a new entry or a row on one
                    const int number = kind[i] == 0 ? k[i] : s_fresh[p[i]] + (inside ? col - end : 0);
                    const bool held = kind[i] == 1 || (kind[i] == 2 && col < end);
                    page[i] = -1;
                    if (held)
                        page[i] = a.page_table[b * a.ld_table + col];
                    else if (number < count && (kind[i] == 0 || inside))
                        page[i] = a.ring[place_of(number)];
                }
#pragma unroll
                for (int i = 0; i < kAtOnce; ++i) {
                    if (j0 + i * kThreads >= items) break;
                    const int b = base + p[i], in = k[i] - first[i][p[i]];
                    if (kind[i] == 0) {
                        a.page_table[b * a.ld_table + s_end[p[i]] + in] = page[i];
                    } else if (kind[i] == 1) {
                        a.ring[place_of(static_cast<int64_t>(count) + k[i])] = page[i];
                    } else {
                        const uint32_t pos = static_cast<uint32_t>(s_len[p[i]]) + in;
                        if (a.slots)
                            a.slots[k[i]] = page[i] < 0
                                                ? -1
                                                : (static_cast<int64_t>(page[i]) << a.page_shift) +
                                                      (pos & ((1u << a.page_shift) - 1));
                        if (a.seqs) a.seqs[k[i]] = b;
                        if (a.positions) a.positions[k[i]] = upto_31_bits(pos);
                    }
                }
            }
        }
        before = all;
        __syncthreads();
    }
    if (fill) {
        for (int t = before.rows + blockIdx.x * kThreads + tid; t < T; t += gridDim.x * kThreads) {
            if (a.slots) a.slots[t] = -1;
            if (a.seqs) a.seqs[t] = -1;
            if (a.positions) a.positions[t] = -1;
        }
    }
    if (lengths && tid == 0) {
        const int taken = min(before.fresh, count);
        const int back = min(before.back, R - count);
        a.ring_state_out[0] = head + taken >= R ? head + taken - R : head + taken;
        a.ring_state_out[1] = count - taken + back;
        a.ring_state_out[2] = before.fresh - taken;
    }
}

}  // namespace

hipError_t launch_batch_tables(const TablesArgs &a, bool in_place, hipStream_t stream) {
    // A workgroup for every 1024 rows, which is what one takes at once, or for every 65536 entries that
    // the table could have to give or take (few of them in most calls).
    const int64_t rows = (a.T + kChunk - 1) / kChunk;
    const int64_t entries = a.n_seqs * static_cast<int64_t>(a.table_cols) >> 16;
    const int64_t most = 4 * static_cast<int64_t>(device_cu_count());
    int64_t grid = rows > entries ? rows : entries;
    grid = grid < 1 ? 1 : grid > most ? most : grid;
    // Lengths in place are written when no workgroup reads them any more.
    const bool two = in_place && grid > 1;
    hipLaunchKernelGGL(batch_tables_kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0,
                       stream, a, two ? kFill : kFill | kLengths);
    if (two) {
        const hipError_t err = hipGetLastError();
        if (err != hipSuccess) return err;
        hipLaunchKernelGGL(batch_tables_kernel, dim3(1), dim3(kThreads), 0, stream, a, kLengths);
    }
    return hipGetLastError();
}

}  // namespace w4
