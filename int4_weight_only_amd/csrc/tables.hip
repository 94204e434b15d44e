// tables.hip -- the page tables, lengths and slots of a serving step from its requests' lengths
// (w4_batch_tables).
//
// Three sums run over the sequences: token rows before a sequence (q_start), pages given out before
// it, pages that came back before it. They are taken by every workgroup for itself, 1024 sequences
// at a time (four of 256 threads each), so that one launch does: what a workgroup then needs of a
// sequence lies in LDS. The rows, the new table entries and the pages that come back are numbered
// through, each thread finds the sequence of its number by bisection, and the workgroups share the
// numbers out.
//
// A page given out is named by its number alone (place head + number of the ring), so that no
// workgroup waits for an entry that another one writes: entries read lie below a span's end, entries
// written at it or after; ring places read hold pages before the call, places written none.
#include "attn_device.h"

namespace w4 {

namespace {

constexpr int kThreads = 256, kPerThread = 4, kChunk = kThreads * kPerThread;
constexpr int kRowsAtOnce = 4;  // consecutive rows of a thread: its stores are 16 bytes and more
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
    const int capacity = a.table_cols << a.page_shift;
    r.over = m < 0;
    r.len = min(max(n, 0), capacity);
    r.tokens = min(max(m, 0), kMostTokens);
    r.begin = min(max(a.spans[2 * b], 0), a.table_cols);
    r.end = min(max(a.spans[2 * b + 1], r.begin), a.table_cols);
    const int64_t keys = static_cast<int64_t>(r.len) + r.tokens;
    r.want = static_cast<int>(
        min((keys + (1 << a.page_shift) - 1) >> a.page_shift, static_cast<int64_t>(a.table_cols)));
    return r;
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

// The last of n ascending numbers that is at most x (the first one is).
__device__ __forceinline__ int find(const int *first, int n, int x) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (first[mid] <= x)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
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
    const int start = blockIdx.x * kThreads + tid, step = gridDim.x * kThreads;
    // the page of number k among those given out, -1 where the ring holds no more
    const auto given = [&](int k) {
        if (k >= count) return -1;
        const int at = head + k;
        return a.ring[at >= R ? at - R : at];
    };

    Sums before = {0, 0, 0};
    if (lengths && tid == 0) a.q_start[0] = 0;
    for (int base = 0; base < a.n_seqs; base += kChunk) {
        const int n = min(a.n_seqs - base, kChunk);
        // the sequences of a thread follow each other
        Request r[kPerThread];
        Sums mine = {0, 0, 0};
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            const int b = base + tid * kPerThread + i;
            if (b < a.n_seqs) {
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
            const int place = tid * kPerThread + i, b = base + place;
            if (b < a.n_seqs) {
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
                    a.kv_len_out[b] = r[i].over ? 0 : r[i].len + r[i].tokens;
                    a.spans_out[2 * b] = r[i].over ? 0 : r[i].begin;
                    a.spans_out[2 * b + 1] = r[i].over ? 0 : r[i].end + got;
                }
            }
        }
        __syncthreads();
        if (fill) {
            // new table entries
            for (int k = before.fresh + start; k < all.fresh; k += step) {
                const int p = find(s_fresh, n, k);
                a.page_table[(base + p) * a.ld_table + s_end[p] + k - s_fresh[p]] = given(k);
            }
            // pages that come back, behind those of the ring
            for (int k = before.back + start; k < all.back && k < R - count; k += step) {
                const int p = find(s_back, n, k);
                const int64_t to = static_cast<int64_t>(head) + count + k;
                a.ring[to >= R ? to - R : to] =
                    a.page_table[(base + p) * a.ld_table + s_begin[p] + k - s_back[p]];
            }
            // rows
            for (int t = before.rows + start; t < all.rows; t += step) {
                const int p = find(s_row, n, t);
                const int pos = s_len[p] + t - s_row[p], col = pos >> a.page_shift;
                int page = -1;
                if (col < s_end[p])
                    page = a.page_table[(base + p) * a.ld_table + col];
                else if (col < a.table_cols)
                    page = given(s_fresh[p] + col - s_end[p]);
                if (a.slots)
                    a.slots[t] = page < 0 ? -1
                                          : (static_cast<int64_t>(page) << a.page_shift) +
                                                (pos & ((1 << a.page_shift) - 1));
                if (a.seqs) a.seqs[t] = base + p;
                if (a.positions) a.positions[t] = pos;
            }
        }
        before = all;
        __syncthreads();
    }
    if (fill) {
        for (int t = before.rows + start; t < T; t += step) {
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
