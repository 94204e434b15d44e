// rope.hip -- rotary positions on the fused q/k/v projection, with the append of k and v to the
// paged cache (w4_rope_append).
//
// A pair (a, b) of a head at position p turns by t = p * f: (a cos t - b sin t, a sin t + b cos t).
// The reduction modulo one turn is done in fp64, where it is off by less than 2^-23 of a turn at
// the largest position, 2^30; an fp32 angle would already be off by 4e-3, the rounding step of
// bf16, at position 10^5.
//
// Memory-bound: qkv is read once, q and the new cache rows are written once. 8 prompts of up to
// 2048 tokens, 28 + 4 + 4 heads of 128: 239 MB in 41 us (46 called from Python), 5.8 TB/s. One
// token: 3.7 us, the launch and two waits for memory (length and page, then the row).
#include "bf16_device.h"
#include "w4_device.h"
#include "w4_launch.h"

namespace w4 {

namespace {

__device__ __forceinline__ void turn(int pos, float inv_freq, float factor, float *c, float *s) {
    constexpr double kInv2Pi = 0.15915494309189533577;
    const double turns = static_cast<double>(pos) * static_cast<double>(inv_freq) * kInv2Pi;
    const float t = static_cast<float>(turns - rint(turns));  // [-1/2, 1/2]
    *c = factor * cospif(2.0f * t);
    *s = factor * sinpif(2.0f * t);
}

// One workgroup per token. The angles of its R / 2 pairs are computed once, into LDS, and serve
// every query and key head; the heads' values move in 16-byte pieces: `u` rotated pieces of a head
// (LAYOUT half: 8 pairs, read and written as two pieces R / 2 apart; interleaved: 4 pairs, one
// piece), then the pieces past R and the value heads, copied. ANY: heads whose R does not fall on
// those pieces (R % 16 for the half layout, R % 8 for the interleaved), see rotate_any. (8 prompts
// of up to 2048 tokens, 32 + 8 + 8 heads of 96: R = 32 55 us, halves of 12 67, 36 interleaved 54;
// element by element 90 and 94.)
enum { kHalf = 0, kInterleaved = 1, kAny = 2 };
constexpr int kThreads = 256;
constexpr int kMaxPairs = 128;

typedef uint32_t uintx4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ void unpack8(const uint16_t *p, float *v) {
    const uintx4_t w = *reinterpret_cast<const uintx4_t *>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void pack8(uint16_t *p, const float *v) {
    uintx4_t w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uintx4_t *>(p) = w;
}

// Elements d .. d + 7 of a head at any even R. The half layout's partners stand R / 2 before or
// after: 16 bytes at any alignment, of both sides where the eight lie in both halves. Those of the
// second half may pass the head's end, into the value heads that follow; those of the first may
// begin before it: `lead`, the row has elements before this head, else they are read one by one.
__device__ __forceinline__ void rotate_any(const uint16_t *src, uint16_t *dst, int d, int R,
                                           int interleaved, bool lead, const float *cosine,
                                           const float *sine) {
    typedef uint32_t uintx4_any_t __attribute__((ext_vector_type(4), aligned(2), may_alias));
    const uintx4_t own = *reinterpret_cast<const uintx4_t *>(src + d);
    const int half = R / 2;
    uint32_t x[8], other[8], out[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = own[i / 2] >> 16 * (i % 2) & 0xFFFFu;
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) other[i] = x[i ^ 1];
    } else {
        uintx4_t after = own, before = own;
        if (d < half) after = *reinterpret_cast<const uintx4_any_t *>(src + d + half);
        if (d >= half || (d + 8 > half && lead))
            before = *reinterpret_cast<const uintx4_any_t *>(src + d - half);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            other[i] = (d + i < half ? after : before)[i / 2] >> 16 * (i % 2) & 0xFFFFu;
        if (d < half && d + 8 > half && !lead) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (d + i >= half) other[i] = src[d + i - half];
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int e = min(d + i, R - 1);
        const bool first = interleaved ? i % 2 == 0 : e < half;
        const int pair = interleaved ? e / 2 : first ? e : e - half;
        const float a = bf16_to_f32(x[i]) * cosine[pair], b = bf16_to_f32(other[i]) * sine[pair];
        out[i] = d + i < R ? to_bf16(first ? a - b : b + a) : x[i];
    }
    const uintx4_t w = {out[0] | out[1] << 16, out[2] | out[3] << 16, out[4] | out[5] << 16,
                        out[6] | out[7] << 16};
    *reinterpret_cast<uintx4_t *>(dst + d) = w;
}

template <int MODE>
__global__ void __launch_bounds__(kThreads) rope_append_kernel(
    const uint16_t *__restrict__ qkv, int64_t ldqkv, int n_heads,
    const int32_t *__restrict__ q_start, const float *__restrict__ inv_freq, int rot_dim,
    int interleaved, float factor, KvView c, uint16_t *__restrict__ q, int64_t ldq,
    int width_shift) {
    __shared__ float cosine[kMaxPairs], sine[kMaxPairs];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x, D = c.head_dim, half = rot_dim / 2;
    RowPlace at;
    if (!place_of_row(c, q_start, static_cast<int>(t), &at)) return;
    for (int i = tid; i < half; i += blockDim.x)
        turn(at.pos, inv_freq[i], factor, &cosine[i], &sine[i]);
    // the token's slot in the cache, if it is appended
    int64_t slot = -1;
    if (at.pos >= 0) {
        const int page = c.table[at.seq * c.ld_table + (at.pos >> c.page_shift)];
        if (page >= 0 && page < c.n_pages)
            slot = static_cast<int64_t>(page) * c.page_stride +
                   static_cast<int64_t>((at.pos & c.page_mask) * c.slot_stride);
    }
    __syncthreads();
    // threads over (head, piece): 2^width_shift of them a head
    const int piece0 = tid & ((1 << width_shift) - 1);
    const int n_rotate = n_heads + c.n_kv;
    for (int h = tid >> width_shift; h < n_rotate + c.n_kv; h += blockDim.x >> width_shift) {
        const uint16_t *src = qkv + t * ldqkv + static_cast<int64_t>(h) * D;
        uint16_t *dst = q + t * ldq + static_cast<int64_t>(h) * D;
        if (h >= n_heads) {
            if (slot < 0) break;
            const int hk = h - n_heads;
            dst = hk < c.n_kv ? c.k + slot + static_cast<int64_t>(hk) * c.head_stride
                              : c.v + slot + static_cast<int64_t>(hk - c.n_kv) * c.head_stride;
        }
        const int rotated = h < n_rotate ? (MODE == kHalf ? half / 8 : rot_dim / 8) : 0;
        const int pieces = h < n_rotate ? rotated + (D - rot_dim) / 8 : D / 8;
        if (MODE == kAny && h < n_rotate) {
            for (int p = piece0; p < D / 8; p += 1 << width_shift)
                rotate_any(src, dst, 8 * p, rot_dim, interleaved, h > 0, cosine, sine);
            continue;
        }
        for (int p = piece0; p < pieces; p += 1 << width_shift) {
            if (p >= rotated) {
                const int d = (h < n_rotate ? rot_dim : 0) + 8 * (p - rotated);
                *reinterpret_cast<uintx4_t *>(dst + d) =
                    *reinterpret_cast<const uintx4_t *>(src + d);
            } else if (MODE == kHalf) {
                float a[8], b[8], x[8], y[8];
                unpack8(src + 8 * p, a);
                unpack8(src + 8 * p + half, b);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float cs = cosine[8 * p + i], sn = sine[8 * p + i];
                    x[i] = a[i] * cs - b[i] * sn;
                    y[i] = a[i] * sn + b[i] * cs;
                }
                pack8(dst + 8 * p, x);
                pack8(dst + 8 * p + half, y);
            } else {
                float a[8], x[8];
                unpack8(src + 8 * p, a);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float cs = cosine[4 * p + i], sn = sine[4 * p + i];
                    x[2 * i] = a[2 * i] * cs - a[2 * i + 1] * sn;
                    x[2 * i + 1] = a[2 * i] * sn + a[2 * i + 1] * cs;
                }
                pack8(dst + 8 * p, x);
            }
        }
    }
}

template <int MODE, typename... Args>
hipError_t launch(int64_t T, int threads, hipStream_t stream, Args... args) {
    hipLaunchKernelGGL(rope_append_kernel<MODE>, dim3(static_cast<unsigned>(T)), dim3(threads), 0,
                       stream, args...);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rope_append(const uint16_t *qkv, int64_t T, int64_t ldqkv, int n_heads,
                              const int32_t *q_start, const float *inv_freq, int rot_dim,
                              bool interleaved, float factor, const KvView &c, uint16_t *q,
                              int64_t ldq, hipStream_t stream) {
    const int mode = rot_dim % (interleaved ? 8 : 16) != 0 ? kAny : interleaved ? kInterleaved
                                                                                : kHalf;
    // threads a head: a power of two that covers its pieces
    const int pieces = mode == kHalf ? (c.head_dim - rot_dim / 2) / 8 : c.head_dim / 8;
    int shift = 0;
    while ((1 << shift) < pieces) ++shift;
    int threads = (n_heads + 2 * c.n_kv) << shift;
    threads = threads >= kThreads ? kThreads : (threads + kWave - 1) / kWave * kWave;
    if (T > static_cast<int64_t>(kMaxThreads) / threads) threads = kThreads / 2;  // (T = 2^24)
    const int il = interleaved ? 1 : 0;
    if (mode == kHalf)
        return launch<kHalf>(T, threads, stream, qkv, ldqkv, n_heads, q_start, inv_freq, rot_dim,
                             il, factor, c, q, ldq, shift);
    if (mode == kInterleaved)
        return launch<kInterleaved>(T, threads, stream, qkv, ldqkv, n_heads, q_start, inv_freq,
                                    rot_dim, il, factor, c, q, ldq, shift);
    return launch<kAny>(T, threads, stream, qkv, ldqkv, n_heads, q_start, inv_freq, rot_dim, il,
                        factor, c, q, ldq, shift);
}

}  // namespace w4
