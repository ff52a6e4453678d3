// Headwise QK-Norm with the position rotation in the same pass, its gradient,
// and the append of rotated keys and of values to a paged cache (element type
// or 4 bits).  Declared in include/qknorm.h.
//
// Mathematics, per head x of head_dim elements at position pos:
//   S = sum_j x_j^2,  r = 1 / sqrt(S / head_dim + eps),  n_j = (x_j * gamma_j) * r
//   y = R(pos) n: for pair i < rotary_dim / 2, (a, b) the pair's elements,
//     a' = a cos_i - b sin_i,  b' = a sin_i + b cos_i  (cos, sin: the table's row pos);
//   elements from rotary_dim on are not rotated.
// Gradient: u = R(pos)^T dy, M = sum_j u_j gamma_j x_j,
//   dx_j = r * (u_j gamma_j - x_j * r^2 * M / head_dim),  dgamma_j = sum over heads and tokens of u_j x_j r.
// 4 bits: a group of 64 elements has s = fp16(max |y| / 7) and codes
//   clamp(rint(y / s), -7, 7).
//
// The vector kernels read each element once and write it once (the gradient reads
// two rows and writes one); memory traffic bounds the rotation, its gradient and
// the element append, instructions the 4-bit append.  The element-wise kernels
// read a head twice, the second time from cache.
#include <cuda_runtime.h>
#include <stdint.h>

#include "qknorm.h"
#include "qknorm_checks.cuh"
#include "qknorm_kernels.cuh"
#include "qknorm_rope.cuh"

namespace qkn {
namespace {

// A position's rotation: inside the table, padding (negative: the row becomes
// zeros) or past the table (the row becomes NaN; nothing is read past it).
enum Turn : int { kTurnRow = 0, kTurnPad = 1, kTurnPast = 2 };
__device__ __forceinline__ int turn_of(int64_t pos, int64_t rows) {
    return pos < 0 ? kTurnPad : (pos >= rows ? kTurnPast : kTurnRow);
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}

template <typename E>
__device__ __forceinline__ float elem_at(const char *row, int i) {
    return Elem<E>::to_float(reinterpret_cast<const typename Elem<E>::Bits *>(row)[i]);
}
template <typename E>
__device__ __forceinline__ void put_elem(char *row, int i, float v) {
    reinterpret_cast<typename Elem<E>::Bits *>(row)[i] = Elem<E>::from_float(v);
}

__device__ __forceinline__ float norm_factor(float s, const RopeParams &p) { return rms_factor(s, p.inv_d, p.eps); }
__device__ __forceinline__ double norm_factor(double s, const RopeParams &p) {
    return 1.0 / sqrt(s / static_cast<double>(p.head_dim) + static_cast<double>(p.eps));
}

// ----------------------------------------------------------------------------
// 4-bit codes in 64 bits.  Scales and codes are the rounded values of the formula
// whatever the order of the head's sums, so that a token's cache entry does not
// depend on the kernel variant that wrote it: 32 bits alone put about one code in
// a million on the other side of its border.  The vector kernel decides in 32
// bits where their error allows it and comes here otherwise (4096 tokens, 8 heads
// of 128: 34 us for the append; 67 us with every key in 64 bits).
__device__ __forceinline__ __half kv4_scale(double amax, bool bad) {
    if (bad) return __ushort_as_half(0x7FFFu);  // a NaN or infinity in the group: the group reads as NaN
    return __double2half(fmin(amax / 7.0, 65504.0));
}
// `inv` = 1 / s.  The product decides except next to a border, where the
// quotient does (exact ties are common: x and s have few bits).
__device__ __forceinline__ uint32_t kv4_code(double y, double s, double inv) {
    double t = y * inv;
    double k = rint(t);
    if (fabs(fabs(t - k) - 0.5) < 1e-9) k = rint(y / s);
    k = fmin(fmax(k, -7.0), 7.0);
    return static_cast<uint32_t>(static_cast<int>(k) + 8);
}

// ----------------------------------------------------------------------------
// Any size, stride and alignment: one warp per head, element accesses, the
// head read twice (the second time from cache).  C: the arithmetic's type.  (The
// prompt that the vector kernel turns in 16.5 us takes 81 us here.)
template <typename E, typename C>
struct ScalarHead {
    const RopeParams &p;
    const char *row, *gamma;
    const float *cs;  // the table's row, null unless `turn` is kTurnRow
    C r;
    int turn;

    __device__ __forceinline__ C normed(int i) const {
        const C x = static_cast<C>(elem_at<E>(row, i));
        if (!gamma) return x;
        return x * static_cast<C>(elem_at<typename Elem<E>::G>(gamma, i)) * r;
    }
    __device__ __forceinline__ void pair(int i, int &i0, int &i1, C &a, C &b) const {
        i0 = p.interleaved ? 2 * i : i;
        i1 = p.interleaved ? 2 * i + 1 : i + p.half;
        const C x = normed(i0), y = normed(i1);
        const C c = static_cast<C>(cs[i]), s = static_cast<C>(cs[i + p.half]);
        a = x * c - y * s;
        b = x * s + y * c;
    }
    // f(i, value) for every element of the head, each by one lane.
    template <typename F>
    __device__ __forceinline__ void each(int lane, F f) const {
        if (turn != kTurnRow) {
            const C v = turn == kTurnPad ? C(0) : C(__uint_as_float(0x7FFFFFFFu));
            for (int i = lane; i < p.head_dim; i += 32) f(i, v);
            return;
        }
        for (int i = lane; i < p.half; i += 32) {
            int i0, i1;
            C a, b;
            pair(i, i0, i1, a, b);
            f(i0, a);
            f(i1, b);
        }
        for (int i = 2 * p.half + lane; i < p.head_dim; i += 32) f(i, normed(i));
    }
};

template <typename E, typename C>
__device__ __forceinline__ ScalarHead<E, C> scalar_head(const RopeParams &p, const char *row, const char *gamma,
                                                        int64_t t, int lane) {
    C s = C(0);
    if (gamma)
        for (int i = lane; i < p.head_dim; i += 32) {
            const C x = static_cast<C>(elem_at<E>(row, i));
            s = fma(x, x, s);
        }
    s = warp_sum(s);
    const int64_t pos = p.positions[t];
    const int turn = turn_of(pos, p.table_rows);
    return ScalarHead<E, C>{p, row, gamma, turn == kTurnRow ? p.table + pos * 2 * p.half : nullptr, norm_factor(s, p), turn};
}

__device__ __forceinline__ int tensor_of(const RopeParams &p, int &h) {
    if (h < p.heads[0]) return 0;
    h -= p.heads[0];
    if (h < p.heads[1]) return 1;
    h -= p.heads[1];
    return 2;
}

// One head of K (which = 1) or V into the 4-bit cache by a whole warp, in 64
// bits; `y` holds the head.  Out of line: the vector kernel comes here for the
// few heads with a scale or code next to a border, and should not pay for it in
// registers.
template <typename E>
__device__ __noinline__ void quantise_head(const RopeParams &p, int which, int64_t t, const char *row, double *y,
                                           uint8_t *codes, __half *scales) {
    const int lane = threadIdx.x & 31;
    if (which == 1) {
        const auto head = scalar_head<E, double>(p, row, p.gamma[1], t, lane);
        head.each(lane, [&](int i, double v) { y[i] = v; });
    } else {
        for (int i = lane; i < p.head_dim; i += 32) y[i] = static_cast<double>(elem_at<E>(row, i));
    }
    __syncwarp();
    for (int g = 0; g < p.head_dim / kKv4Group; ++g) {
        const double a = y[g * kKv4Group + 2 * lane], b = y[g * kKv4Group + 2 * lane + 1];
        double m = fmax(fabs(a), fabs(b));
        const bool bad = __any_sync(0xFFFFFFFFu, !isfinite(a) || !isfinite(b));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        const __half sh = kv4_scale(m, bad);
        const double s = static_cast<double>(__half2float(sh));
        const bool zero = !(s > 0.0);
        const double inv = 1.0 / s;
        const uint32_t lo = zero ? 8u : kv4_code(a, s, inv), hi = zero ? 8u : kv4_code(b, s, inv);
        codes[g * (kKv4Group / 2) + lane] = static_cast<uint8_t>(lo | (hi << 4));
        if (lane == 0) scales[g] = sh;
    }
    __syncwarp();
}

constexpr int kScalarWarps = 8;

template <typename E, int SINK>
__global__ void __launch_bounds__(kScalarWarps * 32) heads_scalar_kernel(const __grid_constant__ RopeParams p) {
    pdl_wait_and_release();
    __shared__ double held[SINK == kSinkKv4 ? kScalarWarps : 1][SINK == kSinkKv4 ? 256 : 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t rows = p.T * p.heads_total;
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * kScalarWarps + warp; item < rows;
         item += static_cast<int64_t>(gridDim.x) * kScalarWarps) {
        const int64_t t = item / p.heads_total;
        int h = static_cast<int>(item - t * p.heads_total);
        const int which = tensor_of(p, h);
        const int64_t head_bytes = static_cast<int64_t>(p.head_dim) * sizeof(typename Elem<E>::Bits);
        const char *row = p.in[which] + t * p.stride[which] + h * head_bytes;
        if (which == 0 || SINK == kSinkRows) {
            char *out = p.out[which] + t * p.stride[which] + h * head_bytes;
            const auto head = scalar_head<E, float>(p, row, p.gamma[which], t, lane);
            head.each(lane, [&](int i, float v) { put_elem<E>(out, i, v); });
            continue;
        }
        const int64_t slot = p.slots[t];
        if (slot < 0 || slot >= p.num_slots) continue;
        const int64_t page = slot / p.page_size, off = slot - page * p.page_size;
        const int kv = which - 1;
        if constexpr (SINK == kSinkCache) {
            char *out = p.cache[kv] + page * p.page_stride[kv] + off * p.token_stride[kv] + h * p.head_stride[kv];
            if (which == 1) {
                const auto head = scalar_head<E, float>(p, row, p.gamma[1], t, lane);
                head.each(lane, [&](int i, float v) { put_elem<E>(out, i, v); });
            } else {
                using B = typename Elem<E>::Bits;
                for (int i = lane; i < p.head_dim; i += 32)
                    reinterpret_cast<B *>(out)[i] = reinterpret_cast<const B *>(row)[i];
            }
        }
        if constexpr (SINK == kSinkKv4) {
            const int64_t cell = (page * p.heads[1] + h) * p.page_size + off;
            quantise_head<E>(p, which, t, row, held[warp], reinterpret_cast<uint8_t *>(p.cache[kv]) + cell * (p.head_dim / 2),
                             p.scales[kv] + cell * (p.head_dim / kKv4Group));
        }
    }
}

// ----------------------------------------------------------------------------
// Gradient, any size and alignment: one warp per head; each warp sums dgamma
// in its own shared memory and the CTA's sums are added in a fixed order.
constexpr int kGradScalarWarps = 4;

template <typename E>
__global__ void __launch_bounds__(kGradScalarWarps * 32) heads_grad_scalar_kernel(const __grid_constant__ RopeGradParams p) {
    pdl_wait_and_release();
    extern __shared__ float sums[];  // [warps][2][head_dim]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int D = p.head_dim;
    float *mine = sums + warp * 2 * D;
    for (int i = lane; i < 2 * D; i += 32) mine[i] = 0.0f;
    __syncwarp();
    const int total = p.heads[0] + p.heads[1];
    const int64_t rows = p.T * total;
    const int64_t head_bytes = static_cast<int64_t>(D) * sizeof(typename Elem<E>::Bits);
    for (int64_t item = static_cast<int64_t>(blockIdx.x) * kGradScalarWarps + warp; item < rows;
         item += static_cast<int64_t>(gridDim.x) * kGradScalarWarps) {
        const int64_t t = item / total;
        int h = static_cast<int>(item - t * total);
        const int w = h < p.heads[0] ? 0 : 1;
        if (w) h -= p.heads[0];
        const char *x = p.x[w] + t * p.x_stride[w] + h * head_bytes;
        const char *dy = p.dy[w] + t * p.dy_stride[w] + h * head_bytes;
        char *dx = p.dx[w] + t * p.dx_stride[w] + h * head_bytes;
        const char *gamma = p.gamma[w];
        const int64_t pos = p.positions[t];
        const int turn = turn_of(pos, p.table_rows);
        if (turn != kTurnRow) {
            const float v = turn == kTurnPad ? 0.0f : __uint_as_float(0x7FFFFFFFu);
            for (int i = lane; i < D; i += 32) {
                put_elem<E>(dx, i, v);
                mine[w * D + i] += v;
            }
            continue;
        }
        const float *cs = p.table + pos * 2 * p.half;
        auto each = [&](auto f) {  // f(i, u_i)
            for (int i = lane; i < p.half; i += 32) {
                const int i0 = p.interleaved ? 2 * i : i, i1 = p.interleaved ? 2 * i + 1 : i + p.half;
                const float a = elem_at<E>(dy, i0), b = elem_at<E>(dy, i1), c = cs[i], s = cs[i + p.half];
                f(i0, a * c + b * s);
                f(i1, b * c - a * s);
            }
            for (int i = 2 * p.half + lane; i < D; i += 32) f(i, elem_at<E>(dy, i));
        };
        float S = 0.0f, M = 0.0f;
        each([&](int i, float u) {
            const float v = elem_at<E>(x, i);
            S = fmaf(v, v, S);
            M = fmaf(u * elem_at<E>(gamma, i), v, M);
        });
        S = qkn::warp_sum(S);
        M = qkn::warp_sum(M);
        const float r = rms_factor(S, p.inv_d, p.eps);
        const float c = r * r * M * p.inv_d;
        // dx may be dy: a lane reads both elements of a pair before it writes them
        for (int i = lane; i < p.half; i += 32) {
            const int i0 = p.interleaved ? 2 * i : i, i1 = p.interleaved ? 2 * i + 1 : i + p.half;
            const float a = elem_at<E>(dy, i0), b = elem_at<E>(dy, i1), cc = cs[i], s = cs[i + p.half];
            const float u0 = a * cc + b * s, u1 = b * cc - a * s;
            const float x0 = elem_at<E>(x, i0), x1 = elem_at<E>(x, i1);
            put_elem<E>(dx, i0, r * (u0 * elem_at<E>(gamma, i0) - x0 * c));
            put_elem<E>(dx, i1, r * (u1 * elem_at<E>(gamma, i1) - x1 * c));
            mine[w * D + i0] += u0 * x0 * r;
            mine[w * D + i1] += u1 * x1 * r;
        }
        for (int i = 2 * p.half + lane; i < D; i += 32) {
            const float u = elem_at<E>(dy, i), v = elem_at<E>(x, i);
            put_elem<E>(dx, i, r * (u * elem_at<E>(gamma, i) - v * c));
            mine[w * D + i] += u * v * r;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * D; i += blockDim.x) {
        float s = 0.0f;
        for (int w = 0; w < kGradScalarWarps; ++w) s += sums[w * 2 * D + i];
        p.partial[static_cast<int64_t>(blockIdx.x) * 2 * D + i] = s;
    }
}

// ----------------------------------------------------------------------------
// Aligned heads: a head is held by p.lanes lanes (a power of two), each with
// two 16-byte vectors placed so that a pair never leaves its lane: vectors u and
// u + rotary_dim / 2 where pairs are (i, i + rotary_dim / 2), any two where they
// are neighbours (those are sorted into first and second elements as they are
// loaded, so that one code turns both).  A warp takes 32 / lanes heads at a time
// of one token and one tensor, several times, the next heads' loads ahead of the
// work on the ones at hand.  What the norm and the
// rotation multiply an element by, but for r, is the same for all of them:
//   a' = r (x_a (gamma_a cos) - x_b (gamma_b sin)),
//   b' = r (x_a (gamma_a sin) + x_b (gamma_b cos)),
// so those four factors of a pair are formed once, and a pair costs four packed
// operations and one by r.
template <typename E>
struct LanePlace {
    int lo, hi;            // first elements of the two vectors
    int pair_lo, pair_hi;  // pairs of the first and second half of the lane's V pairs, negative: not turned
};
template <typename E, typename P>
__device__ __forceinline__ LanePlace<E> lane_place(const P &p, int u) {
    constexpr int V = Elem<E>::kPerVec;
    if (p.interleaved) {
        const int lo = u * V, hi = p.head_dim / 2 + u * V;
        return {lo, hi, lo < 2 * p.half ? lo / 2 : -1, hi < 2 * p.half ? hi / 2 : -1};
    }
    const int nr = p.half / V;
    if (u < nr) return {u * V, p.half + u * V, u * V, u * V + V / 2};
    const int lo = 2 * p.half + 2 * (u - nr) * V;
    return {lo, lo + V, -1, -1};
}

// Neighbouring pairs (x0, x1), (x2, x3), ..: a <- first elements, b <- second, and back.
template <typename E>
__device__ __forceinline__ void part_pairs(uint4 &a, uint4 &b) {
    if constexpr (sizeof(typename Elem<E>::Bits) == 4) {
        const uint4 x = a, y = b;
        a = make_uint4(x.x, x.z, y.x, y.z);
        b = make_uint4(x.y, x.w, y.y, y.w);
    } else {
        constexpr uint32_t first = sizeof(typename Elem<E>::Bits) == 2 ? 0x5410u : 0x6420u;
        constexpr uint32_t second = sizeof(typename Elem<E>::Bits) == 2 ? 0x7632u : 0x7531u;
        const uint4 x = a, y = b;
        a = make_uint4(__byte_perm(x.x, x.y, first), __byte_perm(x.z, x.w, first), __byte_perm(y.x, y.y, first),
                       __byte_perm(y.z, y.w, first));
        b = make_uint4(__byte_perm(x.x, x.y, second), __byte_perm(x.z, x.w, second), __byte_perm(y.x, y.y, second),
                       __byte_perm(y.z, y.w, second));
    }
}
template <typename E>
__device__ __forceinline__ void join_pairs(uint4 &a, uint4 &b) {
    const uint4 x = a, y = b;
    if constexpr (sizeof(typename Elem<E>::Bits) == 4) {
        a = make_uint4(x.x, y.x, x.y, y.y);
        b = make_uint4(x.z, y.z, x.w, y.w);
    } else {
        constexpr uint32_t low = sizeof(typename Elem<E>::Bits) == 2 ? 0x5410u : 0x5140u;
        constexpr uint32_t high = sizeof(typename Elem<E>::Bits) == 2 ? 0x7632u : 0x7362u;
        a = make_uint4(__byte_perm(x.x, y.x, low), __byte_perm(x.x, y.x, high), __byte_perm(x.y, y.y, low),
                       __byte_perm(x.y, y.y, high));
        b = make_uint4(__byte_perm(x.z, y.z, low), __byte_perm(x.z, y.z, high), __byte_perm(x.w, y.w, low),
                       __byte_perm(x.w, y.w, high));
    }
}

// Cosines and sines of the lane's V pairs (1 and 0 where it turns nothing).
template <typename E, typename P>
__device__ __forceinline__ void lane_turns(const P &p, const LanePlace<E> &at, const float *cs, float (&c)[Elem<E>::kPerVec],
                                           float (&s)[Elem<E>::kPerVec]) {
    constexpr int H = Elem<E>::kPerVec / 2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int pair = h ? at.pair_hi : at.pair_lo;
#pragma unroll
        for (int i = 0; i < H; ++i) c[h * H + i] = 1.0f, s[h * H + i] = 0.0f;
        if (pair < 0) continue;
        if constexpr (H >= 4) {
#pragma unroll
            for (int i = 0; i < H; i += 4) {
                const float4 x = __ldg(reinterpret_cast<const float4 *>(cs + pair + i));
                const float4 y = __ldg(reinterpret_cast<const float4 *>(cs + p.half + pair + i));
                c[h * H + i] = x.x, c[h * H + i + 1] = x.y, c[h * H + i + 2] = x.z, c[h * H + i + 3] = x.w;
                s[h * H + i] = y.x, s[h * H + i + 1] = y.y, s[h * H + i + 2] = y.z, s[h * H + i + 3] = y.w;
            }
        } else {
            const float2 x = __ldg(reinterpret_cast<const float2 *>(cs + pair));
            const float2 y = __ldg(reinterpret_cast<const float2 *>(cs + p.half + pair));
            c[h * H] = x.x, c[h * H + 1] = x.y, s[h * H] = y.x, s[h * H + 1] = y.y;
        }
    }
}

template <typename E>
__device__ __forceinline__ void widen_floats(const uint4 &v, float (&x)[Elem<E>::kPerVec]) {
    F2 w[Elem<E>::kPerVec / 2];
    Elem<E>::widen(v, w);
#pragma unroll
    for (int i = 0; i < Elem<E>::kPerVec / 2; ++i) {
        x[2 * i] = f2_lo(w[i]);
        x[2 * i + 1] = f2_hi(w[i]);
    }
}
// gamma of the lane's first and second elements of its pairs.
template <typename E>
__device__ __forceinline__ void lane_gamma(const char *gamma, const LanePlace<E> &at, bool interleaved,
                                           float (&ga)[Elem<E>::kPerVec], float (&gb)[Elem<E>::kPerVec]) {
    using GE = typename Elem<E>::G;
    constexpr int V = Elem<E>::kPerVec, KG = Elem<E>::kGVecs, N = Elem<GE>::kPerVec;
#pragma unroll
    for (int v = 0; v < KG; ++v) {
        float x[N], y[N];
        widen_floats<GE>(ld_gamma(gamma + static_cast<int64_t>(at.lo) * sizeof(GE) + 16 * v), x);
        widen_floats<GE>(ld_gamma(gamma + static_cast<int64_t>(at.hi) * sizeof(GE) + 16 * v), y);
#pragma unroll
        for (int i = 0; i < N; ++i) ga[v * N + i] = x[i], gb[v * N + i] = y[i];
    }
    if (interleaved) {
        float x[V], y[V];
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = ga[i], y[i] = gb[i];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            ga[i] = x[2 * i], gb[i] = x[2 * i + 1];
            ga[V / 2 + i] = y[2 * i], gb[V / 2 + i] = y[2 * i + 1];
        }
    }
}
// Over the lanes of a head: L of them, or `lanes` where L is 0.
template <int L = 0, typename C>
__device__ __forceinline__ C lanes_sum(C v, int lanes) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        if (off < (L > 0 ? L : lanes)) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, off));
    return v;
}

// The factors of a lane's pairs: a' = x_a aa + x_b ab, b' = x_a ba + x_b bb.
template <int N>
struct PairFactors {
    F2 aa[N], ab[N], ba[N], bb[N];
};
template <typename E>
__device__ __forceinline__ PairFactors<Elem<E>::kPerVec / 2> pair_factors(const RopeParams &p, const LanePlace<E> &at,
                                                                          const char *gamma, const float *cs) {
    constexpr int V = Elem<E>::kPerVec;
    float c[V], s[V], ga[V], gb[V];
    lane_turns<E>(p, at, cs, c, s);
    if (gamma) {
        lane_gamma<E>(gamma, at, p.interleaved, ga, gb);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) ga[i] = gb[i] = 1.0f;
    }
    PairFactors<V / 2> f;
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        f.aa[i] = f2(ga[2 * i] * c[2 * i], ga[2 * i + 1] * c[2 * i + 1]);
        f.ab[i] = f2(-gb[2 * i] * s[2 * i], -gb[2 * i + 1] * s[2 * i + 1]);
        f.ba[i] = f2(ga[2 * i] * s[2 * i], ga[2 * i + 1] * s[2 * i + 1]);
        f.bb[i] = f2(gb[2 * i] * c[2 * i], gb[2 * i + 1] * c[2 * i + 1]);
    }
    return f;
}

// Whether the lane turns its pair i (of packed pairs: 2i and 2i + 1).  Elements
// it does not turn are not mixed either: a neighbour's infinity stays there.
template <typename E>
__device__ __forceinline__ bool turned(const LanePlace<E> &at, int i, int n) {
    return (i < n / 2 ? at.pair_lo : at.pair_hi) >= 0;
}

// One head: the lane's parted vectors to normed and turned elements.  Returns r
// (1 without a norm).
template <typename E, int L>
__device__ __forceinline__ float lane_forward(const RopeParams &p, const LanePlace<E> &at, bool norm,
                                             const PairFactors<Elem<E>::kPerVec / 2> &f, const uint4 &va, const uint4 &vb,
                                             F2 (&a)[Elem<E>::kPerVec / 2], F2 (&b)[Elem<E>::kPerVec / 2]) {
    constexpr int N = Elem<E>::kPerVec / 2;
    F2 x[N], y[N];
    Elem<E>::widen(va, x);
    Elem<E>::widen(vb, y);
    float r = 1.0f;
    if (norm) {
        F2 sum = mul2(x[0], x[0]), other = mul2(y[0], y[0]);
#pragma unroll
        for (int i = 1; i < N; ++i) {
            sum = fma2(x[i], x[i], sum);
            other = fma2(y[i], y[i], other);
        }
        r = rms_factor(lanes_sum<L>((f2_lo(sum) + f2_hi(sum)) + (f2_lo(other) + f2_hi(other)), p.lanes), p.inv_d, p.eps);
    }
    const F2 rr = f2(r, r);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        F2 fa = mul2(x[i], f.aa[i]), fb = mul2(y[i], f.bb[i]);
        if (turned(at, i, N)) {
            fa = fma2(y[i], f.ab[i], fa);
            fb = fma2(x[i], f.ba[i], fb);
        }
        a[i] = mul2(fa, rr);
        b[i] = mul2(fb, rr);
    }
    return r;
}

// ----------------------------------------------------------------------------
// Codes (+ 8, in the low four bits) of a lane's pairs, packed and stored.
template <typename E>
__device__ __forceinline__ void store_codes(bool interleaved, uint8_t *codes, const LanePlace<E> &at,
                                            const uint32_t (&ca)[Elem<E>::kPerVec], const uint32_t (&cb)[Elem<E>::kPerVec]) {
    constexpr int V = Elem<E>::kPerVec;
    uint32_t lo = 0, hi = 0;
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            lo |= (ca[i] & 15u) << (8 * i) | (cb[i] & 15u) << (8 * i + 4);
            hi |= (ca[V / 2 + i] & 15u) << (8 * i) | (cb[V / 2 + i] & 15u) << (8 * i + 4);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            lo |= (ca[i] & 15u) << (4 * i);
            hi |= (cb[i] & 15u) << (4 * i);
        }
    }
    if constexpr (V == 8) {
        *reinterpret_cast<uint32_t *>(codes + at.lo / 2) = lo;
        *reinterpret_cast<uint32_t *>(codes + at.hi / 2) = hi;
    } else {
        *reinterpret_cast<uint16_t *>(codes + at.lo / 2) = static_cast<uint16_t>(lo);
        *reinterpret_cast<uint16_t *>(codes + at.hi / 2) = static_cast<uint16_t>(hi);
    }
}

__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ float max_abs(float m, F2 x) { return fmaxf(m, fmaxf(fabsf(f2_lo(x)), fabsf(f2_hi(x)))); }
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// In 32 bits.  With `formed` the elements carry the error of a norm and turn in
// 32 bits, u = 2^-24: at most 10 u of the element (the squared sum's 11
// additions halved, 4 for the root's 2 ulp, one for the last product) and 4 u of
// the head's largest (two roundings of each product times |a cos| + |b sin| <=
// sqrt(2) that largest, and one of their sum).  That holds for an r in (0, 2^50):
// r is 0 where the squared sum has passed fp32's largest number, and from 2^50
// on squares, or elements before their product with r, may have been subnormals,
// which have fewer bits.  Returns the lanes (as a mask) for whose heads a scale
// or a code lies nearer than that to a border, so that 64 bits have to decide, r
// lies outside, or a scale is outside fp16's normal range; nothing of those heads
// is stored.
template <typename E, int L>
__device__ __forceinline__ uint32_t lane_quantise(const RopeParams &p, bool formed, float r, int u, bool there, const LanePlace<E> &at,
                                              const F2 (&a)[Elem<E>::kPerVec / 2], const F2 (&b)[Elem<E>::kPerVec / 2],
                                              uint8_t *codes, __half *scales) {
    constexpr int V = Elem<E>::kPerVec, N = V / 2, H = N / 2;
    constexpr float kU = 5.9604645e-8f;
    // largest of the first and second halves of the pairs' first and second elements
    float m[4] = {};
    F2 zero = f2(0.0f, 0.0f);  // NaN with any element that is not finite
#pragma unroll
    for (int i = 0; i < N; ++i) {
        m[i / H] = max_abs(m[i / H], a[i]);
        m[2 + i / H] = max_abs(m[2 + i / H], b[i]);
        zero = fma2(a[i], f2(0.0f, 0.0f), zero);
        zero = fma2(b[i], f2(0.0f, 0.0f), zero);
    }
    const bool inter = p.interleaved;
    const float mlo = fmaxf(m[0], inter ? m[2] : m[1]), mhi = fmaxf(inter ? m[1] : m[2], m[3]);
    const float err = formed ? 4.0f * kU * lanes_max<L>(fmaxf(mlo, mhi)) : 0.0f;
    const float own = formed ? 10.0f * kU : 0.0f;
    constexpr int groups = L * 2 * V / kKv4Group;  // the lanes hold the head exactly
    const int group_lo = at.lo / kKv4Group, group_hi = at.hi / kKv4Group;
    bool near = f2_lo(zero) != 0.0f || f2_hi(zero) != 0.0f || !(r > 0.0f && r < 1.125899907e15f);
    float slo = 0.0f, shi = 0.0f;
    __half held = __float2half(0.0f);
#pragma unroll
    for (int g = 0; g < groups; ++g) {
        const float top = lanes_max<L>(fmaxf(group_lo == g ? mlo : 0.0f, group_hi == g ? mhi : 0.0f));
        const float q = top * 0.142857149f;
        // fp16 rounds at the middle of q's low 13 bits; kU q is at most one step of q, and q is off by
        // three such steps besides top's error
        const float steps = fabsf(static_cast<float>(static_cast<int>(__float_as_uint(q) & 0x1FFFu) - 0x1000));
        if (top > 0.0f && (!(q >= 1.220703125e-4f && q < 65000.0f) || steps * (kU * q) <= err * 0.15f + (own + 3.0f * kU) * q))
            near = true;
        const __half sh = __float2half_rn(q);
        const float s = __half2float(sh);
        if (group_lo == g) slo = s;
        if (group_hi == g) shi = s;
        if (u == g) held = sh;
    }
    const float ilo = slo > 0.0f ? rcp_approx(slo) : 0.0f, ihi = shi > 0.0f ? rcp_approx(shi) : 0.0f;
    const float ia1 = inter ? ihi : ilo, ib0 = inter ? ilo : ihi;
    // + 1.5 * 2^23 + 8: the nearest integer, 8 added, in the low bits
    const F2 magic = f2(12582920.0f, 12582920.0f), back = f2(-12582920.0f, -12582920.0f), minus = f2(-1.0f, -1.0f);
    float d[4] = {};
    uint32_t ca[V], cb[V];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float fa = i < H ? ilo : ia1, fb = i < H ? ib0 : ihi;
        const F2 ta = mul2(a[i], f2(fa, fa)), tb = mul2(b[i], f2(fb, fb));
        const F2 ka = add2(ta, magic), kb = add2(tb, magic);
        d[i / H] = max_abs(d[i / H], fma2(add2(ka, back), minus, ta));
        d[2 + i / H] = max_abs(d[2 + i / H], fma2(add2(kb, back), minus, tb));
        ca[2 * i] = static_cast<uint32_t>(ka.v), ca[2 * i + 1] = static_cast<uint32_t>(ka.v >> 32);
        cb[2 * i] = static_cast<uint32_t>(kb.v), cb[2 * i + 1] = static_cast<uint32_t>(kb.v >> 32);
    }
    // the reciprocal and the product move a quotient of at most 7.5 by less than 2e-6
    const float dlo = fmaxf(d[0], inter ? d[2] : d[1]), dhi = fmaxf(inter ? d[1] : d[2], d[3]);
    const bool edge = dlo > 0.5f - (err * ilo + 7.5f * own + 2e-6f) || dhi > 0.5f - (err * ihi + 7.5f * own + 2e-6f);
    const uint32_t unsure = __ballot_sync(0xFFFFFFFFu, (near || (formed && edge)) && there);
    if (!formed && edge) {
        // elements as they came often lie on a border exactly: what is left of one after k scales is exact in
        // 32 bits (at most 24 bits above the element's last) and decides; in a tie the even code
        auto settle = [](uint32_t bits, float y, float scale) -> uint32_t {
            const float k = __uint_as_float(bits) - 12582920.0f, left = fmaf(-k, scale, y), far = fabsf(left) - 0.5f * scale;
            const bool move = far > 0.0f || (far == 0.0f && (bits & 1u));
            return move ? (left > 0.0f ? bits + 1u : bits - 1u) : bits;
        };
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float sa = i < H ? slo : (inter ? shi : slo), sb = i < H ? (inter ? slo : shi) : shi;
            ca[2 * i] = settle(ca[2 * i], f2_lo(a[i]), sa);
            ca[2 * i + 1] = settle(ca[2 * i + 1], f2_hi(a[i]), sa);
            cb[2 * i] = settle(cb[2 * i], f2_lo(b[i]), sb);
            cb[2 * i + 1] = settle(cb[2 * i + 1], f2_hi(b[i]), sb);
        }
    }
    const uint32_t mine = (L == 32 ? 0xFFFFFFFFu : (1u << L) - 1u) << ((threadIdx.x & 31) - u);
    if (there && !(unsure & mine)) {
        if (u < groups) scales[u] = held;
        store_codes<E>(inter, codes, at, ca, cb);
    }
    return unsure;
}

constexpr int kVectorWarps = 4;
constexpr int kManyHeads = 2;  // four at a time: 20.4 us for the prompt below that takes 17.9 with two

// CTAs of an SM that the registers are kept low enough for: what the loads of
// so short-lived warps need to overlap (4096 tokens, 32 + 8 heads of 128, bf16,
// packed: 16.5 us at 72 registers, 5.2 TB/s; 17.5 us at the 76 to 108 that the
// compiler takes by itself, 17.6 at 64; E4M3 at 128, four-bit append at 80).
// 72 registers spill 8 to 28 bytes a thread, the 80 of the 4-bit append 152 to 248
// with 16-bit rows, and that is faster all the same where there is work for six
// CTAs: 4096 tokens of 8 K and 8 V heads of 128 take 34.3 us, 36.1 with five, 38.5
// with four and no spills; of 64 tokens 6.1, 6.0 and 5.6.
template <typename E, int SINK>
constexpr int kVectorResident = SINK == kSinkKv4 ? 6 : sizeof(typename Elem<E>::Bits) == 1 ? 4 : 7;

// What a warp of the vector kernels works on: heads [first, end) of token t of
// one tensor, this lane's head of the first lot h.
struct WarpHeads {
    int64_t t;
    int which, first, end, h;
};
__device__ __forceinline__ bool warp_heads(const RopeParams &p, int lanes, WarpHeads &w) {
    const uint32_t item = blockIdx.x * kVectorWarps + (threadIdx.x >> 5);
    const uint32_t t32 = item / static_cast<uint32_t>(p.chunks);
    w.t = t32;
    if (w.t >= p.T) return false;
    int chunk = static_cast<int>(item - t32 * p.chunks);
    w.which = 0;  // Q's chunks, then K's, then V's
    if (chunk >= p.chunks_of[0]) {
        chunk -= p.chunks_of[0];
        w.which = 1;
        if (chunk >= p.chunks_of[1]) {
            chunk -= p.chunks_of[1];
            w.which = 2;
        }
    }
    const int heads = w.which == 0 ? p.chunk_heads : p.chunk_kv_heads;
    w.first = chunk * heads;
    w.end = min(p.heads[w.which], w.first + heads);
    w.h = w.first + (threadIdx.x & 31) / lanes;
    return true;
}

// K's or V's heads into the 4-bit cache, the next heads' loads ahead of the work
// on those at hand.
template <typename E, int L>
__device__ __forceinline__ void heads_to_kv4(const RopeParams &p, const WarpHeads &w) {
    constexpr int V = Elem<E>::kPerVec, kEsz = sizeof(typename Elem<E>::Bits), per = 32 / L;
    const int u = threadIdx.x & (L - 1);
    const LanePlace<E> at = lane_place<E>(p, u);
    const int head_bytes = p.head_dim * kEsz;
    const char *in = p.in[w.which] + w.t * p.stride[w.which] + w.h * head_bytes;
    const int64_t slot = p.slots[w.t];
    if (slot < 0 || slot >= p.num_slots) return;
    uint4 va = make_uint4(0, 0, 0, 0), vb = va, na = va, nb = va;
    if (w.h < w.end) {
        va = ld_stream(in + at.lo * kEsz);
        vb = ld_stream(in + at.hi * kEsz);
    }
    const int64_t page = slot / p.page_size, off = slot - page * p.page_size;
    const int kv = w.which - 1;
    int turn = kTurnRow;
    PairFactors<V / 2> f;
    if (kv == 0) {
        const int64_t pos = p.positions[w.t];
        turn = turn_of(pos, p.table_rows);
        if (turn == kTurnRow) f = pair_factors<E>(p, at, p.gamma[1], p.table + pos * 2 * p.half);
    }
#pragma unroll 1
    for (int from = 0; w.first + from < w.end; from += per, va = na, vb = nb) {
        if (w.h + from + per < w.end) {
            na = ld_stream(in + (from + per) * head_bytes + at.lo * kEsz);
            nb = ld_stream(in + (from + per) * head_bytes + at.hi * kEsz);
        }
        const bool there = w.h + from < w.end;
        uint32_t unsure = 0xFFFFFFFFu;
        if (turn == kTurnRow) {
            if (p.interleaved) part_pairs<E>(va, vb);
            F2 a[V / 2], b[V / 2];
            float r = 1.0f;
            if (kv == 0) {
                r = lane_forward<E, L>(p, at, p.gamma[1] != nullptr, f, va, vb, a, b);
            } else {
                Elem<E>::widen(va, a);
                Elem<E>::widen(vb, b);
            }
            const int64_t cell = (page * p.heads[1] + w.h + from) * p.page_size + off;
            unsure = lane_quantise<E, L>(p, kv == 0, r, u, there, at, a, b,
                                         reinterpret_cast<uint8_t *>(p.cache[kv]) + cell * (p.head_dim / 2),
                                         p.scales[kv] + cell * (p.head_dim / kKv4Group));
        }
        if (unsure) {
            __shared__ double exact[kVectorWarps][L * 2 * V];
            for (int k = 0; k < per; ++k) {
                const int head = w.first + from + k;
                if (head >= w.end || !(unsure >> (k * L) & (L == 32 ? 0xFFFFFFFFu : (1u << L) - 1u))) continue;
                const int64_t cell = (page * p.heads[1] + head) * p.page_size + off;
                quantise_head<E>(p, w.which, w.t, p.in[w.which] + w.t * p.stride[w.which] + head * head_bytes,
                                 exact[threadIdx.x >> 5], reinterpret_cast<uint8_t *>(p.cache[kv]) + cell * (p.head_dim / 2),
                                 p.scales[kv] + cell * (p.head_dim / kKv4Group));
            }
        }
    }
}

template <typename E, int SINK, int L>
__global__ void __launch_bounds__(kVectorWarps * 32, kVectorResident<E, SINK>) heads_vector_kernel(const __grid_constant__ RopeParams p) {
    constexpr int V = Elem<E>::kPerVec;
    constexpr int kEsz = sizeof(typename Elem<E>::Bits);
    constexpr int U = kManyHeads;
    pdl_wait_and_release();
    const int lanes = L > 0 ? L : p.lanes;
    const int u = threadIdx.x & (lanes - 1), per = 32 / lanes;
    WarpHeads w;
    if (!warp_heads(p, lanes, w)) return;
    if constexpr (SINK == kSinkKv4) {
        if (w.which > 0) {
            heads_to_kv4<E, L>(p, w);
            return;
        }
    }
    const int which = w.which;
    const bool active = L > 0 || u < p.units;
    const LanePlace<E> at = lane_place<E>(p, active ? u : 0);
    const int head_bytes = p.head_dim * kEsz;
    const char *in = p.in[which] + w.t * p.stride[which] + w.h * head_bytes;
    uint4 va[U], vb[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
        va[j] = vb[j] = make_uint4(0, 0, 0, 0);
        if (active && w.h + j * per < w.end) {
            va[j] = ld_stream(in + j * per * head_bytes + at.lo * kEsz);
            vb[j] = ld_stream(in + j * per * head_bytes + at.hi * kEsz);
        }
    }
    const int64_t pos = p.positions[w.t];
    char *out;
    int64_t step = head_bytes;
    if (SINK == kSinkCache && which > 0) {
        const int64_t slot = p.slots[w.t];
        if (slot < 0 || slot >= p.num_slots) return;
        const int64_t page = slot / p.page_size, off = slot - page * p.page_size;
        step = p.head_stride[which - 1];
        out = p.cache[which - 1] + page * p.page_stride[which - 1] + off * p.token_stride[which - 1] + w.h * step;
        if (which == 2) {  // values as they are
#pragma unroll
            for (int j = 0; j < U; ++j) {
                if (active && w.h + j * per < w.end) {
                    *reinterpret_cast<uint4 *>(out + j * per * step + at.lo * kEsz) = va[j];
                    *reinterpret_cast<uint4 *>(out + j * per * step + at.hi * kEsz) = vb[j];
                }
            }
            return;
        }
    } else {
        out = p.out[which] + w.t * p.stride[which] + w.h * step;
    }
    const int turn = turn_of(pos, p.table_rows);
    if (turn != kTurnRow) {  // zeros or NaN for all of the token's heads
        F2 x[V / 2];
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float v = turn == kTurnPad ? 0.0f : __uint_as_float(0x7FFFFFFFu);
            x[i] = f2(v, v);
        }
        const uint4 fill = Elem<E>::narrow(x);
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (active && w.h + j * per < w.end) {
                st_stream(out + j * per * step + at.lo * kEsz, fill);
                st_stream(out + j * per * step + at.hi * kEsz, fill);
            }
        }
        return;
    }
    const char *gamma = p.gamma[which];
    const PairFactors<V / 2> f = pair_factors<E>(p, at, gamma, p.table + pos * 2 * p.half);
#pragma unroll
    for (int j = 0; j < U; ++j) {
        if (w.first + j * per >= w.end) break;
        if (p.interleaved) part_pairs<E>(va[j], vb[j]);
        F2 a[V / 2], b[V / 2];
        lane_forward<E, L>(p, at, gamma != nullptr, f, va[j], vb[j], a, b);
        uint4 wa = Elem<E>::narrow(a), wb = Elem<E>::narrow(b);
        if (p.interleaved) join_pairs<E>(wa, wb);
        if (active && w.h + j * per < w.end) {
            st_stream(out + j * per * step + at.lo * kEsz, wa);
            st_stream(out + j * per * step + at.hi * kEsz, wb);
        }
    }
}

// Gradient of aligned heads: the same placing; CTAs stay and take tokens in
// turn, all heads of one tensor by a warp, so that a lane keeps its elements'
// dgamma sums in registers, first over Q's heads, then over K's; they are added
// over the warp's lane groups, then over the warps in order.  128 registers and
// so 16 warps an SM: 16384 tokens of 40 + 8 heads of 128, bf16, take 122 us with
// the sum's launch (5.0 TB/s; 84 to 100 bytes of spills a thread for 16-bit types),
// 136 us at 168 registers; the element-wise kernel 725 us.
constexpr int kGradWarps = 8;

template <typename E, int L>
__global__ void __launch_bounds__(kGradWarps * 32, 2) heads_grad_vector_kernel(const __grid_constant__ RopeGradParams p) {
    constexpr int V = Elem<E>::kPerVec, N = V / 2;
    constexpr int kEsz = sizeof(typename Elem<E>::Bits);
    pdl_wait_and_release();
    extern __shared__ float sums[];  // [warps][head_dim]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int lanes = L > 0 ? L : p.lanes;
    const int u = lane & (lanes - 1), per = 32 / lanes, first = lane / lanes;
    const bool active = L > 0 || u < p.units;
    const LanePlace<E> at = lane_place<E>(p, active ? u : 0);
    const int head_bytes = p.head_dim * kEsz;
    for (int w = 0; w < 2; ++w) {
        F2 ga[N], gb[N], da[N], db[N];
        {
            float x[V], y[V];
            lane_gamma<E>(p.gamma[w], at, p.interleaved, x, y);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                ga[i] = f2(x[2 * i], x[2 * i + 1]);
                gb[i] = f2(y[2 * i], y[2 * i + 1]);
                da[i] = db[i] = f2(0.0f, 0.0f);
            }
        }
        const int heads = p.heads[w], chunks = (heads + p.chunk_heads - 1) / p.chunk_heads;
        const int64_t items = p.T * chunks;
        for (int64_t item = static_cast<int64_t>(blockIdx.x) * kGradWarps + warp; item < items;
             item += static_cast<int64_t>(gridDim.x) * kGradWarps) {
            const uint32_t t32 = static_cast<uint32_t>(item) / static_cast<uint32_t>(chunks);
            const int64_t t = t32;
            const int begin = static_cast<int>(static_cast<uint32_t>(item) - t32 * chunks) * p.chunk_heads;
            const int end = min(heads, begin + p.chunk_heads);
            const char *x0 = p.x[w] + t * p.x_stride[w], *y0 = p.dy[w] + t * p.dy_stride[w];
            char *dx = p.dx[w] + t * p.dx_stride[w];
            uint4 xa = make_uint4(0, 0, 0, 0), xb = xa, ya = xa, yb = xa, nxa = xa, nxb = xa, nya = xa, nyb = xa;
            int h = begin + first;
            if (active && h < end) {
                xa = ld_stream(x0 + h * head_bytes + at.lo * kEsz);
                xb = ld_stream(x0 + h * head_bytes + at.hi * kEsz);
                ya = ld_stream(y0 + h * head_bytes + at.lo * kEsz);
                yb = ld_stream(y0 + h * head_bytes + at.hi * kEsz);
            }
            const int64_t pos = p.positions[t];
            const int turn = turn_of(pos, p.table_rows);
            if (turn != kTurnRow) {  // zero gradients, or NaN and NaN in dgamma
                F2 bad[N];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const float v = turn == kTurnPad ? 0.0f : __uint_as_float(0x7FFFFFFFu);
                    bad[i] = f2(v, v);
                }
                const uint4 v = Elem<E>::narrow(bad);
                for (; active && h < end; h += per) {
                    st_stream(dx + h * head_bytes + at.lo * kEsz, v);
                    st_stream(dx + h * head_bytes + at.hi * kEsz, v);
                    if (turn == kTurnPast)
#pragma unroll
                        for (int i = 0; i < N; ++i) da[i] = db[i] = bad[i];
                }
                continue;
            }
            F2 c[N], s[N], ns[N];
            {
                float cf[V], sf[V];
                lane_turns<E>(p, at, p.table + pos * 2 * p.half, cf, sf);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    c[i] = f2(cf[2 * i], cf[2 * i + 1]);
                    s[i] = f2(sf[2 * i], sf[2 * i + 1]);
                    ns[i] = f2(-sf[2 * i], -sf[2 * i + 1]);
                }
            }
#pragma unroll 1
            for (int h0 = begin; h0 < end; h0 += per, h += per, xa = nxa, xb = nxb, ya = nya, yb = nyb) {
                const bool there = active && h < end;
                if (active && h + per < end) {
                    nxa = ld_stream(x0 + (h + per) * head_bytes + at.lo * kEsz);
                    nxb = ld_stream(x0 + (h + per) * head_bytes + at.hi * kEsz);
                    nya = ld_stream(y0 + (h + per) * head_bytes + at.lo * kEsz);
                    nyb = ld_stream(y0 + (h + per) * head_bytes + at.hi * kEsz);
                }
                if (p.interleaved) {
                    part_pairs<E>(xa, xb);
                    part_pairs<E>(ya, yb);
                }
                F2 a[N], b[N], ua[N], ub[N];
                Elem<E>::widen(xa, a);
                Elem<E>::widen(xb, b);
                Elem<E>::widen(ya, ua);
                Elem<E>::widen(yb, ub);
                F2 S2 = f2(0.0f, 0.0f), M2 = S2;
                F2 ea[N], eb[N];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    if (turned(at, i, N)) {
                        const F2 y = ua[i];
                        ua[i] = fma2(ub[i], s[i], mul2(y, c[i]));
                        ub[i] = fma2(y, ns[i], mul2(ub[i], c[i]));
                    }
                    ea[i] = mul2(ua[i], a[i]);
                    eb[i] = mul2(ub[i], b[i]);
                    S2 = fma2(b[i], b[i], fma2(a[i], a[i], S2));
                    M2 = fma2(eb[i], gb[i], fma2(ea[i], ga[i], M2));
                }
                const float S = lanes_sum<L>(f2_lo(S2) + f2_hi(S2), lanes), M = lanes_sum<L>(f2_lo(M2) + f2_hi(M2), lanes);
                const float r = rms_factor(S, p.inv_d, p.eps), k = -(r * r) * M * p.inv_d;
                const F2 rr = f2(r, r), kk = f2(k, k);
                if (there) {
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        da[i] = fma2(ea[i], rr, da[i]);
                        db[i] = fma2(eb[i], rr, db[i]);
                    }
                }
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    a[i] = mul2(fma2(a[i], kk, mul2(ua[i], ga[i])), rr);
                    b[i] = mul2(fma2(b[i], kk, mul2(ub[i], gb[i])), rr);
                }
                uint4 wa = Elem<E>::narrow(a), wb = Elem<E>::narrow(b);
                if (p.interleaved) join_pairs<E>(wa, wb);
                if (there) {
                    st_stream(dx + h * head_bytes + at.lo * kEsz, wa);
                    st_stream(dx + h * head_bytes + at.hi * kEsz, wb);
                }
            }
        }
        float xa[V], xb[V];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            xa[2 * i] = f2_lo(da[i]), xa[2 * i + 1] = f2_hi(da[i]);
            xb[2 * i] = f2_lo(db[i]), xb[2 * i + 1] = f2_hi(db[i]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            for (int off = lanes; off < 32; off <<= 1) {
                xa[i] += __shfl_xor_sync(0xFFFFFFFFu, xa[i], off);
                xb[i] += __shfl_xor_sync(0xFFFFFFFFu, xb[i], off);
            }
        if (first == 0 && active)
#pragma unroll
            for (int i = 0; i < V; ++i) {  // element i of the pairs' firsts and seconds, back in its place
                const int la = p.interleaved ? (i < V / 2 ? at.lo + 2 * i : at.hi + 2 * i - V) : at.lo + i;
                const int lb = p.interleaved ? la + 1 : at.hi + i;
                sums[warp * p.head_dim + la] = xa[i];
                sums[warp * p.head_dim + lb] = xb[i];
            }
        __syncthreads();
        for (int i = threadIdx.x; i < p.head_dim; i += kGradWarps * 32) {
            float v = 0.0f;
#pragma unroll
            for (int k = 0; k < kGradWarps; ++k) v += sums[k * p.head_dim + i];
            p.partial[(static_cast<int64_t>(blockIdx.x) * 2 + w) * p.head_dim + i] = v;
        }
        __syncthreads();
    }
}

// dgamma = the CTAs' partial sums added in CTA order: 8 lanes of rows per
// column, combined in a fixed order.  `ctas` = 0 (no tokens) writes zeros.
struct GradSumParams {
    const float *partial;
    float *dgamma[2];
    int32_t ctas, head_dim;
};
constexpr int kSumRows = 32;
__global__ void __launch_bounds__(32 * kSumRows) dgamma_sum_kernel(const __grid_constant__ GradSumParams p) {
    pdl_wait_and_release();
    __shared__ float part[kSumRows][33];
    const int c = blockIdx.x * 32 + threadIdx.x, n = 2 * p.head_dim;
    float s = 0.0f;
    if (c < n)
        for (int r = threadIdx.y; r < p.ctas; r += kSumRows) s += p.partial[static_cast<int64_t>(r) * n + c];
    part[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < n) {
        float v = 0.0f;
        for (int r = 0; r < kSumRows; ++r) v += part[r][threadIdx.x];
        p.dgamma[c / p.head_dim][c % p.head_dim] = v;
    }
}

// ----------------------------------------------------------------------------
// Cached tokens of the 4-bit cache back as rows: one thread per 8 elements, a
// row of threads along a token's K, then V elements.  Bound by the rows written:
// 4096 tokens of 8 heads of 128 to bf16 take 8.6 us (2.5 TB/s), 64 tokens 1.8 us.
struct Kv4ReadParams {
    const uint8_t *codes[2];
    const __half *scales[2];
    char *out[2];
    int64_t stride[2];  // bytes
    const int64_t *slots;
    int64_t n, num_slots;
    int32_t page_size, heads, head_dim, words;  // words: 8-element words of a token's heads
    int32_t vector;                             // rows are 16-byte aligned
};
template <typename E>
__global__ void __launch_bounds__(256) kv4_read_kernel(const __grid_constant__ Kv4ReadParams p) {
    pdl_wait_and_release();
    const uint32_t i = blockIdx.x * 256u + threadIdx.x, per_token = 2u * p.words;  // fewer than 2^32 threads
    const uint32_t t = i / per_token;
    if (t >= p.n) return;
    uint32_t w = i - t * per_token;
    const int kv = w >= static_cast<uint32_t>(p.words);
    w -= kv * p.words;
    const uint32_t per_head = p.head_dim / 8, h = w / per_head, j = w - h * per_head;
    const int64_t slot = p.slots[t];
    uint32_t codes = 0x88888888u;
    float s = 0.0f;
    if (slot >= 0 && slot < p.num_slots) {
        const int64_t page = slot / p.page_size, off = slot - page * p.page_size;
        const int64_t cell = (page * p.heads + h) * p.page_size + off;
        codes = reinterpret_cast<const uint32_t *>(p.codes[kv])[cell * per_head + j];
        s = __half2float(p.scales[kv][cell * (p.head_dim / kKv4Group) + j * 8 / kKv4Group]);
    }
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = static_cast<float>(static_cast<int>((codes >> (4 * e)) & 15u) - 8) * s;
    char *out = p.out[kv] + t * p.stride[kv] + static_cast<int64_t>(w) * 8 * sizeof(typename Elem<E>::Bits);
    if (p.vector) {
        constexpr int V = Elem<E>::kPerVec;
#pragma unroll
        for (int k = 0; k < 8 / V; ++k) {
            F2 x[V / 2];
#pragma unroll
            for (int e = 0; e < V / 2; ++e) x[e] = f2(v[k * V + 2 * e], v[k * V + 2 * e + 1]);
            st_stream(out + 16 * k, Elem<E>::narrow(x));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) put_elem<E>(out, e, v[e]);
    }
}

// ----------------------------------------------------------------------------
// Host side.
using namespace checks;

template <int SINK>
const void *scalar_kernel(int dt) {
    switch (dt) {
        case QKN_F32: return (const void *)heads_scalar_kernel<float, SINK>;
        case QKN_BF16: return (const void *)heads_scalar_kernel<__nv_bfloat16, SINK>;
        case QKN_F16: return (const void *)heads_scalar_kernel<__half, SINK>;
        default:
            if constexpr (SINK == kSinkKv4) return nullptr;
            else return (const void *)heads_scalar_kernel<__nv_fp8_e4m3, SINK>;
    }
}

// The kernels for heads of 64, 128 and 256 elements know their lanes; others
// count them as they run (L = 0).
template <typename E, int SINK>
const void *vector_kernel(int lanes, bool exact) {
    constexpr int k64 = 64 / (2 * Elem<E>::kPerVec);
    if (exact && lanes == k64) return (const void *)heads_vector_kernel<E, SINK, k64>;
    if (exact && lanes == 2 * k64) return (const void *)heads_vector_kernel<E, SINK, 2 * k64>;
    if (exact && lanes == 4 * k64) return (const void *)heads_vector_kernel<E, SINK, 4 * k64>;
    if constexpr (SINK == kSinkKv4) return nullptr;
    else return (const void *)heads_vector_kernel<E, SINK, 0>;
}
template <int SINK>
const void *vector_kernel(int dt, int lanes, bool exact) {
    switch (dt) {
        case QKN_F32: return vector_kernel<float, SINK>(lanes, exact);
        case QKN_BF16: return vector_kernel<__nv_bfloat16, SINK>(lanes, exact);
        case QKN_F16: return vector_kernel<__half, SINK>(lanes, exact);
        default:
            if constexpr (SINK == kSinkKv4) return nullptr;
            else return vector_kernel<__nv_fp8_e4m3, SINK>(lanes, exact);
    }
}
template <typename E>
const void *grad_kernel(int lanes, bool exact) {
    constexpr int k64 = 64 / (2 * Elem<E>::kPerVec);
    if (exact && lanes == k64) return (const void *)heads_grad_vector_kernel<E, k64>;
    if (exact && lanes == 2 * k64) return (const void *)heads_grad_vector_kernel<E, 2 * k64>;
    if (exact && lanes == 4 * k64) return (const void *)heads_grad_vector_kernel<E, 4 * k64>;
    return (const void *)heads_grad_vector_kernel<E, 0>;
}

// Lanes of a head for the vector kernels; 0 where the sizes do not fit them.
int vector_lanes(int dtype, int head_dim, int half) {
    const int two = 2 * (16 / elem_bytes(dtype));  // elements of two vectors
    if (head_dim % two != 0 || 2 * half % two != 0 || head_dim / two > 32) return 0;
    int lanes = 1;
    while (lanes < head_dim / two) lanes *= 2;
    return lanes;
}

// How many times a warp takes 32 / lanes heads of a token: what is formed once
// for a token counts less the more often, and the warps become fewer (32 + 8
// heads of 128, bf16, once / twice / four times: 64 tokens rotated 2.03 / 2.09 us,
// 256 3.0 / 2.6, 8192 39.7 / 30.3; gradient of 256 7.9 / 8.5 / 9.6 us, of 1024
// 14.6 / 14.4 / 12.7, of 8192 68 / 59 / 55; four-bit append and read of 1024
// 17.8 / 17.1 / 17.1 us).
int head_groups(int64_t rows, int per, int sms, int most) {
    int n = 1;
    while (n < most && rows >= (int64_t)sms * 24 * per * n) n *= 2;
    return n;
}

template <int SINK>
qkn_status launch_heads(RopeParams &p, int dtype, bool aligned, void *stream) {
    int sms = 0;
    qkn_status st = device_sms(&sms);
    if (st != QKN_OK) return st;
    const int64_t rows = p.T * p.heads_total;
    p.lanes = aligned ? vector_lanes(dtype, p.head_dim, p.half) : 0;
    if (p.lanes > 0) {
        p.units = p.head_dim / (2 * (16 / elem_bytes(dtype)));
        const int per = 32 / p.lanes;
        p.chunk_heads = per * head_groups(rows, per, sms, kManyHeads);
        p.chunk_kv_heads = SINK == kSinkKv4 ? per * head_groups(rows, per, sms, 4) : p.chunk_heads;
        p.chunks = 0;
        for (int i = 0; i < 3; ++i) {
            const int heads = i ? p.chunk_kv_heads : p.chunk_heads;
            p.chunks += p.chunks_of[i] = (p.heads[i] + heads - 1) / heads;
        }
        const int64_t ctas = (p.T * p.chunks + kVectorWarps - 1) / kVectorWarps;
        return launched(launch_pdl(vector_kernel<SINK>(dtype, p.lanes, p.lanes == p.units), dim3((unsigned)ctas),
                                   kVectorWarps * 32, 0, stream, p));
    }
    int64_t grid = (rows + kScalarWarps - 1) / kScalarWarps;
    if (grid > 32 * static_cast<int64_t>(sms)) grid = 32 * static_cast<int64_t>(sms);
    return launched(launch_pdl(scalar_kernel<SINK>(dtype), dim3((unsigned)grid), kScalarWarps * 32, 0, stream, p));
}

// What the three forms share: sizes, the table and the rows that they read.
struct Common {
    int64_t T;
    int32_t head_dim, rotary_dim;
    int64_t table_rows;
    const float *table;
    const int64_t *positions;
    float eps;
    int dtype;
};

qkn_status check_common(const Common &c, int64_t heads) {
    if (c.dtype < QKN_F32 || c.dtype > QKN_FP8_E4M3) return fail(QKN_ERR_INVALID_ARG, "unknown dtype %d", c.dtype);
    if (c.T < 0) return fail(QKN_ERR_INVALID_ARG, "T = %lld < 0", (long long)c.T);
    if (c.head_dim < 1) return fail(QKN_ERR_INVALID_ARG, "head_dim = %d", c.head_dim);
    if (c.head_dim > kRopeMaxHeadDim)
        return fail(QKN_ERR_UNSUPPORTED, "head_dim = %d above %d", c.head_dim, kRopeMaxHeadDim);
    if (c.rotary_dim < 0 || c.rotary_dim > c.head_dim || c.rotary_dim % 2 != 0)
        return fail(QKN_ERR_INVALID_ARG, "rotary_dim = %d must be even and in [0, head_dim = %d]", c.rotary_dim, c.head_dim);
    if (c.table_rows < 0 || c.table_rows >= ((int64_t)1 << 40))
        return fail(QKN_ERR_INVALID_ARG, "table_rows = %lld", (long long)c.table_rows);
    if (!(std::isfinite(c.eps) && c.eps >= 0.0f)) return fail(QKN_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (heads < 1 || heads > (1 << 16)) return fail(QKN_ERR_INVALID_ARG, "%lld heads", (long long)heads);
    if (c.T > 0 && c.T >= ((int64_t)1 << 31) / heads) return fail(QKN_ERR_INVALID_ARG, "T * heads must stay below 2^31");
    if (c.T > 0 && (!c.positions || (!c.table && c.table_rows > 0 && c.rotary_dim > 0)))
        return fail(QKN_ERR_INVALID_ARG, "null positions or cos_sin");
    if ((reinterpret_cast<uintptr_t>(c.positions) & 7u) || (reinterpret_cast<uintptr_t>(c.table) & 3u))
        return fail(QKN_ERR_INVALID_ARG, "positions and cos_sin must be aligned to their elements");
    return QKN_OK;
}

bool elem_aligned(const void *p, int esz) { return reinterpret_cast<uintptr_t>(p) % (unsigned)esz == 0; }

qkn_status check_rows(const char *name, const void *base, int64_t stride, int64_t width, int64_t T, int esz) {
    if (stride < width)
        return fail(QKN_ERR_INVALID_ARG, "%s stride %lld below its width %lld", name, (long long)stride, (long long)width);
    if (!extent_ok(T, stride, width, esz)) return fail(QKN_ERR_INVALID_ARG, "%s: buffer extent overflows", name);
    if (T > 0 && !base) return fail(QKN_ERR_INVALID_ARG, "%s: null pointer", name);
    if (!elem_aligned(base, esz)) return fail(QKN_ERR_INVALID_ARG, "%s: not aligned to its elements", name);
    return QKN_OK;
}

Span rows_span(const void *base, int64_t width, int64_t stride, int64_t T, int esz, const char *name) {
    return Span{base, width * esz, stride * esz, T, name};
}

void fill_common(RopeParams &p, const Common &c, int interleaved) {
    p.T = c.T;
    p.table = c.table;
    p.positions = c.positions;
    p.table_rows = c.table_rows;
    p.head_dim = c.head_dim;
    p.half = c.rotary_dim / 2;
    p.interleaved = interleaved ? 1 : 0;
    p.eps = c.eps;
    p.inv_d = static_cast<float>(1.0 / c.head_dim);
}

struct AppendArgs {
    const void *q_in;
    void *q_out;
    const void *gamma_q;
    int64_t q_stride;
    int32_t q_heads;
    const void *k_in, *gamma_k;
    int64_t k_stride;
    const void *v_in;
    int64_t v_stride;
    int32_t kv_heads;
    int interleaved;
    const int64_t *slots;
};

// Checks and fills everything of an append but the cache; `r` gets the spans
// that nothing may be written over.
qkn_status prepare_append(const Common &c, const AppendArgs &a, RopeParams &p, Span *r, int *nr) {
    if (a.q_heads < 0 || a.kv_heads < 1)
        return fail(QKN_ERR_INVALID_ARG, "q_heads = %d, kv_heads = %d", a.q_heads, a.kv_heads);
    qkn_status st = check_common(c, (int64_t)a.q_heads + 2 * (int64_t)a.kv_heads);
    if (st != QKN_OK) return st;
    const int esz = elem_bytes(c.dtype), gsz = gamma_bytes(c.dtype);
    const int64_t wq = (int64_t)a.q_heads * c.head_dim, wk = (int64_t)a.kv_heads * c.head_dim;
    if (a.q_heads > 0) {
        if ((st = check_rows("q_in", a.q_in, a.q_stride, wq, c.T, esz)) != QKN_OK) return st;
        if ((st = check_rows("q_out", a.q_out, a.q_stride, wq, c.T, esz)) != QKN_OK) return st;
    }
    if ((st = check_rows("k_in", a.k_in, a.k_stride, wk, c.T, esz)) != QKN_OK) return st;
    if ((st = check_rows("v_in", a.v_in, a.v_stride, wk, c.T, esz)) != QKN_OK) return st;
    if (a.q_heads > 0 && !a.gamma_q != !a.gamma_k)
        return fail(QKN_ERR_INVALID_ARG, "gamma_q and gamma_k: both (norm) or neither (rotation only)");
    if (!elem_aligned(a.gamma_q, gsz) || !elem_aligned(a.gamma_k, gsz))
        return fail(QKN_ERR_INVALID_ARG, "gamma: not aligned to its elements");
    if (c.T > 0 && !a.slots) return fail(QKN_ERR_INVALID_ARG, "null slots");
    if (reinterpret_cast<uintptr_t>(a.slots) & 7u) return fail(QKN_ERR_INVALID_ARG, "slots must be 8-byte aligned");
    p = RopeParams{};
    fill_common(p, c, a.interleaved);
    p.in[0] = static_cast<const char *>(a.q_in);
    p.in[1] = static_cast<const char *>(a.k_in);
    p.in[2] = static_cast<const char *>(a.v_in);
    p.out[0] = static_cast<char *>(a.q_out);
    p.stride[0] = a.q_stride * esz;
    p.stride[1] = a.k_stride * esz;
    p.stride[2] = a.v_stride * esz;
    p.gamma[0] = static_cast<const char *>(a.gamma_q);
    p.gamma[1] = static_cast<const char *>(a.gamma_k);
    p.heads[0] = a.q_heads;
    p.heads[1] = p.heads[2] = a.kv_heads;
    p.heads_total = a.q_heads + 2 * a.kv_heads;
    p.slots = a.slots;
    int n = 0;
    r[n++] = rows_span(a.q_heads > 0 ? a.q_in : nullptr, wq, a.q_stride, c.T, esz, "q_in");
    r[n++] = rows_span(a.k_in, wk, a.k_stride, c.T, esz, "k_in");
    r[n++] = rows_span(a.v_in, wk, a.v_stride, c.T, esz, "v_in");
    r[n++] = flat(a.q_heads > 0 ? a.gamma_q : nullptr, (int64_t)c.head_dim * gsz, "gamma_q");
    r[n++] = flat(a.gamma_k, (int64_t)c.head_dim * gsz, "gamma_k");
    r[n++] = flat(c.table, c.table_rows * c.rotary_dim * 4, "cos_sin");
    r[n++] = flat(c.positions, c.T * 8, "positions");
    r[n++] = flat(a.slots, c.T * 8, "slots");
    *nr = n;
    return QKN_OK;
}

bool rows_aligned(const RopeParams &p) {
    bool v = true;
    for (int i = 0; i < 3; ++i)
        if (p.heads[i]) v = v && aligned16(p.in[i]) && p.stride[i] % 16 == 0;
    for (int i = 0; i < 2; ++i) v = v && aligned16(p.out[i]) && aligned16(p.gamma[i]);
    return v && aligned16(p.table);
}

// A cache tensor's cells must not share memory: each stride has to clear the
// extent of the smaller ones.
bool cells_apart(int64_t head_dim, int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2) {
    int64_t n[3] = {n0, n1, n2}, s[3] = {s0, s1, s2};
    for (int i = 0; i < 3; ++i)
        for (int j = i + 1; j < 3; ++j)
            if (s[j] < s[i] || (s[j] == s[i] && n[j] < n[i])) {
                const int64_t a = s[i], b = n[i];
                s[i] = s[j];
                n[i] = n[j];
                s[j] = a;
                n[j] = b;
            }
    __int128 extent = head_dim;
    for (int i = 0; i < 3; ++i) {
        if (n[i] > 1 && s[i] < extent) return false;
        if (n[i] > 1) extent += (__int128)(n[i] - 1) * s[i];
    }
    return true;
}

constexpr int64_t kMaxCell = (int64_t)1 << 60;

qkn_status check_pages(int64_t num_pages, int32_t page_size) {
    if (num_pages < 0 || page_size < 1 || num_pages >= ((int64_t)1 << 40) / page_size)
        return fail(QKN_ERR_INVALID_ARG, "num_pages = %lld, page_size = %d", (long long)num_pages, page_size);
    return QKN_OK;
}

constexpr int64_t kGradCtas = 592;  // partial sums kept: 4 CTAs on each of 148 SMs

int64_t grad_ctas(int64_t rows) { return rows < kGradCtas ? rows : kGradCtas; }

template <typename E>
const void *read_kernel() {
    return (const void *)kv4_read_kernel<E>;
}

}  // namespace
}  // namespace qkn

using namespace qkn;
using namespace qkn::checks;

extern "C" {

qkn_status qknorm_headwise_rope(const void *q_in, void *q_out, const void *gamma_q, int64_t q_stride, int32_t q_heads,
                                const void *k_in, void *k_out, const void *gamma_k, int64_t k_stride, int32_t k_heads,
                                int64_t T, int32_t head_dim, const float *cos_sin, int64_t table_rows,
                                int32_t rotary_dim, int32_t interleaved, const int64_t *positions, float eps,
                                qkn_dtype dtype, void *stream) {
    if (q_heads < 1 || k_heads < 1) return fail(QKN_ERR_INVALID_ARG, "q_heads = %d, k_heads = %d", q_heads, k_heads);
    const Common c{T, head_dim, rotary_dim, table_rows, cos_sin, positions, eps, (int)dtype};
    qkn_status st = check_common(c, (int64_t)q_heads + k_heads);
    if (st != QKN_OK) return st;
    const int esz = elem_bytes(dtype), gsz = gamma_bytes(dtype);
    const int64_t wq = (int64_t)q_heads * head_dim, wk = (int64_t)k_heads * head_dim;
    if ((st = check_rows("q_in", q_in, q_stride, wq, T, esz)) != QKN_OK) return st;
    if ((st = check_rows("q_out", q_out, q_stride, wq, T, esz)) != QKN_OK) return st;
    if ((st = check_rows("k_in", k_in, k_stride, wk, T, esz)) != QKN_OK) return st;
    if ((st = check_rows("k_out", k_out, k_stride, wk, T, esz)) != QKN_OK) return st;
    if (T > 0 && (!gamma_q || !gamma_k)) return fail(QKN_ERR_INVALID_ARG, "null gamma");
    if (!elem_aligned(gamma_q, gsz) || !elem_aligned(gamma_k, gsz))
        return fail(QKN_ERR_INVALID_ARG, "gamma: not aligned to its elements");
    if (T == 0) return ok();
    const Span w[] = {rows_span(q_out, wq, q_stride, T, esz, "q_out"), rows_span(k_out, wk, k_stride, T, esz, "k_out")};
    const Span r[] = {rows_span(q_in, wq, q_stride, T, esz, "q_in"),
                      rows_span(k_in, wk, k_stride, T, esz, "k_in"),
                      flat(gamma_q, (int64_t)head_dim * gsz, "gamma_q"),
                      flat(gamma_k, (int64_t)head_dim * gsz, "gamma_k"),
                      flat(cos_sin, table_rows * rotary_dim * 4, "cos_sin"),
                      flat(positions, T * 8, "positions")};
    const int in_place[] = {0, 0, 1, 1};
    if ((st = check_written(w, 2, r, 6, in_place, 4)) != QKN_OK) return st;
    RopeParams p{};
    fill_common(p, c, interleaved);
    p.in[0] = static_cast<const char *>(q_in);
    p.in[1] = static_cast<const char *>(k_in);
    p.out[0] = static_cast<char *>(q_out);
    p.out[1] = static_cast<char *>(k_out);
    p.stride[0] = q_stride * esz;
    p.stride[1] = k_stride * esz;
    p.gamma[0] = static_cast<const char *>(gamma_q);
    p.gamma[1] = static_cast<const char *>(gamma_k);
    p.heads[0] = q_heads;
    p.heads[1] = k_heads;
    p.heads_total = q_heads + k_heads;
    return launch_heads<kSinkRows>(p, dtype, rows_aligned(p), stream);
}

qkn_status qknorm_rope_append(const void *q_in, void *q_out, const void *gamma_q, int64_t q_stride, int32_t q_heads,
                              const void *k_in, const void *gamma_k, int64_t k_stride, const void *v_in,
                              int64_t v_stride, int32_t kv_heads, int64_t T, int32_t head_dim, const float *cos_sin,
                              int64_t table_rows, int32_t rotary_dim, int32_t interleaved, const int64_t *positions,
                              void *k_cache, const int64_t *k_cache_strides, void *v_cache,
                              const int64_t *v_cache_strides, int64_t num_pages, int32_t page_size,
                              const int64_t *slots, float eps, qkn_dtype dtype, void *stream) {
    const Common c{T, head_dim, rotary_dim, table_rows, cos_sin, positions, eps, (int)dtype};
    const AppendArgs a{q_in, q_out, gamma_q, q_stride, q_heads, k_in, gamma_k, k_stride, v_in, v_stride, kv_heads,
                       interleaved, slots};
    RopeParams p;
    Span r[8];
    int nr = 0;
    qkn_status st = prepare_append(c, a, p, r, &nr);
    if (st != QKN_OK) return st;
    if ((st = check_pages(num_pages, page_size)) != QKN_OK) return st;
    if (!k_cache_strides || !v_cache_strides) return fail(QKN_ERR_INVALID_ARG, "null cache strides");
    const int esz = elem_bytes(dtype);
    p.num_slots = num_pages * page_size;
    p.page_size = page_size;
    Span w[3];
    int nw = 0;
    if (q_heads > 0) w[nw++] = rows_span(q_out, (int64_t)q_heads * head_dim, q_stride, T, esz, "q_out");
    bool aligned = rows_aligned(p);
    for (int i = 0; i < 2; ++i) {
        const int64_t *s = i ? v_cache_strides : k_cache_strides;
        void *base = i ? v_cache : k_cache;
        const char *name = i ? "v_cache" : "k_cache";
        if (s[0] < 0 || s[1] < 0 || s[2] < 0 || s[0] > kMaxCell || s[1] > kMaxCell || s[2] > kMaxCell)
            return fail(QKN_ERR_INVALID_ARG, "%s: bad strides", name);
        if (!cells_apart(head_dim, num_pages, s[0], page_size, s[1], kv_heads, s[2]))
            return fail(QKN_ERR_INVALID_ARG, "%s: cells overlap one another", name);
        const __int128 in_page = (__int128)(page_size - 1) * s[1] + (__int128)(kv_heads - 1) * s[2] + head_dim;
        const __int128 whole = num_pages ? in_page + (__int128)(num_pages - 1) * s[0] : 0;
        if (whole * esz >= ((__int128)1 << 62)) return fail(QKN_ERR_INVALID_ARG, "%s: buffer extent overflows", name);
        if (T > 0 && num_pages > 0 && !base) return fail(QKN_ERR_INVALID_ARG, "%s: null pointer", name);
        if (!elem_aligned(base, esz)) return fail(QKN_ERR_INVALID_ARG, "%s: not aligned to its elements", name);
        // pages as rows where the other two strides stay inside one, else the whole extent
        w[nw++] = num_pages == 0 ? Span{nullptr, 0, 0, 0, name}
                  : in_page <= s[0] || num_pages == 1
                      ? Span{base, (int64_t)in_page * esz, s[0] * esz, num_pages, name}
                      : flat(base, (int64_t)whole * esz, name);
        p.cache[i] = static_cast<char *>(base);
        p.page_stride[i] = s[0] * esz;
        p.token_stride[i] = s[1] * esz;
        p.head_stride[i] = s[2] * esz;
        aligned = aligned && aligned16(base) && p.page_stride[i] % 16 == 0 && p.token_stride[i] % 16 == 0 &&
                  p.head_stride[i] % 16 == 0;
    }
    if (T == 0) return ok();
    const int in_place[] = {0, 0};
    if ((st = check_written(w, nw, r, nr, in_place, q_heads > 0 ? 2 : 0)) != QKN_OK) return st;
    return launch_heads<kSinkCache>(p, dtype, aligned, stream);
}

qkn_status qknorm_rope_append_kv4(const void *q_in, void *q_out, const void *gamma_q, int64_t q_stride, int32_t q_heads,
                                  const void *k_in, const void *gamma_k, int64_t k_stride, const void *v_in,
                                  int64_t v_stride, int32_t kv_heads, int64_t T, int32_t head_dim,
                                  const float *cos_sin, int64_t table_rows, int32_t rotary_dim, int32_t interleaved,
                                  const int64_t *positions, void *k_codes, void *k_scales, void *v_codes,
                                  void *v_scales, int64_t num_pages, int32_t page_size, const int64_t *slots, float eps,
                                  qkn_dtype dtype, void *stream) {
    const Common c{T, head_dim, rotary_dim, table_rows, cos_sin, positions, eps, (int)dtype};
    const AppendArgs a{q_in, q_out, gamma_q, q_stride, q_heads, k_in, gamma_k, k_stride, v_in, v_stride, kv_heads,
                       interleaved, slots};
    RopeParams p;
    Span r[8];
    int nr = 0;
    qkn_status st = prepare_append(c, a, p, r, &nr);
    if (st != QKN_OK) return st;
    if (dtype == QKN_FP8_E4M3) return fail(QKN_ERR_UNSUPPORTED, "the 4-bit cache takes float32, bfloat16 or float16 rows");
    int64_t codes = 0, scales = 0;
    if ((st = check_kv4(num_pages, page_size, kv_heads, head_dim, k_codes, k_scales, v_codes, v_scales,
                        T > 0 && num_pages > 0, &codes, &scales)) != QKN_OK)
        return st;
    if (T == 0) return ok();
    p.num_slots = num_pages * page_size;
    p.page_size = page_size;
    p.cache[0] = static_cast<char *>(k_codes);
    p.cache[1] = static_cast<char *>(v_codes);
    p.scales[0] = static_cast<__half *>(k_scales);
    p.scales[1] = static_cast<__half *>(v_scales);
    Span w[5];
    int nw = 0;
    const int esz = elem_bytes(dtype);
    if (q_heads > 0) w[nw++] = rows_span(q_out, (int64_t)q_heads * head_dim, q_stride, T, esz, "q_out");
    if (num_pages > 0) {
        w[nw++] = flat(k_codes, codes, "k_codes");
        w[nw++] = flat(k_scales, scales, "k_scales");
        w[nw++] = flat(v_codes, codes, "v_codes");
        w[nw++] = flat(v_scales, scales, "v_scales");
    }
    const int in_place[] = {0, 0};
    if ((st = check_written(w, nw, r, nr, in_place, q_heads > 0 ? 2 : 0)) != QKN_OK) return st;
    return launch_heads<kSinkKv4>(p, dtype, rows_aligned(p), stream);
}

qkn_status qknorm_kv4_read(const void *k_codes, const void *k_scales, const void *v_codes, const void *v_scales,
                           int64_t num_pages, int32_t page_size, int32_t kv_heads, int32_t head_dim,
                           const int64_t *slots, int64_t n, void *k_out, int64_t k_stride, void *v_out,
                           int64_t v_stride, qkn_dtype dtype, void *stream) {
    if (dtype < QKN_F32 || dtype > QKN_FP8_E4M3) return fail(QKN_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (dtype == QKN_FP8_E4M3) return fail(QKN_ERR_UNSUPPORTED, "the 4-bit cache gives float32, bfloat16 or float16 rows");
    if (n < 0) return fail(QKN_ERR_INVALID_ARG, "n = %lld < 0", (long long)n);
    int64_t codes = 0, scales = 0;
    qkn_status st = check_kv4(num_pages, page_size, kv_heads, head_dim, k_codes, k_scales, v_codes, v_scales,
                              n > 0 && num_pages > 0, &codes, &scales);
    if (st != QKN_OK) return st;
    const int esz = elem_bytes(dtype);
    const int64_t w = (int64_t)kv_heads * head_dim;
    if ((st = check_rows("k_out", k_out, k_stride, w, n, esz)) != QKN_OK) return st;
    if ((st = check_rows("v_out", v_out, v_stride, w, n, esz)) != QKN_OK) return st;
    if (n > 0 && !slots) return fail(QKN_ERR_INVALID_ARG, "null slots");
    if (reinterpret_cast<uintptr_t>(slots) & 7u) return fail(QKN_ERR_INVALID_ARG, "slots must be 8-byte aligned");
    if (n == 0) return ok();
    Kv4ReadParams p{};
    p.words = (int32_t)(w / 8);
    const __int128 threads = (__int128)n * 2 * p.words;
    if (threads >= ((__int128)1 << 32) - 256) return fail(QKN_ERR_INVALID_ARG, "n * kv_heads * head_dim too large");
    const Span ws[] = {rows_span(k_out, w, k_stride, n, esz, "k_out"), rows_span(v_out, w, v_stride, n, esz, "v_out")};
    const Span rs[] = {num_pages ? flat(k_codes, codes, "k_codes") : flat(nullptr, 0, ""),
                       num_pages ? flat(k_scales, scales, "k_scales") : flat(nullptr, 0, ""),
                       num_pages ? flat(v_codes, codes, "v_codes") : flat(nullptr, 0, ""),
                       num_pages ? flat(v_scales, scales, "v_scales") : flat(nullptr, 0, ""), flat(slots, n * 8, "slots")};
    if ((st = check_written(ws, 2, rs, 5, nullptr, 0)) != QKN_OK) return st;
    p.codes[0] = static_cast<const uint8_t *>(k_codes);
    p.codes[1] = static_cast<const uint8_t *>(v_codes);
    p.scales[0] = static_cast<const __half *>(k_scales);
    p.scales[1] = static_cast<const __half *>(v_scales);
    p.out[0] = static_cast<char *>(k_out);
    p.out[1] = static_cast<char *>(v_out);
    p.stride[0] = k_stride * esz;
    p.stride[1] = v_stride * esz;
    p.slots = slots;
    p.n = n;
    p.vector = aligned16(k_out) && aligned16(v_out) && p.stride[0] % 16 == 0 && p.stride[1] % 16 == 0;
    p.num_slots = num_pages * page_size;
    p.page_size = page_size;
    p.heads = kv_heads;
    p.head_dim = head_dim;
    const void *fn = dtype == QKN_F32    ? read_kernel<float>()
                     : dtype == QKN_BF16 ? read_kernel<__nv_bfloat16>()
                                         : read_kernel<__half>();
    return launched(launch_pdl(fn, dim3((unsigned)((threads + 255) / 256)), 256, 0, stream, p));
}

int64_t qknorm_headwise_rope_backward_workspace_bytes(int64_t T, int32_t q_heads, int32_t k_heads, int32_t head_dim) {
    if (T < 0 || q_heads < 1 || k_heads < 1 || head_dim < 1 || head_dim > kRopeMaxHeadDim) return -1;
    const int64_t heads = (int64_t)q_heads + k_heads;
    if (heads > (1 << 16) || (T > 0 && T >= ((int64_t)1 << 31) / heads)) return -1;
    return grad_ctas(T * heads) * 2 * head_dim * 4;
}

qkn_status qknorm_headwise_rope_backward(const void *q_in, int64_t q_stride, const void *dq_out, int64_t dq_out_stride,
                                         void *dq_in, int64_t dq_in_stride, const void *gamma_q, float *dgamma_q,
                                         int32_t q_heads, const void *k_in, int64_t k_stride, const void *dk_out,
                                         int64_t dk_out_stride, void *dk_in, int64_t dk_in_stride, const void *gamma_k,
                                         float *dgamma_k, int32_t k_heads, int64_t T, int32_t head_dim,
                                         const float *cos_sin, int64_t table_rows, int32_t rotary_dim,
                                         int32_t interleaved, const int64_t *positions, float eps, void *workspace,
                                         int64_t workspace_bytes, qkn_dtype dtype, void *stream) {
    if (q_heads < 1 || k_heads < 1) return fail(QKN_ERR_INVALID_ARG, "q_heads = %d, k_heads = %d", q_heads, k_heads);
    const Common c{T, head_dim, rotary_dim, table_rows, cos_sin, positions, eps, (int)dtype};
    qkn_status st = check_common(c, (int64_t)q_heads + k_heads);
    if (st != QKN_OK) return st;
    if (dtype == QKN_FP8_E4M3) return fail(QKN_ERR_UNSUPPORTED, "gradients take float32, bfloat16 or float16");
    const int esz = elem_bytes(dtype), gsz = gamma_bytes(dtype);
    const int64_t width[2] = {(int64_t)q_heads * head_dim, (int64_t)k_heads * head_dim};
    const void *x[2] = {q_in, k_in}, *dy[2] = {dq_out, dk_out}, *gamma[2] = {gamma_q, gamma_k};
    void *dx[2] = {dq_in, dk_in};
    const int64_t xs[2] = {q_stride, k_stride}, dys[2] = {dq_out_stride, dk_out_stride}, dxs[2] = {dq_in_stride, dk_in_stride};
    const char *names[2][3] = {{"q_in", "dq_out", "dq_in"}, {"k_in", "dk_out", "dk_in"}};
    RopeGradParams p{};
    Span w[5], r[9];
    int nw = 0, nr = 0;
    bool aligned = aligned16(cos_sin);
    for (int i = 0; i < 2; ++i) {
        if ((st = check_rows(names[i][0], x[i], xs[i], width[i], T, esz)) != QKN_OK) return st;
        if ((st = check_rows(names[i][1], dy[i], dys[i], width[i], T, esz)) != QKN_OK) return st;
        if ((st = check_rows(names[i][2], dx[i], dxs[i], width[i], T, esz)) != QKN_OK) return st;
        if (T > 0 && !gamma[i]) return fail(QKN_ERR_INVALID_ARG, "null gamma");
        if (!elem_aligned(gamma[i], gsz)) return fail(QKN_ERR_INVALID_ARG, "gamma: not aligned to its elements");
        w[nw++] = rows_span(dx[i], width[i], dxs[i], T, esz, names[i][2]);
        r[nr++] = rows_span(x[i], width[i], xs[i], T, esz, names[i][0]);
        r[nr++] = rows_span(dy[i], width[i], dys[i], T, esz, names[i][1]);
        r[nr++] = flat(gamma[i], (int64_t)head_dim * gsz, "gamma");
        p.x[i] = static_cast<const char *>(x[i]);
        p.dy[i] = static_cast<const char *>(dy[i]);
        p.dx[i] = static_cast<char *>(dx[i]);
        p.x_stride[i] = xs[i] * esz;
        p.dy_stride[i] = dys[i] * esz;
        p.dx_stride[i] = dxs[i] * esz;
        p.gamma[i] = static_cast<const char *>(gamma[i]);
        aligned = aligned && aligned16(x[i]) && aligned16(dy[i]) && aligned16(dx[i]) && aligned16(gamma[i]) &&
                  p.x_stride[i] % 16 == 0 && p.dy_stride[i] % 16 == 0 && p.dx_stride[i] % 16 == 0;
    }
    if (!dgamma_q || !dgamma_k) return fail(QKN_ERR_INVALID_ARG, "null dgamma");
    if (!elem_aligned(dgamma_q, 4) || !elem_aligned(dgamma_k, 4) || !elem_aligned(workspace, 4))
        return fail(QKN_ERR_INVALID_ARG, "dgamma and the workspace must be 4-byte aligned");
    const int64_t need = qknorm_headwise_rope_backward_workspace_bytes(T, q_heads, k_heads, head_dim);
    if (workspace_bytes < need || (need > 0 && !workspace))
        return fail(QKN_ERR_INVALID_ARG, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes, (long long)need);
    w[nw++] = flat(dgamma_q, (int64_t)head_dim * 4, "dgamma_q");
    w[nw++] = flat(dgamma_k, (int64_t)head_dim * 4, "dgamma_k");
    if (need > 0) w[nw++] = flat(workspace, need, "workspace");
    r[nr++] = flat(cos_sin, table_rows * rotary_dim * 4, "cos_sin");
    r[nr++] = flat(positions, T * 8, "positions");
    const int in_place[] = {0, 0, 0, 1, 1, 3, 1, 4};  // dx over its own x or dy
    if ((st = check_written(w, nw, r, nr, in_place, 8)) != QKN_OK) return st;
    p.partial = static_cast<float *>(workspace);
    p.heads[0] = q_heads;
    p.heads[1] = k_heads;
    p.T = T;
    p.table = cos_sin;
    p.positions = positions;
    p.table_rows = table_rows;
    p.head_dim = head_dim;
    p.half = rotary_dim / 2;
    p.interleaved = interleaved ? 1 : 0;
    p.eps = eps;
    p.inv_d = static_cast<float>(1.0 / head_dim);
    const int64_t rows = T * ((int64_t)q_heads + k_heads);
    int64_t ctas = 0;
    if (T > 0) {
        p.lanes = aligned ? vector_lanes(dtype, head_dim, p.half) : 0;
        const void *fn;
        unsigned threads;
        size_t smem;
        if (p.lanes > 0) {
            p.units = head_dim / (2 * (16 / esz));
            int sms = 0;
            if ((st = device_sms(&sms)) != QKN_OK) return st;
            const int groups = head_groups(rows, 32 / p.lanes, sms, 4);
            p.chunk_heads = (32 / p.lanes) * groups;
            const int64_t items = T * (((int64_t)q_heads + p.chunk_heads - 1) / p.chunk_heads);  // Q's, the most
            const int64_t k_items = T * (((int64_t)k_heads + p.chunk_heads - 1) / p.chunk_heads);
            ctas = ((items > k_items ? items : k_items) + kGradWarps - 1) / kGradWarps;
            if (ctas > 2 * (int64_t)sms) ctas = 2 * (int64_t)sms;  // what is resident
            threads = kGradWarps * 32;
            smem = (size_t)kGradWarps * head_dim * 4;
            const bool exact = p.lanes == p.units;
            fn = dtype == QKN_F32    ? grad_kernel<float>(p.lanes, exact)
                 : dtype == QKN_BF16 ? grad_kernel<__nv_bfloat16>(p.lanes, exact)
                                     : grad_kernel<__half>(p.lanes, exact);
        } else {
            ctas = (rows + kGradScalarWarps - 1) / kGradScalarWarps;
            threads = kGradScalarWarps * 32;
            smem = (size_t)kGradScalarWarps * 2 * head_dim * 4;
            fn = dtype == QKN_F32    ? (const void *)heads_grad_scalar_kernel<float>
                 : dtype == QKN_BF16 ? (const void *)heads_grad_scalar_kernel<__nv_bfloat16>
                                     : (const void *)heads_grad_scalar_kernel<__half>;
        }
        if (ctas > grad_ctas(rows)) ctas = grad_ctas(rows);
        if ((st = launched(launch_pdl(fn, dim3((unsigned)ctas), threads, smem, stream, p))) != QKN_OK) return st;
    }
    GradSumParams g{};
    g.partial = p.partial;
    g.dgamma[0] = dgamma_q;
    g.dgamma[1] = dgamma_k;
    g.ctas = (int32_t)ctas;
    g.head_dim = head_dim;
    return launched(launch_pdl((const void *)dgamma_sum_kernel, dim3((unsigned)((2 * head_dim + 31) / 32)), dim3(32, kSumRows),
                               0, stream, g));
}

}  // extern "C"
