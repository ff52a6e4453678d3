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
// Every kernel is bound by memory traffic: each element is read once and
// written once (the gradient reads two rows and writes one).
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
// 4-bit codes.  Scales and codes are formed in 64 bits: they are then the
// rounded values of the formula whatever the order of the head's sums, so a
// token's cache entry does not depend on the kernel variant that wrote it
// (in 32 bits about one code in a million lands on the other side of its
// border).
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
// head read twice (the second time from cache).  C: the arithmetic's type.
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
            double *y = held[warp];
            if (which == 1) {
                const auto head = scalar_head<E, double>(p, row, p.gamma[1], t, lane);
                head.each(lane, [&](int i, double v) { y[i] = v; });
            } else {
                for (int i = lane; i < p.head_dim; i += 32) y[i] = static_cast<double>(elem_at<E>(row, i));
            }
            __syncwarp();
            const int64_t cell = (page * p.heads[1] + h) * p.page_size + off;
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
                reinterpret_cast<uint8_t *>(p.cache[kv])[cell * (p.head_dim / 2) + g * (kKv4Group / 2) + lane] =
                    static_cast<uint8_t>(lo | (hi << 4));
                if (lane == 0) p.scales[kv][cell * (p.head_dim / kKv4Group) + g] = sh;
            }
            __syncwarp();
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
// are neighbours.  A warp takes 32 / lanes heads at a time of one token and one
// tensor, U times, all loads first; the token's cosines and sines and the
// tensor's gamma are loaded once for all of them.
template <typename E>
struct LanePlace {
    int lo, hi;          // first elements of the two vectors
    bool turn_lo, turn_hi;
};
template <typename E, typename P>
__device__ __forceinline__ LanePlace<E> lane_place(const P &p, int u) {
    constexpr int V = Elem<E>::kPerVec;
    if (p.interleaved) {
        const int lo = u * V, hi = p.head_dim / 2 + u * V;
        return {lo, hi, lo < 2 * p.half, hi < 2 * p.half};
    }
    const int nr = p.half / V;
    if (u < nr) return {u * V, p.half + u * V, true, true};
    const int lo = 2 * p.half + 2 * (u - nr) * V;
    return {lo, lo + V, false, false};
}

// The lane's cosines and sines: of its V pairs (lo[e], hi[e]), or with
// neighbouring pairs of the V / 2 pairs of lo, then of hi.
template <typename E, typename P>
__device__ __forceinline__ void lane_turns(const P &p, const LanePlace<E> &at, const float *cs, float (&c)[Elem<E>::kPerVec],
                                           float (&s)[Elem<E>::kPerVec]) {
    constexpr int V = Elem<E>::kPerVec;
#pragma unroll
    for (int i = 0; i < V; i += 2) {
        const bool lo = !p.interleaved || i < V / 2;
        const int pair = p.interleaved ? (lo ? at.lo / 2 + i : at.hi / 2 + i - V / 2) : at.lo + i;
        if (cs && (lo ? at.turn_lo : at.turn_hi)) {
            const float2 a = __ldg(reinterpret_cast<const float2 *>(cs + pair));
            const float2 b = __ldg(reinterpret_cast<const float2 *>(cs + p.half + pair));
            c[i] = a.x, c[i + 1] = a.y, s[i] = b.x, s[i + 1] = b.y;
        } else {
            c[i] = c[i + 1] = 1.0f, s[i] = s[i + 1] = 0.0f;
        }
    }
}

// Rotates the lane's elements in place (`back`: by the opposite angle).
template <typename E, typename C>
__device__ __forceinline__ void lane_rotate(bool interleaved, C (&a)[Elem<E>::kPerVec], C (&b)[Elem<E>::kPerVec],
                                            const float (&c)[Elem<E>::kPerVec], const float (&s)[Elem<E>::kPerVec], C sign) {
    constexpr int V = Elem<E>::kPerVec;
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const C x = a[2 * i], y = a[2 * i + 1], sn = static_cast<C>(s[i]) * sign, cn = static_cast<C>(c[i]);
            a[2 * i] = x * cn - y * sn;
            a[2 * i + 1] = x * sn + y * cn;
            const C z = b[2 * i], w = b[2 * i + 1], sm = static_cast<C>(s[V / 2 + i]) * sign, cm = static_cast<C>(c[V / 2 + i]);
            b[2 * i] = z * cm - w * sm;
            b[2 * i + 1] = z * sm + w * cm;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const C x = a[i], y = b[i], sn = static_cast<C>(s[i]) * sign, cn = static_cast<C>(c[i]);
            a[i] = x * cn - y * sn;
            b[i] = x * sn + y * cn;
        }
    }
}

template <typename E, typename C>
__device__ __forceinline__ void widen_to(const uint4 &v, C (&x)[Elem<E>::kPerVec]) {
    F2 w[Elem<E>::kPerVec / 2];
    Elem<E>::widen(v, w);
#pragma unroll
    for (int i = 0; i < Elem<E>::kPerVec / 2; ++i) {
        x[2 * i] = static_cast<C>(f2_lo(w[i]));
        x[2 * i + 1] = static_cast<C>(f2_hi(w[i]));
    }
}
template <typename E>
__device__ __forceinline__ uint4 narrow_from(const float (&x)[Elem<E>::kPerVec]) {
    F2 w[Elem<E>::kPerVec / 2];
#pragma unroll
    for (int i = 0; i < Elem<E>::kPerVec / 2; ++i) w[i] = f2(x[2 * i], x[2 * i + 1]);
    return Elem<E>::narrow(w);
}
// gamma of the lane's vector at element `at`, as floats.
template <typename E>
__device__ __forceinline__ void lane_gamma(const char *gamma, int at, float (&g)[Elem<E>::kPerVec]) {
    using GE = typename Elem<E>::G;
    constexpr int KG = Elem<E>::kGVecs, N = Elem<GE>::kPerVec;
#pragma unroll
    for (int v = 0; v < KG; ++v) {
        float x[N];
        widen_to<GE, float>(ld_gamma(gamma + static_cast<int64_t>(at) * sizeof(GE) + 16 * v), x);
#pragma unroll
        for (int i = 0; i < N; ++i) g[v * N + i] = x[i];
    }
}
__device__ __forceinline__ float lanes_sum(float v, int lanes) { return segment_sum(v, lanes); }
__device__ __forceinline__ double lanes_sum(double v, int lanes) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        if (off < lanes) v += __shfl_xor_sync(0xFFFFFFFFu, v, off);
    return v;
}

// Norm and rotation of the lane's elements, in C.
template <typename E, typename C>
__device__ __forceinline__ void lane_forward(const RopeParams &p, bool norm, int turn, const float (&ga)[Elem<E>::kPerVec],
                                             const float (&gb)[Elem<E>::kPerVec], const float (&c)[Elem<E>::kPerVec],
                                             const float (&s)[Elem<E>::kPerVec], C (&a)[Elem<E>::kPerVec],
                                             C (&b)[Elem<E>::kPerVec]) {
    constexpr int V = Elem<E>::kPerVec;
    if (norm) {
        C even = C(0), odd = C(0);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            even = fma(a[i], a[i], even);
            odd = fma(b[i], b[i], odd);
        }
        const C r = norm_factor(lanes_sum(even + odd, p.lanes), p);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            a[i] = a[i] * static_cast<C>(ga[i]) * r;
            b[i] = b[i] * static_cast<C>(gb[i]) * r;
        }
    }
    lane_rotate<E, C>(p.interleaved, a, b, c, s, C(1));
    if (turn != kTurnRow) {
        const C v = turn == kTurnPad ? C(0) : C(__uint_as_float(0x7FFFFFFFu));
#pragma unroll
        for (int i = 0; i < V; ++i) a[i] = b[i] = v;
    }
}

// The lane's elements to codes and, by the first lanes, the groups' scales.
template <int V>
__device__ __forceinline__ void store_codes(uint8_t *codes, int at, const uint32_t (&c)[V]) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) w |= c[i] << (4 * i);
    if constexpr (V == 8) *reinterpret_cast<uint32_t *>(codes + at / 2) = w;
    else *reinterpret_cast<uint16_t *>(codes + at / 2) = static_cast<uint16_t>(w);
}
template <typename E>
__device__ __forceinline__ void lane_quantise(const RopeParams &p, int u, bool store, const LanePlace<E> &at,
                                              const double (&a)[Elem<E>::kPerVec], const double (&b)[Elem<E>::kPerVec],
                                              uint8_t *codes, __half *scales) {
    constexpr int V = Elem<E>::kPerVec;
    double ma = 0.0, mb = 0.0;
    bool bad_a = false, bad_b = false;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        ma = fmax(ma, fabs(a[i]));
        mb = fmax(mb, fabs(b[i]));
        bad_a |= !isfinite(a[i]);
        bad_b |= !isfinite(b[i]);
    }
    const int group_a = at.lo / kKv4Group, group_b = at.hi / kKv4Group, groups = p.head_dim / kKv4Group;
    const int lane = threadIdx.x & 31;
    const uint32_t seg = (p.lanes == 32 ? 0xFFFFFFFFu : ((1u << p.lanes) - 1u) << (lane & ~(p.lanes - 1)));
    double sa = 0.0, sb = 0.0;
    for (int g = 0; g < groups; ++g) {
        double m = fmax(group_a == g ? ma : 0.0, group_b == g ? mb : 0.0);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1)
            if (off < p.lanes) m = fmax(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
        const bool bad = (__ballot_sync(0xFFFFFFFFu, (group_a == g && bad_a) || (group_b == g && bad_b)) & seg) != 0;
        const __half sh = kv4_scale(m, bad);
        const double s = static_cast<double>(__half2float(sh));
        if (group_a == g) sa = s;
        if (group_b == g) sb = s;
        if (store && u == g) scales[g] = sh;
    }
    uint32_t ca[V], cb[V];
    const double ia = 1.0 / sa, ib = 1.0 / sb;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        ca[i] = sa > 0.0 ? kv4_code(a[i], sa, ia) : 8u;
        cb[i] = sb > 0.0 ? kv4_code(b[i], sb, ib) : 8u;
    }
    if (store) {
        store_codes<V>(codes, at.lo, ca);
        store_codes<V>(codes, at.hi, cb);
    }
}

constexpr int kVectorWarps = 8;

template <typename E, int U, int SINK>
__global__ void __launch_bounds__(kVectorWarps * 32) heads_vector_kernel(const __grid_constant__ RopeParams p) {
    constexpr int V = Elem<E>::kPerVec;
    constexpr int kEsz = sizeof(typename Elem<E>::Bits);
    pdl_wait_and_release();
    const uint32_t item = blockIdx.x * kVectorWarps + (threadIdx.x >> 5);
    const uint32_t t32 = item / static_cast<uint32_t>(p.chunks);
    const int64_t t = t32;
    if (t >= p.T) return;
    int chunk = static_cast<int>(item - t32 * p.chunks);
    const int lane = threadIdx.x & 31, u = lane & (p.lanes - 1), per = 32 / p.lanes, first = lane / p.lanes;
    // which tensor: Q's chunks, then K's, then V's
    int which = 0;
    if (chunk >= p.chunks_of[0]) {
        chunk -= p.chunks_of[0];
        which = 1;
        if (chunk >= p.chunks_of[1]) {
            chunk -= p.chunks_of[1];
            which = 2;
        }
    }
    const int heads = p.heads[which];
    const bool active = u < p.units;
    const LanePlace<E> at = lane_place<E>(p, active ? u : 0);
    const char *in = p.in[which] + t * p.stride[which];
    const int head_bytes = p.head_dim * kEsz;

    if (SINK == kSinkKv4 && which > 0) {  // one head of a lane group at a time, in 64 bits
        const int h = chunk * per + first;
        const bool there = active && h < heads;
        uint4 va = make_uint4(0, 0, 0, 0), vb = va;
        if (there) {
            va = ld_stream(in + static_cast<int64_t>(h) * head_bytes + at.lo * kEsz);
            vb = ld_stream(in + static_cast<int64_t>(h) * head_bytes + at.hi * kEsz);
        }
        const int64_t slot = p.slots[t];
        if constexpr (SINK == kSinkKv4) {
            double a[V], b[V];
            widen_to<E, double>(va, a);
            widen_to<E, double>(vb, b);
            if (which == 1) {
                const int64_t pos = p.positions[t];
                const int turn = turn_of(pos, p.table_rows);
                float c[V], s[V], ga[V] = {}, gb[V] = {};
                lane_turns<E>(p, at, turn == kTurnRow ? p.table + pos * 2 * p.half : nullptr, c, s);
                if (p.gamma[1]) {
                    lane_gamma<E>(p.gamma[1], at.lo, ga);
                    lane_gamma<E>(p.gamma[1], at.hi, gb);
                }
                lane_forward<E, double>(p, p.gamma[1] != nullptr, turn, ga, gb, c, s, a, b);
            }
            const bool store = there && slot >= 0 && slot < p.num_slots;
            const int64_t page = store ? slot / p.page_size : 0;
            const int64_t cell = (page * heads + h) * p.page_size + (store ? slot - page * p.page_size : 0);
            const int kv = which - 1;
            lane_quantise<E>(p, u, store, at, a, b, reinterpret_cast<uint8_t *>(p.cache[kv]) + cell * (p.head_dim / 2),
                             p.scales[kv] + cell * (p.head_dim / kKv4Group));
        }
        return;
    }

    uint4 va[U], vb[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
        const int h = (chunk * U + j) * per + first;
        va[j] = vb[j] = make_uint4(0, 0, 0, 0);
        if (active && h < heads) {
            va[j] = ld_stream(in + static_cast<int64_t>(h) * head_bytes + at.lo * kEsz);
            vb[j] = ld_stream(in + static_cast<int64_t>(h) * head_bytes + at.hi * kEsz);
        }
    }
    char *out;
    int64_t step = head_bytes;
    if (SINK == kSinkRows || which == 0) {
        out = p.out[which] + t * p.stride[which];
    } else {
        const int64_t slot = p.slots[t];
        if (slot < 0 || slot >= p.num_slots) return;
        const int64_t page = slot / p.page_size, off = slot - page * p.page_size;
        out = p.cache[which - 1] + page * p.page_stride[which - 1] + off * p.token_stride[which - 1];
        step = p.head_stride[which - 1];
        if (which == 2) {
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int h = (chunk * U + j) * per + first;
                if (active && h < heads) {
                    *reinterpret_cast<uint4 *>(out + h * step + at.lo * kEsz) = va[j];
                    *reinterpret_cast<uint4 *>(out + h * step + at.hi * kEsz) = vb[j];
                }
            }
            return;
        }
    }
    const int64_t pos = p.positions[t];
    const int turn = turn_of(pos, p.table_rows);
    float c[V], s[V], ga[V] = {}, gb[V] = {};
    lane_turns<E>(p, at, turn == kTurnRow ? p.table + pos * 2 * p.half : nullptr, c, s);
    const char *gamma = p.gamma[which];
    if (gamma) {
        lane_gamma<E>(gamma, at.lo, ga);
        lane_gamma<E>(gamma, at.hi, gb);
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
        const int h = (chunk * U + j) * per + first;
        float a[V], b[V];
        widen_to<E, float>(va[j], a);
        widen_to<E, float>(vb[j], b);
        lane_forward<E, float>(p, gamma != nullptr, turn, ga, gb, c, s, a, b);
        if (active && h < heads) {
            st_stream(out + h * step + at.lo * kEsz, narrow_from<E>(a));
            st_stream(out + h * step + at.hi * kEsz, narrow_from<E>(b));
        }
    }
}

// Gradient of aligned heads: the same placing; CTAs stay and take tokens and
// heads in turn, so that a lane keeps its elements' dgamma sums in registers,
// first over Q's heads, then over K's; they are added over the warp's lane
// groups, then over the warps in order.
template <typename E, int U>
__global__ void __launch_bounds__(kVectorWarps * 32) heads_grad_vector_kernel(const __grid_constant__ RopeGradParams p) {
    constexpr int V = Elem<E>::kPerVec;
    constexpr int kEsz = sizeof(typename Elem<E>::Bits);
    pdl_wait_and_release();
    extern __shared__ float sums[];  // [warps][head_dim]
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int u = lane & (p.lanes - 1), per = 32 / p.lanes, first = lane / p.lanes;
    const bool active = u < p.units;
    const LanePlace<E> at = lane_place<E>(p, active ? u : 0);
    const int head_bytes = p.head_dim * kEsz;
    for (int w = 0; w < 2; ++w) {
        float ga[V], gb[V], da[V] = {}, db[V] = {};
        lane_gamma<E>(p.gamma[w], at.lo, ga);
        lane_gamma<E>(p.gamma[w], at.hi, gb);
        const int heads = p.heads[w];
        const uint32_t chunks = (heads + per * U - 1) / (per * U);
        const int64_t items = p.T * chunks;
        for (int64_t item = static_cast<int64_t>(blockIdx.x) * kVectorWarps + warp; item < items;
             item += static_cast<int64_t>(gridDim.x) * kVectorWarps) {
            const uint32_t t32 = static_cast<uint32_t>(item) / chunks;
            const int64_t t = t32;
            const int chunk = static_cast<int>(static_cast<uint32_t>(item) - t32 * chunks);
            uint4 xa[U], xb[U], ya[U], yb[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int h = (chunk * U + j) * per + first;
                xa[j] = xb[j] = ya[j] = yb[j] = make_uint4(0, 0, 0, 0);
                if (active && h < heads) {
                    const char *x = p.x[w] + t * p.x_stride[w] + static_cast<int64_t>(h) * head_bytes;
                    const char *y = p.dy[w] + t * p.dy_stride[w] + static_cast<int64_t>(h) * head_bytes;
                    xa[j] = ld_stream(x + at.lo * kEsz);
                    xb[j] = ld_stream(x + at.hi * kEsz);
                    ya[j] = ld_stream(y + at.lo * kEsz);
                    yb[j] = ld_stream(y + at.hi * kEsz);
                }
            }
            const int64_t pos = p.positions[t];
            const int turn = turn_of(pos, p.table_rows);
            float c[V], s[V];
            lane_turns<E>(p, at, turn == kTurnRow ? p.table + pos * 2 * p.half : nullptr, c, s);
#pragma unroll
            for (int j = 0; j < U; ++j) {
                const int h = (chunk * U + j) * per + first;
                float a[V], b[V], ua[V], ub[V];
                widen_to<E, float>(xa[j], a);
                widen_to<E, float>(xb[j], b);
                widen_to<E, float>(ya[j], ua);
                widen_to<E, float>(yb[j], ub);
                lane_rotate<E, float>(p.interleaved, ua, ub, c, s, -1.0f);
                float S = 0.0f, M = 0.0f;
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    S = fmaf(a[i], a[i], S);
                    S = fmaf(b[i], b[i], S);
                    M = fmaf(ua[i] * ga[i], a[i], M);
                    M = fmaf(ub[i] * gb[i], b[i], M);
                }
                S = lanes_sum(S, p.lanes);
                M = lanes_sum(M, p.lanes);
                const float r = rms_factor(S, p.inv_d, p.eps);
                const float k = r * r * M * p.inv_d;
                const bool there = active && h < heads;
                const float past = __uint_as_float(0x7FFFFFFFu);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float ea = ua[i] * a[i] * r, eb = ub[i] * b[i] * r;
                    a[i] = r * (ua[i] * ga[i] - a[i] * k);
                    b[i] = r * (ub[i] * gb[i] - b[i] * k);
                    if (turn != kTurnRow) ea = eb = a[i] = b[i] = turn == kTurnPad ? 0.0f : past;
                    da[i] += there ? ea : 0.0f;
                    db[i] += there ? eb : 0.0f;
                }
                if (there) {
                    char *dx = p.dx[w] + t * p.dx_stride[w] + static_cast<int64_t>(h) * head_bytes;
                    st_stream(dx + at.lo * kEsz, narrow_from<E>(a));
                    st_stream(dx + at.hi * kEsz, narrow_from<E>(b));
                }
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
            for (int off = p.lanes; off < 32; off <<= 1) {
                da[i] += __shfl_xor_sync(0xFFFFFFFFu, da[i], off);
                db[i] += __shfl_xor_sync(0xFFFFFFFFu, db[i], off);
            }
        if (first == 0 && active)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                sums[warp * p.head_dim + at.lo + i] = da[i];
                sums[warp * p.head_dim + at.hi + i] = db[i];
            }
        __syncthreads();
        for (int i = threadIdx.x; i < p.head_dim; i += kVectorWarps * 32) {
            float v = 0.0f;
#pragma unroll
            for (int k = 0; k < kVectorWarps; ++k) v += sums[k * p.head_dim + i];
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
// Cached tokens of the 4-bit cache back as rows: one thread per 8 elements.
struct Kv4ReadParams {
    const uint8_t *codes[2];
    const __half *scales[2];
    char *out[2];
    int64_t stride[2];  // bytes
    const int64_t *slots;
    int64_t n, num_slots;
    int32_t page_size, heads, head_dim, words;  // words: 8-element words of a token's heads
};
template <typename E>
__global__ void __launch_bounds__(256) kv4_read_kernel(const __grid_constant__ Kv4ReadParams p) {
    pdl_wait_and_release();
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t total = p.n * 2 * p.words;
    if (i >= total) return;
    const int64_t t = i / (2 * p.words);
    int w = static_cast<int>(i - t * 2 * p.words);
    const int kv = w >= p.words;
    w -= kv * p.words;
    const int per_head = p.head_dim / 8, h = w / per_head, j = w - h * per_head;
    const int64_t slot = p.slots[t];
    uint32_t codes = 0x88888888u;
    float s = 0.0f;
    if (slot >= 0 && slot < p.num_slots) {
        const int64_t page = slot / p.page_size, off = slot - page * p.page_size;
        const int64_t cell = (page * p.heads + h) * p.page_size + off;
        codes = reinterpret_cast<const uint32_t *>(p.codes[kv])[cell * per_head + j];
        s = __half2float(p.scales[kv][cell * (p.head_dim / kKv4Group) + j * 8 / kKv4Group]);
    }
    char *out = p.out[kv] + t * p.stride[kv];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float v = static_cast<float>(static_cast<int>((codes >> (4 * e)) & 15u) - 8) * s;
        put_elem<E>(out, w * 8 + e, v);
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

template <int SINK, int U>
const void *vector_kernel(int dt) {
    switch (dt) {
        case QKN_F32: return (const void *)heads_vector_kernel<float, U, SINK>;
        case QKN_BF16: return (const void *)heads_vector_kernel<__nv_bfloat16, U, SINK>;
        case QKN_F16: return (const void *)heads_vector_kernel<__half, U, SINK>;
        default:
            if constexpr (SINK == kSinkKv4) return nullptr;
            else return (const void *)heads_vector_kernel<__nv_fp8_e4m3, U, SINK>;
    }
}

// Lanes of a head for the vector kernels; 0 where the sizes do not fit them.
int vector_lanes(int dtype, int head_dim, int half) {
    const int two = 2 * (16 / elem_bytes(dtype));  // elements of two vectors
    if (head_dim % two != 0 || 2 * half % two != 0 || head_dim / two > 32) return 0;
    int lanes = 1;
    while (lanes < head_dim / two) lanes *= 2;
    return lanes;
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
        // four heads in flight per lane group once that leaves every SM warps enough
        const int U = rows >= (int64_t)sms * 32 * per * 4 ? 4 : 1;
        p.chunks = 0;
        for (int i = 0; i < 3; ++i) {
            const int n = per * (SINK == kSinkKv4 && i > 0 ? 1 : U);
            p.chunks_of[i] = (p.heads[i] + n - 1) / n;
            p.chunks += p.chunks_of[i];
        }
        const int64_t ctas = (p.T * p.chunks + kVectorWarps - 1) / kVectorWarps;
        const void *fn = U == 4 ? vector_kernel<SINK, 4>(dtype) : vector_kernel<SINK, 1>(dtype);
        return launched(launch_pdl(fn, dim3((unsigned)ctas), kVectorWarps * 32, 0, stream, p));
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
    if (heads < 1 || heads > (1 << 20)) return fail(QKN_ERR_INVALID_ARG, "%lld heads", (long long)heads);
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
    if (threads > ((__int128)1 << 31) * 255) return fail(QKN_ERR_INVALID_ARG, "n * kv_heads * head_dim too large");
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
    if (heads > (1 << 20) || (T > 0 && T >= ((int64_t)1 << 31) / heads)) return -1;
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
            const int64_t heads = (int64_t)kVectorWarps * (32 / p.lanes);
            ctas = (rows + heads - 1) / heads;
            threads = kVectorWarps * 32;
            smem = (size_t)kVectorWarps * head_dim * 4;
            fn = dtype == QKN_F32    ? (const void *)heads_grad_vector_kernel<float, 2>
                 : dtype == QKN_BF16 ? (const void *)heads_grad_vector_kernel<__nv_bfloat16, 2>
                                     : (const void *)heads_grad_vector_kernel<__half, 2>;
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
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((2 * head_dim + 31) / 32));
    cfg.blockDim = dim3(32, kSumRows);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *args[] = {&g};
    return launched(cudaLaunchKernelExC(&cfg, (const void *)dgamma_sum_kernel, args));
}

}  // extern "C"
