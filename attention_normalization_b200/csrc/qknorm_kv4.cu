// Attention over the paged 4-bit cache (qknorm_kv4_attention in
// include/qknorm.h).
//
// Mathematics, for a query row q of a sequence with `len` cached tokens and
// the query at position pos: over the tokens t <= pos (t > pos - window with a
// window) of its sequence,
//   s_t = scale * sum_d q_d k_td,  m = max s_t,  p_t = exp(s_t - m),  l = sum p_t,
//   out_d = sum_t p_t v_td / l,  lse = m + log l,
// with k_td = (code - 8) * (the scale of d's group).  A row without tokens
// gives zeros and lse = -infinity.
#include <cuda_runtime.h>
#include <stdint.h>

#include "qknorm.h"
#include "qknorm_checks.cuh"
#include "qknorm_kernels.cuh"
#include "qknorm_rope.cuh"

namespace qkn {
namespace {

struct Kv4AttnParams {
    const char *q;
    char *out;
    float *lse;                  // [T][q_heads], may be null
    int64_t q_stride, out_stride;  // bytes
    const uint8_t *codes[2];
    const __half *scales[2];
    const int32_t *block_table;  // [B][max_pages]
    const int32_t *seq_lens;     // [B]
    const int32_t *q_start;      // [B + 1], null: one row per sequence
    int64_t T, table_stride, num_pages;
    int32_t max_pages, page_size, B, q_heads, kv_heads, group, max_q_len, max_seq_len, window;
    float scale;
};

// Rows and cached tokens of sequence b, kept inside the buffers.
struct Seq {
    int64_t row0;
    int32_t rows, len;
};
__device__ __forceinline__ Seq sequence(const Kv4AttnParams &p, int b) {
    Seq s{b, 1, 0};
    if (p.q_start) {
        const int64_t a = p.q_start[b], e = p.q_start[b + 1];
        s.row0 = a;
        s.rows = a < 0 || e <= a ? 0 : static_cast<int32_t>(e - a < p.max_q_len ? e - a : p.max_q_len);
    }
    if (s.row0 + s.rows > p.T) s.rows = s.row0 < p.T ? static_cast<int32_t>(p.T - s.row0) : 0;
    int64_t len = p.seq_lens[b];
    const int64_t held = static_cast<int64_t>(p.max_pages) * p.page_size;
    if (len > p.max_seq_len) len = p.max_seq_len;
    if (len > held) len = held;
    s.len = len < 0 ? 0 : static_cast<int32_t>(len);
    return s;
}

// One warp per row and query head; lane l holds elements l * D / 32 ...
template <typename E, int D>
__global__ void __launch_bounds__(256) kv4_attention_simple(const __grid_constant__ Kv4AttnParams p) {
    pdl_wait_and_release();
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.y;
    const Seq s = sequence(p, b);
    const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + warp;
    const int i = static_cast<int>(item / p.q_heads), h = static_cast<int>(item % p.q_heads);
    if (i >= s.rows) return;
    const int64_t row = s.row0 + i;
    const int kvh = h / p.group;
    float q[N], o[N];
    const char *qp = p.q + row * p.q_stride + static_cast<int64_t>(h) * D * sizeof(E);
    for (int e = 0; e < N; ++e) {
        q[e] = Elem<E>::to_float(reinterpret_cast<const typename Elem<E>::Bits *>(qp)[lane * N + e]) * p.scale;
        o[e] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    const int pos = s.len - s.rows + i;
    const int first = p.window > 0 && pos - p.window + 1 > 0 ? pos - p.window + 1 : 0;
    for (int t = first; t <= pos; ++t) {
        const int32_t page = p.block_table[b * p.table_stride + t / p.page_size];
        if (page < 0 || page >= p.num_pages) continue;
        const int64_t cell = (static_cast<int64_t>(page) * p.kv_heads + kvh) * p.page_size + t % p.page_size;
        const int at = lane * N;
        float sc[2];
        float v[2][N];
        for (int kv = 0; kv < 2; ++kv) {
            sc[kv] = __half2float(p.scales[kv][cell * (D / kKv4Group) + at / kKv4Group]);
            for (int e = 0; e < N; ++e) {
                const uint8_t c = p.codes[kv][cell * (D / 2) + (at + e) / 2];
                v[kv][e] = static_cast<float>(static_cast<int>((e & 1) ? c >> 4 : c & 15) - 8) * sc[kv];
            }
        }
        float dot = 0.0f;
        for (int e = 0; e < N; ++e) dot += q[e] * v[0][e];
        dot = warp_sum(dot);
        const float mn = fmaxf(m, dot);
        const float up = mn == -INFINITY ? 1.0f : __expf(m - mn), w = dot == -INFINITY ? 0.0f : __expf(dot - mn);
        l = l * up + w;
        for (int e = 0; e < N; ++e) o[e] = o[e] * up + w * v[1][e];
        m = mn;
    }
    char *op = p.out + row * p.out_stride + static_cast<int64_t>(h) * D * sizeof(E);
    for (int e = 0; e < N; ++e)
        reinterpret_cast<typename Elem<E>::Bits *>(op)[lane * N + e] = Elem<E>::from_float(l == 0.0f ? 0.0f : o[e] / l);
    if (lane == 0 && p.lse) p.lse[row * p.q_heads + h] = l == 0.0f ? -INFINITY : m + __logf(l);
}

using namespace checks;

template <typename E>
const void *simple_kernel(int d) {
    return d == 64    ? (const void *)kv4_attention_simple<E, 64>
           : d == 128 ? (const void *)kv4_attention_simple<E, 128>
                      : (const void *)kv4_attention_simple<E, 256>;
}

}  // namespace
}  // namespace qkn

using namespace qkn;
using namespace qkn::checks;

extern "C" {

int64_t qknorm_kv4_attention_workspace_bytes(int64_t T, int32_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                             int32_t max_q_len, int32_t max_seq_len) {
    if (T < 0 || B < 0 || q_heads < 1 || kv_heads < 1 || head_dim < 1 || max_q_len < 1 || max_seq_len < 0) return -1;
    return 0;
}

qkn_status qknorm_kv4_attention(const void *q, int64_t q_stride, void *out, int64_t out_stride, float *lse,
                                int32_t q_heads, const void *k_codes, const void *k_scales, const void *v_codes,
                                const void *v_scales, int64_t num_pages, int32_t page_size, int32_t kv_heads,
                                int32_t head_dim, const int32_t *block_table, int32_t max_pages,
                                const int32_t *seq_lens, const int32_t *q_start, int64_t T, int32_t B,
                                int32_t max_q_len, int32_t max_seq_len, int32_t window, float scale, void *workspace,
                                int64_t workspace_bytes, qkn_dtype dtype, void *stream) {
    if (dtype < QKN_F32 || dtype > QKN_FP8_E4M3) return fail(QKN_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (dtype != QKN_BF16 && dtype != QKN_F16) return fail(QKN_ERR_UNSUPPORTED, "attention takes bfloat16 or float16 queries");
    int64_t codes = 0, scales = 0;
    if (T < 0 || B < 0 || max_q_len < 1 || max_seq_len < 0 || max_pages < 0 || window < 0)
        return fail(QKN_ERR_INVALID_ARG, "T = %lld, B = %d, max_q_len = %d, max_seq_len = %d, max_pages = %d, window = %d",
                    (long long)T, B, max_q_len, max_seq_len, max_pages, window);
    qkn_status st = check_kv4(num_pages, page_size, kv_heads, head_dim, k_codes, k_scales, v_codes, v_scales,
                              T > 0 && num_pages > 0, &codes, &scales);
    if (st != QKN_OK) return st;
    if (q_heads < 1 || q_heads % kv_heads != 0)
        return fail(QKN_ERR_INVALID_ARG, "q_heads = %d must be a multiple of kv_heads = %d", q_heads, kv_heads);
    if (!(std::isfinite(scale))) return fail(QKN_ERR_INVALID_ARG, "scale must be finite");
    if (T >= ((int64_t)1 << 31) / q_heads) return fail(QKN_ERR_INVALID_ARG, "T * q_heads must stay below 2^31");
    if (B > 65535) return fail(QKN_ERR_UNSUPPORTED, "at most 65535 sequences");
    if (!q_start && (max_q_len != 1 || T < B))
        return fail(QKN_ERR_INVALID_ARG, "without q_start row b is sequence b's one query: T >= B, max_q_len 1");
    const int64_t width = (int64_t)q_heads * head_dim;
    if (q_stride < width || out_stride < width)
        return fail(QKN_ERR_INVALID_ARG, "row stride below the width %lld", (long long)width);
    if (!extent_ok(T, q_stride, width, 2) || !extent_ok(T, out_stride, width, 2))
        return fail(QKN_ERR_INVALID_ARG, "buffer extent overflows");
    if (T > 0 && B > 0 && (!q || !out || !seq_lens || (!block_table && max_pages > 0)))
        return fail(QKN_ERR_INVALID_ARG, "null pointer");
    if (((uintptr_t)q | (uintptr_t)out) & 1u || ((uintptr_t)lse | (uintptr_t)block_table | (uintptr_t)seq_lens | (uintptr_t)q_start) & 3u)
        return fail(QKN_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
    const int64_t need = qknorm_kv4_attention_workspace_bytes(T, B, q_heads, kv_heads, head_dim, max_q_len, max_seq_len);
    if (need < 0) return fail(QKN_ERR_INVALID_ARG, "sizes out of range");
    if (workspace_bytes < need || (need > 0 && !workspace))
        return fail(QKN_ERR_INVALID_ARG, "workspace of %lld bytes, %lld needed", (long long)workspace_bytes, (long long)need);
    if (need > 0 && !aligned16(workspace)) return fail(QKN_ERR_INVALID_ARG, "the workspace must be 16-byte aligned");
    if (T == 0 || B == 0) return ok();
    Span w[3], r[8];
    int nw = 0, nr = 0;
    w[nw++] = Span{out, width * 2, out_stride * 2, T, "out"};
    if (lse) w[nw++] = flat(lse, T * q_heads * 4, "lse");
    if (need > 0) w[nw++] = flat(workspace, need, "workspace");
    r[nr++] = Span{q, width * 2, q_stride * 2, T, "q"};
    if (num_pages > 0) {
        r[nr++] = flat(k_codes, codes, "k_codes");
        r[nr++] = flat(k_scales, scales, "k_scales");
        r[nr++] = flat(v_codes, codes, "v_codes");
        r[nr++] = flat(v_scales, scales, "v_scales");
    }
    r[nr++] = flat(block_table, (int64_t)B * max_pages * 4, "block_table");
    r[nr++] = flat(seq_lens, (int64_t)B * 4, "seq_lens");
    r[nr++] = flat(q_start, ((int64_t)B + 1) * 4, "q_start");
    if ((st = check_written(w, nw, r, nr, nullptr, 0)) != QKN_OK) return st;
    Kv4AttnParams p{};
    p.q = static_cast<const char *>(q);
    p.out = static_cast<char *>(out);
    p.lse = lse;
    p.q_stride = q_stride * 2;
    p.out_stride = out_stride * 2;
    p.codes[0] = static_cast<const uint8_t *>(k_codes);
    p.codes[1] = static_cast<const uint8_t *>(v_codes);
    p.scales[0] = static_cast<const __half *>(k_scales);
    p.scales[1] = static_cast<const __half *>(v_scales);
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.q_start = q_start;
    p.T = T;
    p.table_stride = max_pages;
    p.num_pages = num_pages;
    p.max_pages = max_pages;
    p.page_size = page_size;
    p.B = B;
    p.q_heads = q_heads;
    p.kv_heads = kv_heads;
    p.group = q_heads / kv_heads;
    p.max_q_len = max_q_len;
    p.max_seq_len = max_seq_len;
    p.window = window;
    p.scale = scale;
    const void *fn = dtype == QKN_BF16 ? simple_kernel<__nv_bfloat16>(head_dim) : simple_kernel<__half>(head_dim);
    const int64_t items = (int64_t)max_q_len * q_heads;
    return launched(launch_pdl(fn, dim3((unsigned)((items + 7) / 8), (unsigned)B), 256, 0, stream, p));
}

}  // extern "C"
