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

#include <atomic>

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
    int32_t q_vector, out_vector;  // rows move as 16-byte (8-byte) vectors
    int32_t n_tiles;               // query tile: 8 * n_tiles rows
    int32_t row_tiles;             // query tiles of a sequence at most
    int32_t shared;                // whether units are cut at the CTAs' shares (else one CTA per unit)
    float *part_o;                 // shared: [grid][2][rows of a tile][head_dim], partial outputs
    float2 *part_s;                // and their (exponent, sum) pairs
    int32_t *starts;               // [B * row_tiles] first tile of each sequence and query tile, then the share
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

// a / b for 0 <= a < 2^21, b > 0: (a + 1/2) / b lies at least 1 / (2b) from the
// integers, further than the reciprocal's error can move it.
__device__ __forceinline__ int small_div(int a, int b) {
    return static_cast<int>((static_cast<float>(a) + 0.5f) * __frcp_rn(static_cast<float>(b)));
}

// Four elements of the output, sum / total (zeros for a row without tokens).
template <typename E>
__device__ __forceinline__ void store_row(const Kv4AttnParams &p, int64_t row, int64_t at, const float4 &sum, float total) {
    const float f = total == 0.0f ? 0.0f : 1.0f / total;
    typename Elem<E>::Bits *out = reinterpret_cast<typename Elem<E>::Bits *>(p.out + row * p.out_stride) + at;
    const uint32_t lo = Elem<E>::narrow_word(f2(sum.x * f, sum.y * f)), hi = Elem<E>::narrow_word(f2(sum.z * f, sum.w * f));
    if (p.out_vector) {
        *reinterpret_cast<uint2 *>(out) = make_uint2(lo, hi);
    } else {
        out[0] = static_cast<uint16_t>(lo);
        out[1] = static_cast<uint16_t>(lo >> 16);
        out[2] = static_cast<uint16_t>(hi);
        out[3] = static_cast<uint16_t>(hi >> 16);
    }
}
__device__ __forceinline__ float finish_lse(float m, float total) {  // base 2 -> natural
    return total == 0.0f ? -INFINITY : (m + log2f(total)) * 0.6931471805599453f;
}

// ----------------------------------------------------------------------------
// A unit is a tile of 8 * NT query rows of one sequence that read the same KV
// head (row r = token r / group, head r % group) with the 16-token tiles they
// see.  With many units or short sequences a CTA takes one; otherwise all units'
// tiles, end to end, are cut into equal shares, one per resident CTA, whatever
// the sequences' lengths, and a unit that a cut goes through is joined by a
// second launch.  A CTA's warps take a unit's tiles in turn, each with its own
// running maximum, sum and output, joined at the end of the unit.
//
// Scores are formed transposed, S^T = K Q^T, and so is the output, O^T = V^T P^T,
// with mma.m16n8k16: the 16 rows are cached tokens (or value dims), the 8
// columns query rows, so that one decoded token with up to 8 heads per KV head
// wastes nothing of a tile, and a thread's score columns are its output
// columns.  The codes are the A operand straight from registers: a nibble
// n = code + 8 becomes a half by one logic operation (1024 + n or 64 + n) and one
// exact subtraction, nine operations for eight nibbles.  Five are enough for the
// subnormals n 2^-24 and n 2^-20 that masked words are already, with the 8 taken
// off the sums; but the tensor cores align a sum's terms by their exponent
// fields, and a subnormal's leading zeros are bits the sum loses (errors of 2^-10
// of a code step were seen).
// The group scales stay out of the products: a key's scale multiplies the
// finished dot product of its group, a value's scale its weight, so each product
// is code * half, exact in fp32.
//
// Queries are scaled by a power of two per row to fit halves without loss
// (elements 2^-24 below the row's largest lose bits that fp32 sums of the row
// would not see either).  Weights are rounded to halves, 2^-11 relative, for
// what the tensor cores multiply.  What is rounded is p * (value scale), each
// group of dims against a reference of its own, the largest such product of the
// row so far, kept at 2^7 or more: a product loses bits below 2^-21 of it and
// goes to zero below 2^-32, whatever the other groups' scales are.  (One
// reference for all groups loses the tail of a group whose scales lie far below
// another's.)  The row sum l takes the unrounded weights.
//
// References are whole powers of two, so moving one rounds nothing.  They move
// only when a scaled weight would exceed 2^15, or a weight 2^75 where the values
// are (nearly) zeros: one vote per step.  The exact maximum is not needed, as O
// has its group's reference until the end and l the first group's.
// Instructions bound it: 308 a warp for 16 tokens of 128 dims and 8 rows,
// 146 of them codes to halves and 16 products (one B200: one token for each of 64
// sequences of 1024 to 4096 tokens, 32 heads over 8, 61 us, 2.9 TB/s; one of
// 131072 tokens 45 us, 3.2 TB/s; the loads alone take 47 and 41 us; with one
// reference for all groups 60 and 45 us).  4 warps a
// CTA: with 8 the batch took 72 us.
constexpr int kAttnWarps = 4;
constexpr int kLeastShare = 32;  // tiles: 8 for each warp
// What beginning and ending a unit costs a CTA, in tiles: shares are equal in
// tiles and units alike (64 sequences of 1024 to 4096 tokens, 8 KV heads: 63.4 us
// without this, 60.3 us with it).
constexpr int kUnitCost = 16;
constexpr float kOffset = 8.0f, kLargest = 32768.0f, kMostWeight = 3.7778931862957162e22f;  // 2^75

template <int D>
struct Kv4Tile {  // bytes of one 16-token tile of one KV head
    static constexpr int kGroups = D / kKv4Group;
    static constexpr int kCodes = 16 * D / 2;
    static constexpr int kScales = 16 * kGroups * 2;
    static constexpr int kBytes = 2 * (kCodes + kScales);  // K codes, V codes, K scales, V scales
    static constexpr int kStages = D == 256 ? 2 : 3;       // steps of two tiles in a warp's ring
    static constexpr int kRing = kStages * 2 * kBytes;
};

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t mask_or(uint32_t w, uint32_t mask, uint32_t magic) {  // (w & mask) | magic
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(w), "r"(mask), "r"(magic));
    return d;
}
__device__ __forceinline__ uint32_t sub_half2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// Codes i and i + 4 of w as halves, i = 0 .. 3.
__device__ __forceinline__ void codes8(uint32_t w, uint32_t (&h)[4]) {
    const uint32_t x = w >> 8;
    h[0] = sub_half2(mask_or(w, 0x000F000Fu, 0x64006400u), 0x64086408u);  // 1024 + n - 1032
    h[1] = sub_half2(mask_or(w, 0x00F000F0u, 0x54005400u), 0x54805480u);  // 64 + n - 72
    h[2] = sub_half2(mask_or(x, 0x000F000Fu, 0x64006400u), 0x64086408u);
    h[3] = sub_half2(mask_or(x, 0x00F000F0u, 0x54005400u), 0x54805480u);
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// d = A B (no addend).
__device__ __forceinline__ void mma16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
    return d;
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float lg2(float x) {
    float y;
    asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Which tokens the rows [r0, r0 + n) of a sequence see: tiles [first, last) of 16.
struct TileRange {
    int first, last;
};
__device__ __forceinline__ TileRange tile_range(const Kv4AttnParams &p, const Seq &s, int r0, int n) {
    const int rows = s.rows * p.group;
    const int r1 = (r0 + n < rows ? r0 + n : rows) - 1;
    const int lo = s.len - s.rows + small_div(r0, p.group), hi = s.len - s.rows + small_div(r1, p.group);  // positions
    TileRange t{0, hi < 0 ? 0 : hi / 16 + 1};
    if (p.window > 0 && lo - p.window + 1 > 0) t.first = (lo - p.window + 1) / 16;
    if (t.first > t.last) t.first = t.last;
    return t;
}

template <typename E, int D, int NT>
__device__ __forceinline__ void attend_unit(const Kv4AttnParams &p, const Seq &seq, int b, int kvh, int r0, int chunk_first,
                                            int chunk_last, int slot) {
    using Tile = Kv4Tile<D>;
    constexpr int G = Tile::kGroups, R = 8 * NT;
    constexpr int H = NT == 1 && D <= 128 ? 2 : 1;  // tiles whose products are formed together, as registers allow
    extern __shared__ __align__(128) char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
    const int rows = seq.rows * p.group;
    const int base_pos = seq.len - seq.rows;  // position of the sequence's row 0

    constexpr int kStages = Tile::kStages, kStep = 2 * Tile::kBytes;
    char *mine = smem + warp * Tile::kRing;
    const int32_t *table = p.block_table + b * p.table_stride;

    // A step is two tiles; lanes 0 - 15 load the first, 16 - 31 the second.  A
    // lane's pieces of a tile: 16 bytes of codes for every 16 lanes, kept as
    // [group][token][half] (V's tokens in the order 0, 2, .. 14, 1, 3, .., so
    // that both operands' reads are free of bank conflicts), and one 16-byte
    // piece of scales.
    constexpr int kPieces = D / 32;  // of a token
    const int half_warp = lane >> 4, sub = lane & 15;
    const int token = sub / kPieces, part = sub % kPieces;
    const uint32_t base_dst = smem_u32(mine) + half_warp * Tile::kBytes;
    const uint32_t piece_dst = (part / 2) * 512 + (part & 1) * 16;
    const int kv = sub / (Tile::kScales / 16);  // 0: K's scales, 1: V's, above: none
    const int64_t head_cell = static_cast<int64_t>(kvh) * p.page_size;
    const uint8_t *k_src = p.codes[0] + head_cell * (D / 2) + sub * 16;
    const uint8_t *v_src = p.codes[1] + head_cell * (D / 2) + sub * 16;
    const char *s_src = reinterpret_cast<const char *>(p.scales[kv & 1] + head_cell * G) + (sub % (Tile::kScales / 16)) * 16;
    const uint32_t page_codes = static_cast<uint32_t>(p.kv_heads) * p.page_size * (D / 2);
    const uint32_t page_scales = static_cast<uint32_t>(p.kv_heads) * p.page_size * (G * 2);

    // The tile this lane loads next: its number, its page's place in the table,
    // its place in the page, and the page, read one step ahead of the copy.
    constexpr int kAhead = 2 * kAttnWarps;
    const uint32_t page_tiles = static_cast<uint32_t>(p.page_size) / 16;
    const uint32_t step_pages = kAhead / page_tiles, step_rest = kAhead % page_tiles;
    int load_tile = chunk_first + 2 * warp + half_warp;
    uint32_t load_page = static_cast<uint32_t>(load_tile) / page_tiles, load_off = static_cast<uint32_t>(load_tile) % page_tiles;
    int32_t page = -1, pages[kStages];
#pragma unroll
    for (int i = 0; i < kStages; ++i) {  // the first steps' pages, all at once
        uint32_t at = load_page + i * step_pages, off = load_off + i * step_rest;
        while (off >= page_tiles) off -= page_tiles, ++at;
        pages[i] = load_tile + i * kAhead < chunk_last ? __ldg(table + at) : -1;
    }
    uint32_t held = 0;  // bits 0 and 1: the step's two tiles are there; the next steps' above

    // This thread's part of query row 8 j + g: dims 64 gr + 16 c .. + 15.
    uint4 raw[NT][G][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const int r = r0 + 8 * j + g, i = small_div(r, p.group);
        const int64_t row = seq.row0 + i;
        const int head = kvh * p.group + r - i * p.group;
        const char *src = p.q + row * p.q_stride + (static_cast<int64_t>(head) * D + 16 * c) * sizeof(E);
#pragma unroll
        for (int gr = 0; gr < G; ++gr)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                raw[j][gr][h] = make_uint4(0, 0, 0, 0);
                if (r >= rows) continue;
                if (p.q_vector) {
                    raw[j][gr][h] = *reinterpret_cast<const uint4 *>(src + gr * 128 + h * 16);
                } else {
                    const uint16_t *u = reinterpret_cast<const uint16_t *>(src + gr * 128 + h * 16);
                    raw[j][gr][h] = make_uint4(u[0] | u[1] << 16, u[2] | u[3] << 16, u[4] | u[5] << 16, u[6] | u[7] << 16);
                }
            }
    }

    auto issue = [&](int stage) {
        const bool there = page >= 0 && page < p.num_pages;
        const uint32_t both = __ballot_sync(0xFFFFFFFFu, there);
        held = (held >> 2) | ((both & 1u) | (both >> 16 & 1u) * 2u) << (2 * (kStages - 1));
        if (there) {
            const uint32_t at = base_dst + stage * kStep;
            const uint64_t codes = static_cast<uint64_t>(static_cast<uint32_t>(page)) * page_codes + load_off * Tile::kCodes;
            const uint64_t scales = static_cast<uint64_t>(static_cast<uint32_t>(page)) * page_scales + load_off * Tile::kScales;
            const uint8_t *k = k_src + codes, *v = v_src + codes;
            const uint32_t k_dst = at + piece_dst + token * 32;
            const uint32_t v_dst = at + Tile::kCodes + piece_dst;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const int t = token + i * (16 / kPieces);
                cp_async16(k_dst + i * (16 / kPieces) * 32, k + i * 256);
                cp_async16(v_dst + (((t & 1) << 3) | (t >> 1)) * 32, v + i * 256);
            }
            if (kv < 2) cp_async16(at + 2 * Tile::kCodes + sub * 16, s_src + scales);
        }
        cp_commit();
        load_tile += kAhead;
        load_page += step_pages;
        load_off += step_rest;
        if (load_off >= page_tiles) load_off -= page_tiles, ++load_page;
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        page = pages[i];
        issue(i);
    }
    page = pages[kStages - 1];

    // Queries: this thread's B operands and, for its score columns 2c and 2c + 1, the row's factor and limits.
    uint32_t q[NT][G][8];
    float qmul[NT][2];
    int top[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        float x[G][16];
        float amax = 0.0f;
#pragma unroll
        for (int gr = 0; gr < G; ++gr) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                F2 w[4];
                Elem<E>::widen(raw[j][gr][h], w);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x[gr][8 * h + 2 * e] = f2_lo(w[e]);
                    x[gr][8 * h + 2 * e + 1] = f2_hi(w[e]);
                }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[gr][e]));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
        int ex = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
        ex = amax == 0.0f ? 14 : max(ex, -100);
        const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - ex) << 23);  // 2^(14 - ex)
        // back, times the caller's scale and log2(e)
        const float mul = p.scale * 1.4426950408889634f * __uint_as_float(static_cast<uint32_t>(127 - 14 + ex) << 23);
#pragma unroll
        for (int gr = 0; gr < G; ++gr)
#pragma unroll
            for (int w = 0; w < 2; ++w)  // word w of the codes: pairs (i, i + 4)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    q[j][gr][4 * w + i] = pack_half2(x[gr][8 * w + i] * up, x[gr][8 * w + i + 4] * up);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            qmul[j][e] = __shfl_sync(0xFFFFFFFFu, mul, (2 * c + e) * 4);
            top[j][e] = base_pos + small_div(r0 + 8 * j + 2 * c + e, p.group);
        }
    }
    const int lowest = base_pos + small_div(r0, p.group);                                    // the tile's first row
    const int highest = base_pos + small_div(min(r0 + R, rows) - 1, p.group);

    // ref: kOffset - the rows' reference exponents for l and the first group (infinity: none yet; rows that see
    // nothing need none); apart: the other groups' references over it, as powers of two (2^-41 to 2^41)
    float o[NT][D / 16][4] = {};
    float ref[NT][2], l[NT][2];
    F2 apart[NT][G];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            ref[j][e] = r0 + 8 * j + 2 * c + e < rows && top[j][e] >= 0 ? INFINITY : kOffset;
            l[j][e] = 0.0f;
        }
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int gr = 0; gr < G; ++gr) apart[j][gr] = f2(1.0f, 1.0f);
    bool unset = true;  // some row has no reference yet
    int stage = 0;
#pragma unroll 1
    for (int tile = chunk_first + 2 * warp; tile < chunk_last; tile += kAhead) {
        issue(stage == 0 ? kStages - 1 : stage - 1);
        page = load_tile < chunk_last ? __ldg(table + load_page) : -1;
        cp_wait<kStages - 1>();
        __syncwarp();
        const char *step = mine + stage * kStep;
        stage = stage + 1 == kStages ? 0 : stage + 1;
        if ((held & 3u) == 0) continue;
#pragma unroll 1
        for (int part = 0; part < 2 / H; ++part) {
            const char *at = step + part * Tile::kBytes;
            const int t0 = (tile + part) * 16;
            const uint32_t there = held >> part & (H == 2 ? 3u : 1u);
            float s[H][NT][4];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const char *kc = at + h * Tile::kBytes;
                const __half *ks = reinterpret_cast<const __half *>(kc + 2 * Tile::kCodes);
#pragma unroll
                for (int gr = 0; gr < G; ++gr) {
                    const uint2 ka = *reinterpret_cast<const uint2 *>(kc + gr * 512 + g * 32 + c * 8);
                    const uint2 kb = *reinterpret_cast<const uint2 *>(kc + gr * 512 + (g + 8) * 32 + c * 8);
                    const float sa = __half2float(ks[g * G + gr]), sb = __half2float(ks[(g + 8) * G + gr]);
                    uint32_t a[2][4], bq[2][4];
                    codes8(ka.x, a[0]);
                    codes8(ka.y, a[1]);
                    codes8(kb.x, bq[0]);
                    codes8(kb.y, bq[1]);
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        float acc[4];
                        mma16816_first(acc, a[0][0], bq[0][0], a[0][1], bq[0][1], q[j][gr][0], q[j][gr][1]);
#pragma unroll
                        for (int w = 0; w < 2; ++w)
#pragma unroll
                            for (int i = w == 0 ? 2 : 0; i < 4; i += 2)
                                mma16816(acc, a[w][i], bq[w][i], a[w][i + 1], bq[w][i + 1], q[j][gr][4 * w + i],
                                         q[j][gr][4 * w + i + 1]);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            s[h][j][e] = gr == 0 ? acc[e] * (e < 2 ? sa : sb) : fmaf(acc[e], e < 2 ? sa : sb, s[h][j][e]);
                    }
                }
            }
            float vscale[H][G][2];
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const __half *vs = reinterpret_cast<const __half *>(at + h * Tile::kBytes + 2 * Tile::kCodes + Tile::kScales);
#pragma unroll
                for (int gr = 0; gr < G; ++gr) {
                    vscale[h][gr][0] = __half2float(vs[g * G + gr]);
                    vscale[h][gr][1] = __half2float(vs[(g + 8) * G + gr]);
                }
            }
            // weights: packed products with the value scales, and what l grows by
            uint32_t pk[H][NT][G][2];
            float grown[H][NT][2];
            float big = 0.0f, most = 0.0f;
            auto weigh = [&](int h, int j, uint32_t hide) {
                float w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[e] = hide >> e & 1u ? 0.0f : ex2(fmaf(s[h][j][e], qmul[j][e & 1], ref[j][e & 1]));
                grown[h][j][0] = w[0] + w[2];
                grown[h][j][1] = w[1] + w[3];
                most = fmaxf(most, fmaxf(grown[h][j][0], grown[h][j][1]));
#pragma unroll
                for (int gr = 0; gr < G; ++gr) {
                    float x[4];
                    const F2 lo = gr == 0 ? f2(w[0], w[1]) : mul2(f2(w[0], w[1]), apart[j][gr]);
                    const F2 hi = gr == 0 ? f2(w[2], w[3]) : mul2(f2(w[2], w[3]), apart[j][gr]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {  // a hidden token's scale may be anything
                        const F2 of = e < 2 ? lo : hi;
                        x[e] = hide >> e & 1u ? 0.0f : (e & 1 ? f2_hi(of) : f2_lo(of)) * vscale[h][gr][e >> 1];
                        big = fmaxf(big, x[e]);
                    }
                    pk[h][j][gr][0] = pack_half2(x[0], x[1]);
                    pk[h][j][gr][1] = pack_half2(x[2], x[3]);
                }
            };
            const bool masked =
                there != (H == 2 ? 3u : 1u) || t0 + 16 * H - 1 > lowest || (p.window > 0 && t0 <= highest - p.window);
            uint32_t hidden = 0;  // bit 4 (NT h + j) + e
            if (masked) {
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int j = 0; j < NT; ++j) {
                        uint32_t hide = 0;
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int t = t0 + 16 * h + g + (e & 2) * 4, pos = top[j][e & 1];
                            if (t > pos || (p.window > 0 && t <= pos - p.window) || !(there >> h & 1u)) hide |= 1u << e;
                        }
                        weigh(h, j, hide);
                        hidden |= hide << (4 * (NT * h + j));
                    }
            } else {
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int j = 0; j < NT; ++j) weigh(h, j, 0u);
            }
            if (unset || __any_sync(0xFFFFFFFFu, big > kLargest || most > kMostWeight)) {
                float lv[H][G][2];  // log2 of the value scales, kept to what halves can hold
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int gr = 0; gr < G; ++gr)
#pragma unroll
                        for (int t = 0; t < 2; ++t) lv[h][gr][t] = fminf(fmaxf(lg2(vscale[h][gr][t]), -24.0f), 16.0f);
                bool none = false;
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float before = ref[j][e];
#pragma unroll
                        for (int gr = 0; gr < G; ++gr) {
                            float y = -INFINITY;
#pragma unroll
                            for (int h = 0; h < H; ++h)
#pragma unroll
                                for (int t = 0; t < 2; ++t)
                                    if (!(hidden >> (4 * (NT * h + j) + 2 * t + e) & 1u))
                                        y = fmaxf(y, fmaf(s[h][j][2 * t + e], qmul[j][e], lv[h][gr][t]));
                            y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 4));
                            y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 8));
                            y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 16));
                            const float wide = e ? f2_hi(apart[j][gr]) : f2_lo(apart[j][gr]);
                            const int over = (__float_as_int(wide) >> 23) - 127;
                            const float was = before + static_cast<float>(over), r = fminf(was, floorf(kOffset - y));
                            const float f = r == was ? 1.0f : ex2(r - was);
                            if (gr == 0) {
                                ref[j][e] = r;
                                none |= r == INFINITY;
                                l[j][e] *= f;
                            } else {  // 2^0 while there is no reference (a NaN becomes the integer 0)
                                const float now = __int_as_float((static_cast<int>(r - ref[j][e]) + 127) << 23);
                                apart[j][gr] = e ? f2(f2_lo(apart[j][gr]), now) : f2(now, f2_hi(apart[j][gr]));
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                o[j][4 * gr + i][e] *= f;
                                o[j][4 * gr + i][e + 2] *= f;
                            }
                        }
                    }
                unset = __any_sync(0xFFFFFFFFu, none);
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int j = 0; j < NT; ++j) weigh(h, j, hidden >> (4 * (NT * h + j)));
            }
#pragma unroll
            for (int h = 0; h < H; ++h) {
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    l[j][0] += grown[h][j][0];
                    l[j][1] += grown[h][j][1];
#pragma unroll
                    for (int gr = 0; gr < G; ++gr) {
                        pk[h][j][gr][0] = transpose8x8(pk[h][j][gr][0]);
                        pk[h][j][gr][1] = transpose8x8(pk[h][j][gr][1]);
                    }
                }
                const char *vc = at + h * Tile::kBytes + Tile::kCodes;
#pragma unroll
                for (int gr = 0; gr < G; ++gr) {
                    const char *vg = vc + gr * 512 + g * 4;
                    const uint32_t w0 = *reinterpret_cast<const uint32_t *>(vg + c * 32);         // token 2c
                    const uint32_t w1 = *reinterpret_cast<const uint32_t *>(vg + (8 + c) * 32);   // 2c + 1
                    const uint32_t w2 = *reinterpret_cast<const uint32_t *>(vg + (4 + c) * 32);   // 2c + 8
                    const uint32_t w3 = *reinterpret_cast<const uint32_t *>(vg + (12 + c) * 32);  // 2c + 9
#pragma unroll
                    for (int d = 0; d < 2; ++d) {  // dims 8g + 4d .. + 3: pairs of tokens
                        const uint32_t sel = d ? 0x7632u : 0x5410u;
                        uint32_t a[4], bq[4];
                        codes8(__byte_perm(w0, w1, sel), a);
                        codes8(__byte_perm(w2, w3, sel), bq);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int j = 0; j < NT; ++j)
                                mma16816(o[j][gr * 4 + d * 2 + i], a[2 * i], a[2 * i + 1], bq[2 * i], bq[2 * i + 1],
                                         pk[h][j][gr][0], pk[h][j][gr][1]);
                    }
                }
            }
        }
        __syncwarp();
    }
    cp_wait<0>();
    __syncwarp();

    // Join the warps: O, the exponent m - kOffset and l of each row, in shared memory.
    float *joined = reinterpret_cast<float *>(mine);
    float *stat = joined + R * D;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[j][e] += __shfl_xor_sync(0xFFFFFFFFu, l[j][e], 4);
            l[j][e] += __shfl_xor_sync(0xFFFFFFFFu, l[j][e], 8);
            l[j][e] += __shfl_xor_sync(0xFFFFFFFFu, l[j][e], 16);
            const int r = 8 * j + 2 * c + e;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {  // dims 64 gr + 8 g + 2 (i % 4), + 1, back to the first group's reference
                const float wide = e ? f2_hi(apart[j][i / 4]) : f2_lo(apart[j][i / 4]);
                const float f = i < 4 ? 1.0f : __int_as_float((254 << 23) - __float_as_int(wide));
                *reinterpret_cast<float2 *>(joined + r * D + (i / 4) * 64 + g * 8 + (i % 4) * 2) =
                    make_float2(o[j][i][e] * f, o[j][i][e + 2] * f);
            }
            if (g == 0) {  // a row whose scores are all NaN has no reference: its sum carries the NaN
                stat[r] = l[j][e] == 0.0f ? -INFINITY : (ref[j][e] == INFINITY ? 0.0f : -ref[j][e]);
                stat[R + r] = l[j][e];
            }
        }
    __syncthreads();
    constexpr int kStride = Tile::kRing / 4;
    const float *all = reinterpret_cast<const float *>(smem);
    for (int i = threadIdx.x; i < R * (D / 4); i += kAttnWarps * 32) {
        const int r = i / (D / 4), d = (i % (D / 4)) * 4;
        if (r0 + r >= rows) break;
        float top_m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) top_m = fmaxf(top_m, all[w * kStride + R * D + r]);
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float total = 0.0f;
#pragma unroll
        for (int w = 0; w < kAttnWarps; ++w) {
            const float *pw = all + w * kStride;
            const float mw = pw[R * D + r];
            const float f = mw == -INFINITY ? 0.0f : ex2(mw - top_m);
            const float4 v = *reinterpret_cast<const float4 *>(pw + r * D + d);
            sum.x = fmaf(v.x, f, sum.x);
            sum.y = fmaf(v.y, f, sum.y);
            sum.z = fmaf(v.z, f, sum.z);
            sum.w = fmaf(v.w, f, sum.w);
            total = fmaf(pw[R * D + R + r], f, total);
        }
        const int qi = small_div(r0 + r, p.group);
        const int64_t row = seq.row0 + qi;
        const int head = kvh * p.group + r0 + r - qi * p.group;
        if (slot >= 0) {
            const int64_t cell = static_cast<int64_t>(slot) * R + r;
            *reinterpret_cast<float4 *>(p.part_o + cell * D + d) = sum;
            if (d == 0) p.part_s[cell] = make_float2(top_m, total);
        } else {
            store_row<E>(p, row, static_cast<int64_t>(head) * D + d, sum, total);
            if (d == 0 && p.lse) p.lse[row * p.q_heads + head] = finish_lse(top_m, total);
        }
    }
}

// What a (sequence, query tile) pair costs: for each KV head kUnitCost and its
// tiles, at least one for rows that exist (a row without tokens is still
// answered).  All units' together are below 2^31 (the host sees to it).
__device__ __forceinline__ int pair_tiles(const Kv4AttnParams &p, int pair, int tile_rows) {
    const int b = p.row_tiles == 1 ? pair : pair / p.row_tiles, r0 = (pair - b * p.row_tiles) * tile_rows;
    const Seq s = sequence(p, b);
    if (r0 >= s.rows * p.group) return 0;
    const TileRange t = tile_range(p, s, r0, tile_rows);
    return (kUnitCost + max(t.last - t.first, 1)) * p.kv_heads;
}

// This CTA's share of all units' tiles: how many, and the pair it begins in,
// `at` tiles into it.
struct Share {
    int tiles, at, pair;
};
__device__ __forceinline__ Share find_share(const Kv4AttnParams &p, int tile_rows) {
    __shared__ int sums[kAttnWarps];
    __shared__ Share found;
    const int n = p.B * p.row_tiles, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slice = (n + kAttnWarps * 32 - 1) / (kAttnWarps * 32);
    const int i0 = min(static_cast<int>(threadIdx.x) * slice, n), i1 = min(i0 + slice, n);
    int sum = 0;
    for (int i = i0; i < i1; ++i) sum += pair_tiles(p, i, tile_rows);
    int before = sum;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, before, off);
        if (lane >= off) before += v;
    }
    if (lane == 31) sums[warp] = before;
    if (threadIdx.x == 0) found = Share{0, 0, 0};
    __syncthreads();
    int total = 0;
    before -= sum;
#pragma unroll
    for (int w = 0; w < kAttnWarps; ++w) {
        if (w < warp) before += sums[w];
        total += sums[w];
    }
    const int share = max(static_cast<int>((static_cast<unsigned>(total) + gridDim.x - 1) / gridDim.x), kLeastShare);
    const int64_t start = static_cast<int64_t>(share) * blockIdx.x;
    const int first = start < total ? static_cast<int>(start) : total;
    if (blockIdx.x == 0 || (first >= before && first < before + sum)) {
        int at = before;
        for (int i = i0; i < i1; ++i) {
            const int c = slice == 1 ? sum : pair_tiles(p, i, tile_rows);
            if (blockIdx.x == 0) p.starts[i] = at;
            if (first >= at && first < at + c) found = Share{min(share, total - first), first - at, i};
            at += c;
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) p.starts[n] = share;
    __syncthreads();
    return found;
}

// CTAs resident on an SM.  Of 128 dims three: with 8 rows (160 registers) 131072
// tokens take 45 us where four (128 registers) take 50, with 16 rows (168, and 104
// bytes of spills a thread) chunks take 346 us where two without spills took 386.
// Of 64 dims the spills are 48 bytes.
template <int D, int NT>
constexpr int kResident = D == 64 ? (NT == 1 ? 5 : 4) : D == 128 ? 3 : 2;

template <typename E, int D, int NT>
__global__ void __launch_bounds__(kAttnWarps * 32, kResident<D, NT>) kv4_attention_kernel(const __grid_constant__ Kv4AttnParams p) {
    constexpr int R = 8 * NT;
    pdl_wait_and_release();
    if (!p.shared) {
        const int rt = blockIdx.x / p.kv_heads, kvh = blockIdx.x % p.kv_heads, b = blockIdx.y;
        const Seq seq = sequence(p, b);
        if (rt * R >= seq.rows * p.group) return;
        const TileRange range = tile_range(p, seq, rt * R, R);
        attend_unit<E, D, NT>(p, seq, b, kvh, rt * R, range.first, range.last, -1);
        return;
    }
    Share mine = find_share(p, R);
    for (int pair = mine.pair; mine.tiles > 0; ++pair) {
        const int b = pair / p.row_tiles, r0 = pair % p.row_tiles * R;
        if (b >= p.B) return;
        const Seq seq = sequence(p, b);
        if (r0 >= seq.rows * p.group) continue;
        const TileRange range = tile_range(p, seq, r0, R);
        const int count = max(range.last - range.first, 1);
        const int cost = kUnitCost + count;
        for (int kvh = mine.at / cost; kvh < p.kv_heads && mine.tiles > 0; ++kvh) {
            const int past = mine.at - kvh * cost, part = min(cost - past, mine.tiles);  // of the unit's cost
            mine.tiles -= part;
            mine.at += part;
            const int skip = max(past - kUnitCost, 0), take = past + part - kUnitCost - skip;  // of its tiles
            if (take <= 0) break;  // the share ends before the unit's first tile
            // a CTA has at most one unit that it only ends (or passes through) and one that it only begins
            const int slot = take == count ? -1 : static_cast<int>(blockIdx.x) * 2 + (skip == 0 ? 1 : 0);
            attend_unit<E, D, NT>(p, seq, b, kvh, r0, range.first + skip, min(range.first + skip + take, range.last), slot);
            __syncthreads();  // the ring is written again
        }
        mine.at = 0;
    }
}

// Joins the units that the shares cut: one CTA per unit and row, its warps
// taking the partial results in turn.
constexpr int kJoinWarps = 8;
template <typename E, int D>
__global__ void __launch_bounds__(kJoinWarps * 32) kv4_join_kernel(const __grid_constant__ Kv4AttnParams p) {
    pdl_wait_and_release();
    __shared__ float held[kJoinWarps][D + 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int pair = static_cast<int>(blockIdx.x) / p.kv_heads, kvh = static_cast<int>(blockIdx.x) % p.kv_heads;
    const int tile_rows = 8 * p.n_tiles, r0 = pair % p.row_tiles * tile_rows;
    const Seq seq = sequence(p, pair / p.row_tiles);
    const int r = r0 + static_cast<int>(blockIdx.y);
    if (r >= seq.rows * p.group) return;
    const TileRange range = tile_range(p, seq, r0, tile_rows);
    const int count = max(range.last - range.first, 1);
    const int share = p.starts[p.B * p.row_tiles], start = p.starts[pair] + kvh * (kUnitCost + count) + kUnitCost;
    const int cta0 = start / share;
    const int n = (start + count - 1) / share - cta0 + 1;
    if (n == 1) return;
    const int64_t row = seq.row0 + r / p.group;
    const int head = kvh * p.group + r % p.group;
    // partial k: the first CTA's begun unit, then the later ones' ended (or passed) unit
    auto cell_of = [&](int k) -> int64_t { return static_cast<int64_t>((cta0 + k) * 2 + (k == 0 ? 1 : 0)) * tile_rows + blockIdx.y; };
    // each warp joins its share against its own largest exponent, read by lane
    constexpr int N = D / 32;
    float sum[N] = {};
    float total = 0.0f, most = -INFINITY;
    for (int k0 = 0; warp + k0 * kJoinWarps < n; k0 += 32) {
        const int mine = warp + (k0 + lane) * kJoinWarps, here = min(32, (n - warp + kJoinWarps - 1) / kJoinWarps - k0);
        const float2 st = lane < here ? p.part_s[cell_of(mine)] : make_float2(-INFINITY, 0.0f);
        float m = fmaxf(most, st.x);
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
        const float back = most == -INFINITY ? 0.0f : ex2(most - m);
        total *= back;
#pragma unroll
        for (int e = 0; e < N; ++e) sum[e] *= back;
        most = m;
        const float f = st.x == -INFINITY ? 0.0f : ex2(st.x - m), part = st.y * f;
#pragma unroll 4
        for (int i = 0; i < here; ++i) {
            const float *o = p.part_o + cell_of(warp + (k0 + i) * kJoinWarps) * D + lane;
            const float fi = __shfl_sync(0xFFFFFFFFu, f, i);
            total += __shfl_sync(0xFFFFFFFFu, part, i);
#pragma unroll
            for (int e = 0; e < N; ++e) sum[e] = fmaf(o[32 * e], fi, sum[e]);
        }
    }
#pragma unroll
    for (int e = 0; e < N; ++e) held[warp][lane + 32 * e] = sum[e];
    if (lane == 0) {
        held[warp][D] = total;
        held[warp][D + 1] = most;
    }
    __syncthreads();
    if (threadIdx.x < D / 4) {
        float top_m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) top_m = fmaxf(top_m, held[w][D + 1]);
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        float all = 0.0f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
            const float *h = held[w] + threadIdx.x * 4;
            const float f = held[w][D + 1] == -INFINITY ? 0.0f : ex2(held[w][D + 1] - top_m);
            v.x = fmaf(h[0], f, v.x);
            v.y = fmaf(h[1], f, v.y);
            v.z = fmaf(h[2], f, v.z);
            v.w = fmaf(h[3], f, v.w);
            all = fmaf(held[w][D], f, all);
        }
        store_row<E>(p, row, static_cast<int64_t>(head) * D + threadIdx.x * 4, v, all);
        if (threadIdx.x == 0 && p.lse) p.lse[row * p.q_heads + head] = finish_lse(top_m, all);
    }
}

using namespace checks;

// How a call is cut up, from sizes the host knows.
constexpr int64_t kMaxRows = 1 << 20;  // max_q_len * q_heads
// Positions lie between -kMaxRows and this; a tile past one and the difference
// of a position and a window still fit 32 bits.
constexpr int64_t kMaxTokens = ((int64_t)1 << 31) - ((int64_t)1 << 21);

struct Plan {
    int32_t n_tiles, row_tiles;
    int32_t ctas;  // shares (0: one CTA per unit)
    int64_t pairs;
};
constexpr int kSms = 148;

// Query tiles of a call and the CTAs that fit the SMs at once.
Plan tiled(int32_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t max_q_len, int64_t *slots) {
    Plan pl{};
    const int64_t rows = (int64_t)max_q_len * (q_heads / kv_heads);
    // 16 rows where there are more than 8 (4 sequences' chunks of 509 rows, 128 dims: 340 us, 470 us with 8 rows;
    // two tokens of 8 heads each: 37 against 40 us); of 256 dims they do not fit the registers
    pl.n_tiles = rows <= 8 || head_dim == 256 ? 1 : 2;
    pl.row_tiles = (int32_t)((rows + 8 * pl.n_tiles - 1) / (8 * pl.n_tiles));
    pl.pairs = (int64_t)B * pl.row_tiles;
    const int64_t resident = pl.n_tiles == 1 ? (head_dim == 64 ? kResident<64, 1> : head_dim == 128 ? kResident<128, 1> : kResident<256, 1>)
                                             : (head_dim == 64 ? kResident<64, 2> : head_dim == 128 ? kResident<128, 2> : 2);
    *slots = kSms * resident;
    return pl;
}

int64_t share_ctas(int64_t units, int64_t tiles, int64_t slots) {
    const int64_t most = (units * (tiles + kUnitCost) + kLeastShare - 1) / kLeastShare;
    return most < slots ? most : slots;
}

// Units of at most so many tiles are never cut into shares (see plan()).
int64_t whole_tiles(int32_t head_dim) { return head_dim == 64 ? 128 : 64; }

Plan plan(int32_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t max_q_len, int32_t max_seq_len,
          int32_t window) {
    int64_t slots = 0;
    Plan pl = tiled(B, q_heads, kv_heads, head_dim, max_q_len, &slots);
    const int64_t units = pl.pairs * kv_heads, tiles = ((int64_t)max_seq_len + 15) / 16;
    // what a unit reads at most: with a window no more than its rows see (64 sequences to 32768 tokens, a window of 512,
    // whole units 21 us, shares 28; 4 with a window of 2048 18.6 and 15.8)
    const int64_t seen = window > 0 ? ((int64_t)window + max_q_len - 1 + 15) / 16 : tiles, longest = seen < tiles ? seen : tiles;
    // One CTA a unit where units are many, or short enough that shares and a join
    // cost more than their balance gains.  Whole units against shares in us, 32
    // heads over 8, B sequences to L tokens:
    //   one token each, 128 dims: 128 to 4096 104 / 107, 128 to 2048 60 / 69, 64 to 4096 65 / 60.5,
    //     64 to 2048 38.5 / 40.9, 64 to 1024 24.7 / 30.5, 16 to 8192 59 / 36, 8 to 2048 17.6 / 15.3,
    //     4 to 2048 17.7 / 12.4, 4 to 1024 10.5 / 12.5;
    //   64 dims, where a tile is half the work: 128 to 4096 67 / 73, 64 to 4096 48 / 43, 64 to 2048 26.5 / 30.7,
    //     16 to 4096 22.8 / 19.4, 16 to 2048 13.1 / 18.1, 8 to 2048 12.8 / 12.9, 4 to 4096 22.4 / 13.0, 4 to 2048 12.8 / 12.0;
    //   256 dims: 128 to 2048 119 / 127, 64 to 2048 73 / 72, 64 to 1024 44 / 50, 16 to 2048 31.6 / 28.2, 16 to 1024 18.9 / 22.9,
    //     4 to 2048 30.4 / 17.7, 4 to 1024 18.3 / 17.4, 4 to 512 11.5 / 17.4;
    //   tiles of 16 rows, whose shares cost more to join, 128 dims (444 CTAs at once): 4 chunks of 64 (512 units) to 4096
    //     75 / 104, to 16384 274 / 282, one of 200 (400 units) to 4096 80 / 105, to 32768 573 / 575, 16 of 9 (384) to 4096
    //     75 / 79, to 8192 140 / 124, 16 of 8 (256) to 4096 70 / 60; 64 dims (592): 64 of 4 (512) to 4096 58 / 70, to 8192
    //     108 / 101, 16 of 9 (384) to 4096 55 / 53, 16 of 8 (256) to 2048 22 / 33.
    const int64_t whole = whole_tiles(head_dim);
    const bool many = pl.n_tiles == 2 ? 4 * units >= 3 * slots && longest <= 256 : units >= slots && longest <= 2 * whole;
    if (units >= 2 * slots || longest <= whole || many || units * (tiles + kUnitCost) >= ((int64_t)1 << 31)) return pl;
    pl.ctas = (int32_t)share_ctas(units, tiles, slots);
    return pl;
}

// Partial outputs and sums of every share's two ends, the pairs' first tiles.
int64_t share_bytes(int64_t ctas, int64_t pairs, int32_t n_tiles, int32_t head_dim) {
    return ctas == 0 ? 0 : ctas * 2 * 8 * n_tiles * (head_dim + 2) * 4 + (pairs + 1) * 4;
}

template <typename E, int D, int NT>
qkn_status launch_attention(const Kv4AttnParams &p, dim3 grid, dim3 join_grid, void *stream) {
    constexpr size_t smem = (size_t)kAttnWarps * Kv4Tile<D>::kRing;
    static_assert((size_t)8 * NT * (D + 2) * 4 <= Kv4Tile<D>::kRing, "a warp's partial result must fit its ring");
    const void *fn = (const void *)kv4_attention_kernel<E, D, NT>;
    if (smem > 48 * 1024) {  // once for each device; setting it again does no harm
        static std::atomic<uint64_t> set{0};
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        const uint64_t bit = uint64_t(1) << (dev & 63);
        if (e == cudaSuccess && (dev > 63 || !(set.load(std::memory_order_relaxed) & bit))) {
            e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
            if (e == cudaSuccess) set.fetch_or(bit, std::memory_order_relaxed);
        }
        if (e != cudaSuccess) return launched(e);
    }
    qkn_status st = launched(launch_pdl(fn, grid, kAttnWarps * 32, smem, stream, p));
    if (st != QKN_OK || !p.shared) return st;
    return launched(launch_pdl((const void *)kv4_join_kernel<E, D>, join_grid, kJoinWarps * 32, 0, stream, p));
}
template <typename E>
qkn_status launch_attention(const Kv4AttnParams &p, int d, dim3 grid, dim3 join_grid, void *stream) {
    if (p.n_tiles == 1)
        return d == 64    ? launch_attention<E, 64, 1>(p, grid, join_grid, stream)
               : d == 128 ? launch_attention<E, 128, 1>(p, grid, join_grid, stream)
                          : launch_attention<E, 256, 1>(p, grid, join_grid, stream);
    return d == 64 ? launch_attention<E, 64, 2>(p, grid, join_grid, stream)
                   : launch_attention<E, 128, 2>(p, grid, join_grid, stream);
}

}  // namespace
}  // namespace qkn

using namespace qkn;
using namespace qkn::checks;

extern "C" {

int64_t qknorm_kv4_attention_workspace_bytes(int64_t T, int32_t B, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                             int32_t max_q_len, int32_t max_seq_len) {
    if (T < 0 || B < 0 || q_heads < 1 || kv_heads < 1 || head_dim < 1 || max_q_len < 1 || max_seq_len < 0 ||
        q_heads % kv_heads != 0 || head_dim > kRopeMaxHeadDim || T >= ((int64_t)1 << 31) / q_heads)
        return -1;
    if ((int64_t)max_q_len * q_heads > kMaxRows) return -1;
    // enough for every call of at most these sizes: calls that are cut into shares have fewer than 2 * slots units,
    // of 8 rows more CTAs fit than of 16 but their tiles hold half as many
    int64_t slots = 0;
    const Plan pl = tiled(B, q_heads, kv_heads, head_dim, max_q_len, &slots);
    const int64_t tiles = ((int64_t)max_seq_len + 15) / 16;
    if (tiles <= whole_tiles(head_dim)) return 0;
    const int64_t units = pl.pairs * kv_heads < 2 * slots ? pl.pairs * kv_heads : 2 * slots - 1;
    return share_bytes(share_ctas(units, tiles, slots), units / kv_heads, pl.n_tiles, head_dim);
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
    if ((int64_t)max_q_len * q_heads > kMaxRows)
        return fail(QKN_ERR_UNSUPPORTED, "max_q_len = %d too long: call in chunks of rows", max_q_len);
    const int64_t held = (int64_t)max_pages * page_size, longest = held < max_seq_len ? held : max_seq_len;
    if (longest > kMaxTokens)
        return fail(QKN_ERR_UNSUPPORTED, "sequences of up to %lld tokens, at most %lld", (long long)longest, (long long)kMaxTokens);
    const Plan pl = plan(B, q_heads, kv_heads, head_dim, max_q_len, max_seq_len, window);
    const int64_t need = share_bytes(pl.ctas, pl.pairs, pl.n_tiles, head_dim);
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
    p.window = window < longest ? window : 0;  // no token is further back
    p.scale = scale;
    p.q_vector = aligned16(q) && p.q_stride % 16 == 0;
    p.out_vector = ((uintptr_t)out & 7u) == 0 && p.out_stride % 8 == 0;
    p.n_tiles = pl.n_tiles;
    p.row_tiles = pl.row_tiles;
    p.shared = pl.ctas > 0;
    if (p.shared) {
        const int64_t cells = (int64_t)pl.ctas * 2 * 8 * pl.n_tiles;
        p.part_o = static_cast<float *>(workspace);
        p.part_s = reinterpret_cast<float2 *>(p.part_o + cells * head_dim);
        p.starts = reinterpret_cast<int32_t *>(p.part_s + cells);
    }
    const int64_t tile_rows = 8 * pl.n_tiles, rows = (int64_t)max_q_len * p.group;
    const dim3 grid = p.shared ? dim3((unsigned)pl.ctas) : dim3((unsigned)(pl.row_tiles * kv_heads), (unsigned)B);
    const dim3 join_grid((unsigned)(pl.pairs * kv_heads), (unsigned)(rows < tile_rows ? rows : tile_rows));
    return dtype == QKN_BF16 ? launch_attention<__nv_bfloat16>(p, head_dim, grid, join_grid, stream)
                             : launch_attention<__half>(p, head_dim, grid, join_grid, stream);
}

}  // extern "C"
