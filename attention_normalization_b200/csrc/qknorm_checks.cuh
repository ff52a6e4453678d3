// Host-side argument checks shared by the entry points of qknorm_rope.cu and
// qknorm_kv4.cu.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "qknorm.h"
#include "qknorm_plan.h"
#include "qknorm_rope.cuh"

namespace qkn {

void set_last_error(const char *msg);  // qknorm_api.cu

namespace checks {

inline qkn_status fail(qkn_status st, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    set_last_error(buf);
    return st;
}

inline qkn_status ok() {
    set_last_error("");
    return QKN_OK;
}

inline int elem_bytes(int dt) { return dt == QKN_F32 ? 4 : (dt == QKN_FP8_E4M3 ? 1 : 2); }
inline int gamma_bytes(int dt) { return dt == QKN_F32 ? 4 : 2; }
inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// `rows` runs of `width` bytes, `stride` bytes apart.
struct Span {
    const void *base;
    int64_t width, stride, rows;
    const char *name;
};
inline Span flat(const void *p, int64_t bytes, const char *name) { return Span{p, bytes, bytes, 1, name}; }

// First written span that meets another span: a message and INVALID_ARG.  A
// written span may be exactly one of `same` (in place); null bases are absent.
inline qkn_status check_written(const Span *w, int nw, const Span *r, int nr, const int *in_place, int n_in_place) {
    auto meets = [](const Span &a, const Span &b) {
        return a.base && b.base &&
               qknorm_regions_overlap(reinterpret_cast<uint64_t>(a.base), a.width, a.stride, a.rows,
                                      reinterpret_cast<uint64_t>(b.base), b.width, b.stride, b.rows);
    };
    for (int i = 0; i < nw; ++i) {
        for (int j = i + 1; j < nw; ++j)
            if (meets(w[i], w[j])) return fail(QKN_ERR_INVALID_ARG, "%s and %s overlap", w[i].name, w[j].name);
        for (int j = 0; j < nr; ++j) {
            bool same = false;  // in_place: pairs (written index, read index) that may coincide
            for (int k = 0; k + 1 < n_in_place; k += 2)
                same |= in_place[k] == i && in_place[k + 1] == j && w[i].base == r[j].base && w[i].stride == r[j].stride &&
                        w[i].width == r[j].width;
            if (!same && meets(w[i], r[j])) return fail(QKN_ERR_INVALID_ARG, "%s overlaps %s", w[i].name, r[j].name);
        }
    }
    return QKN_OK;
}

// Rows of T must stay addressable.
inline bool extent_ok(int64_t rows, int64_t stride, int64_t width, int64_t esz) {
    if (rows <= 0) return true;
    const __int128 bytes = ((__int128)(rows - 1) * stride + width) * esz;
    return stride >= 0 && bytes < ((__int128)1 << 62);
}

// Sizes and pointers of a 4-bit cache; the bytes of its code and scale tensors.
inline qkn_status check_kv4(int64_t num_pages, int32_t page_size, int32_t kv_heads, int32_t head_dim, const void *k_codes,
                            const void *k_scales, const void *v_codes, const void *v_scales, bool used, int64_t *codes,
                            int64_t *scales) {
    if (head_dim != 64 && head_dim != 128 && head_dim != 256)
        return fail(head_dim < 1 ? QKN_ERR_INVALID_ARG : QKN_ERR_UNSUPPORTED,
                    "the 4-bit cache takes head_dim 64, 128 or 256, got %d", head_dim);
    if (page_size < 1 || page_size > (1 << 20) || num_pages < 0 || kv_heads < 1 || kv_heads > (1 << 20))
        return fail(QKN_ERR_INVALID_ARG, "num_pages = %lld, page_size = %d, kv_heads = %d", (long long)num_pages,
                    page_size, kv_heads);
    if (page_size % kKv4PageMultiple != 0)
        return fail(QKN_ERR_UNSUPPORTED, "the 4-bit cache's page_size must be a multiple of %d, got %d", kKv4PageMultiple,
                    page_size);
    if ((int64_t)kv_heads * page_size * (head_dim / 2) >= ((int64_t)1 << 31))
        return fail(QKN_ERR_UNSUPPORTED, "a page of the 4-bit cache must stay below 2 GiB");
    const __int128 cells = (__int128)num_pages * kv_heads * page_size;
    if (cells * head_dim >= ((__int128)1 << 60)) return fail(QKN_ERR_INVALID_ARG, "cache extent overflows");
    *codes = (int64_t)cells * (head_dim / 2);
    *scales = (int64_t)cells * (head_dim / kKv4Group) * 2;
    if (used && (!k_codes || !k_scales || !v_codes || !v_scales)) return fail(QKN_ERR_INVALID_ARG, "null cache pointer");
    if (!aligned16(k_codes) || !aligned16(k_scales) || !aligned16(v_codes) || !aligned16(v_scales))
        return fail(QKN_ERR_INVALID_ARG, "the 4-bit cache's tensors must be 16-byte aligned");
    return QKN_OK;
}

// One launch with programmatic stream serialization (the kernel waits for the
// one before it itself).
template <typename P>
inline cudaError_t launch_pdl(const void *fn, dim3 grid, dim3 block, size_t smem, void *stream, const P &p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void *args[] = {const_cast<P *>(&p)};
    return cudaLaunchKernelExC(&cfg, fn, args);
}

// SMs of the current device (148 on a B200), for grid sizes.
inline qkn_status device_sms(int *sms) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess || *sms < 1) return fail(QKN_ERR_CUDA, "device query: %s", cudaGetErrorString(e));
    return QKN_OK;
}

inline qkn_status launched(cudaError_t e) {
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return fail(QKN_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
    return ok();
}

}  // namespace checks
}  // namespace qkn
