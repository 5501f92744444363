// attnres_cache_api.cu -- C entry points of the compressed source cache:
// argument validation and workspace sizing (include/attnres.h).
#include <cmath>
#include <cstring>

#include "attnres.h"
#include "cached.cuh"
#include "kernels.cuh"

namespace attnres {
namespace {

int sm_count() {  // of the current device, queried once each; 0 on error
    static int cache[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 0;
    if (dev < 64 && cache[dev] > 0) return cache[dev];
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    if (dev < 64) cache[dev] = n;
    return n;
}

bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1u)) == 0; }

// Bytes from the first to behind the last of N rows, ld bytes apart.
size_t span(int64_t N, int64_t ld, size_t row) { return N <= 0 ? 0 : static_cast<size_t>(N - 1) * ld + row; }

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
}

attnres_status check_format(int32_t D, int32_t bits) {
    if (D < 8 || D > ATTNRES_MAX_D || (bits != 4 && bits != 8)) return ATTNRES_ERR_INVALID_ARG;
    return D % 8 ? ATTNRES_ERR_ALIGNMENT : ATTNRES_OK;
}

attnres_status check_records(const void* rows, int64_t row_ld, int64_t N, int32_t D, int32_t bits) {
    if (N < 0 || row_ld < static_cast<int64_t>(cache_row_bytes(D, bits))) return ATTNRES_ERR_INVALID_ARG;
    if (row_ld % 16) return ATTNRES_ERR_ALIGNMENT;
    if (N == 0) return ATTNRES_OK;
    if (!rows) return ATTNRES_ERR_INVALID_ARG;
    return aligned(rows, 16) ? ATTNRES_OK : ATTNRES_ERR_ALIGNMENT;
}

// bf16 rows, ld elements apart
attnres_status check_rows(const void* p, int64_t ld, int64_t N, int32_t D) {
    if (ld < D) return ATTNRES_ERR_INVALID_ARG;
    if (ld % 8) return ATTNRES_ERR_ALIGNMENT;
    if (N == 0) return ATTNRES_OK;
    if (!p) return ATTNRES_ERR_INVALID_ARG;
    return aligned(p, 16) ? ATTNRES_OK : ATTNRES_ERR_ALIGNMENT;
}

attnres_status check_cached(const attnres_cached_params* p) {
    if (!p) return ATTNRES_ERR_INVALID_ARG;
    attnres_status st = check_format(p->D, p->bits);
    if (st != ATTNRES_OK) return st;
    if (p->S < 1 || p->S + (p->live ? 1 : 0) > ATTNRES_MAX_S) return ATTNRES_ERR_INVALID_ARG;
    if (p->R < 1 || p->R > p->D || p->key_offset < 0 || p->key_offset > p->D - p->R) return ATTNRES_ERR_INVALID_ARG;
    if (p->out_norm != 0 && p->out_norm != 1) return ATTNRES_ERR_INVALID_ARG;
    if (!std::isfinite(p->eps) || p->eps < 0.0f || !std::isfinite(p->scale)) return ATTNRES_ERR_INVALID_ARG;
    for (int s = 0; s < p->S; ++s) {
        st = check_records(p->rows[s], p->row_ld, p->N, p->D, p->bits);
        if (st != ATTNRES_OK) return st;
    }
    return p->live ? check_rows(p->live, p->live_ld, p->N, p->D) : ATTNRES_OK;
}

void fill(const attnres_cached_params* p, const void* q, const void* w_o, CachedArgs* a) {
    std::memset(a, 0, sizeof *a);
    for (int s = 0; s < p->S; ++s) a->rows[s] = static_cast<const unsigned char*>(p->rows[s]);
    a->N = p->N;
    a->row_ld = p->row_ld;
    a->live_ld = p->live_ld;
    a->S = p->S;
    a->D = p->D;
    a->R = p->R;
    a->ko = p->key_offset;
    a->codes = cache_code_bytes(p->D, p->bits);
    a->stat = cache_stat_offset(p->D, p->bits);
    a->tag = cache_tag(p->R, p->key_offset, p->bits);
    a->eps = p->eps;
    a->scale = p->scale;
    a->live = static_cast<const uint16_t*>(p->live);
    a->q = static_cast<const uint16_t*>(q);
    a->w_o = p->out_norm ? static_cast<const uint16_t*>(w_o) : nullptr;
}

}  // namespace
}  // namespace attnres

using namespace attnres;

extern "C" {

size_t attnres_cache_row_bytes(int32_t D, int32_t bits) {
    return check_format(D, bits) == ATTNRES_OK ? cache_row_bytes(D, bits) : 0;
}

attnres_status attnres_cache_write(const void* src, int64_t src_ld, int64_t N, int32_t D, int32_t bits, int32_t R,
                                   int32_t key_offset, void* rows, int64_t row_ld, void* stream) {
    attnres_status st = check_format(D, bits);
    if (st != ATTNRES_OK) return st;
    if (R < 1 || R > D || key_offset < 0 || key_offset > D - R) return ATTNRES_ERR_INVALID_ARG;
    if ((st = check_records(rows, row_ld, N, D, bits)) != ATTNRES_OK) return st;
    if ((st = check_rows(src, src_ld, N, D)) != ATTNRES_OK) return st;
    if (N == 0) return ATTNRES_OK;
    if (overlap(src, span(N, src_ld * 2, static_cast<size_t>(D) * 2), rows, span(N, row_ld, cache_row_bytes(D, bits))))
        return ATTNRES_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (!sms) return ATTNRES_ERR_CUDA;
    CacheRowsArgs a{};
    a.x = static_cast<const uint16_t*>(src);
    a.rows = static_cast<unsigned char*>(rows);
    a.N = N;
    a.x_ld = src_ld;
    a.row_ld = row_ld;
    a.D = D;
    a.R = R;
    a.ko = key_offset;
    a.codes = cache_code_bytes(D, bits);
    a.stat = cache_stat_offset(D, bits);
    a.tag = cache_tag(R, key_offset, bits);
    return launch_cache_write(a, bits, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTNRES_OK
                                                                                              : ATTNRES_ERR_CUDA;
}

attnres_status attnres_cache_load(const void* rows, int64_t row_ld, int64_t N, int32_t D, int32_t bits, void* dst,
                                  int64_t dst_ld, void* stream) {
    attnres_status st = check_format(D, bits);
    if (st != ATTNRES_OK) return st;
    if ((st = check_records(rows, row_ld, N, D, bits)) != ATTNRES_OK) return st;
    if ((st = check_rows(dst, dst_ld, N, D)) != ATTNRES_OK) return st;
    if (N == 0) return ATTNRES_OK;
    if (overlap(dst, span(N, dst_ld * 2, static_cast<size_t>(D) * 2), rows, span(N, row_ld, cache_row_bytes(D, bits))))
        return ATTNRES_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (!sms) return ATTNRES_ERR_CUDA;
    CacheRowsArgs a{};
    a.out = static_cast<uint16_t*>(dst);
    a.rows = static_cast<unsigned char*>(const_cast<void*>(rows));
    a.N = N;
    a.x_ld = dst_ld;
    a.row_ld = row_ld;
    a.D = D;
    a.codes = cache_code_bytes(D, bits);
    a.stat = cache_stat_offset(D, bits);
    a.tag = cache_tag(0, 0, bits);
    return launch_cache_load(a, bits, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTNRES_OK
                                                                                             : ATTNRES_ERR_CUDA;
}

attnres_status attnres_cached_fwd(const attnres_cached_params* p, const void* q, const void* w_o, void* y, float* alpha,
                                  float* rstd, float* logit, float* o_rstd, void* stream) {
    const attnres_status st = check_cached(p);
    if (st != ATTNRES_OK) return st;
    if (p->N == 0) return ATTNRES_OK;
    if (!q || !y || !alpha || !rstd || !logit) return ATTNRES_ERR_INVALID_ARG;
    if (p->out_norm && (!w_o || !o_rstd)) return ATTNRES_ERR_INVALID_ARG;
    if (!aligned(y, 16) || !aligned(q, 2) || !aligned(alpha, 4) || !aligned(rstd, 4) || !aligned(logit, 4))
        return ATTNRES_ERR_ALIGNMENT;
    if (p->out_norm && (!aligned(w_o, 16) || !aligned(o_rstd, 4))) return ATTNRES_ERR_ALIGNMENT;
    // y is written while other tokens are still read
    const size_t row = static_cast<size_t>(p->D) * 2, n_y = static_cast<size_t>(p->N) * row;
    for (int s = 0; s < p->S; ++s)
        if (overlap(y, n_y, p->rows[s], span(p->N, p->row_ld, cache_row_bytes(p->D, p->bits)))) return ATTNRES_ERR_INVALID_ARG;
    if (p->live && overlap(y, n_y, p->live, span(p->N, p->live_ld * 2, row))) return ATTNRES_ERR_INVALID_ARG;
    const int sms = sm_count();
    if (!sms) return ATTNRES_ERR_CUDA;
    CachedArgs a;
    fill(p, q, w_o, &a);
    a.alpha = alpha;
    a.rstd = rstd;
    a.logit = logit;
    a.o_rstd = o_rstd;
    a.y = static_cast<uint16_t*>(y);
    return launch_cached_fwd(a, p->bits, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ATTNRES_OK
                                                                                                : ATTNRES_ERR_CUDA;
}

size_t attnres_cached_bwd_workspace_bytes(const attnres_cached_params* p) {
    if (check_cached(p) != ATTNRES_OK || p->N == 0) return 0;
    const int sms = sm_count();
    if (!sms) return 0;
    return static_cast<size_t>(cached_bwd_grid(p->S, p->live != nullptr, p->N, p->D, p->bits, sms)) * (p->R + (p->out_norm ? p->D : 0)) * sizeof(float);
}

attnres_status attnres_cached_bwd(const attnres_cached_params* p, const void* q, const void* w_o, const void* dy,
                                  const float* alpha, const float* rstd, const float* logit, const float* o_rstd,
                                  void* const* dsrc, int64_t dsrc_ld, void* dlive, int64_t dlive_ld, void* dq,
                                  float* dq_f32, void* dw_o, float* dw_o_f32, void* workspace, size_t workspace_bytes,
                                  void* stream) {
    attnres_status st = check_cached(p);
    if (st != ATTNRES_OK) return st;
    if (!dq || (p->out_norm && !dw_o)) return ATTNRES_ERR_INVALID_ARG;
    if (dlive && !p->live) return ATTNRES_ERR_INVALID_ARG;
    if (!aligned(dq, 2) || !aligned(dq_f32, 4) || (p->out_norm && (!aligned(dw_o, 2) || !aligned(dw_o_f32, 4))))
        return ATTNRES_ERR_ALIGNMENT;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p->N == 0) {  // empty sums are zero; nothing else is touched
        const size_t R = p->R, D = p->D;
        if (cudaMemsetAsync(dq, 0, R * 2, s) != cudaSuccess ||
            (dq_f32 && cudaMemsetAsync(dq_f32, 0, R * 4, s) != cudaSuccess) ||
            (p->out_norm && cudaMemsetAsync(dw_o, 0, D * 2, s) != cudaSuccess) ||
            (p->out_norm && dw_o_f32 && cudaMemsetAsync(dw_o_f32, 0, D * 4, s) != cudaSuccess))
            return ATTNRES_ERR_CUDA;
        return ATTNRES_OK;
    }
    if (!q || !dy || !alpha || !rstd || !logit || (p->out_norm && (!w_o || !o_rstd))) return ATTNRES_ERR_INVALID_ARG;
    if (!aligned(dy, 16) || !aligned(q, 2) || !aligned(alpha, 4) || !aligned(rstd, 4) || !aligned(logit, 4))
        return ATTNRES_ERR_ALIGNMENT;
    if (p->out_norm && (!aligned(w_o, 16) || !aligned(o_rstd, 4))) return ATTNRES_ERR_ALIGNMENT;
    // the gradients: rows of their own, apart from each other and from what the kernel reads
    const size_t row = static_cast<size_t>(p->D) * 2;
    const size_t n_rec = span(p->N, p->row_ld, cache_row_bytes(p->D, p->bits));
    const size_t n_d = span(p->N, dsrc_ld * 2, row), n_dl = span(p->N, dlive_ld * 2, row);
    const size_t n_live = p->live ? span(p->N, p->live_ld * 2, row) : 0;
    const int outs = (dsrc ? p->S : 0) + (dlive ? 1 : 0);
    if (dlive && (st = check_rows(dlive, dlive_ld, p->N, p->D)) != ATTNRES_OK) return st;
    for (int i = 0; dsrc && i < p->S; ++i)
        if ((st = check_rows(dsrc[i], dsrc_ld, p->N, p->D)) != ATTNRES_OK) return st;
    for (int i = 0; i < outs; ++i) {
        const bool l = dlive && i == outs - 1;
        const void* o = l ? dlive : dsrc[i];
        const size_t n = l ? n_dl : n_d;
        for (int j = 0; j < i; ++j)
            if (overlap(o, n, dsrc[j], n_d)) return ATTNRES_ERR_INVALID_ARG;
        for (int j = 0; j < p->S; ++j)
            if (overlap(o, n, p->rows[j], n_rec)) return ATTNRES_ERR_INVALID_ARG;
        if (overlap(o, n, p->live, n_live) || overlap(o, n, dy, static_cast<size_t>(p->N) * row)) return ATTNRES_ERR_INVALID_ARG;
    }
    const int sms = sm_count();
    if (!sms) return ATTNRES_ERR_CUDA;
    const int grid = cached_bwd_grid(p->S, p->live != nullptr, p->N, p->D, p->bits, sms);
    const int W = p->R + (p->out_norm ? p->D : 0);
    if (!workspace || workspace_bytes < static_cast<size_t>(grid) * W * sizeof(float)) return ATTNRES_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return ATTNRES_ERR_ALIGNMENT;
    CachedBwdArgs b;
    std::memset(&b, 0, sizeof b);
    fill(p, q, w_o, &b.c);
    b.c.alpha = const_cast<float*>(alpha);
    b.c.rstd = const_cast<float*>(rstd);
    b.c.logit = const_cast<float*>(logit);
    b.c.o_rstd = const_cast<float*>(o_rstd);
    b.want_dsrc = dsrc != nullptr;
    for (int i = 0; dsrc && i < p->S; ++i) b.dsrc[i] = static_cast<uint16_t*>(dsrc[i]);
    b.dsrc_ld = dsrc_ld;
    b.wide_src = p->D % 16 == 0 && dsrc_ld % 16 == 0;
    for (int i = 0; dsrc && i < p->S; ++i) b.wide_src = b.wide_src && aligned(dsrc[i], 32);
    b.wide_live = p->D % 16 == 0 && dlive_ld % 16 == 0 && aligned(dlive, 32);
    b.dlive = static_cast<uint16_t*>(dlive);
    b.dlive_ld = dlive_ld;
    b.dy = static_cast<const uint16_t*>(dy);
    b.part = static_cast<float*>(workspace);
    if (launch_cached_bwd(b, p->bits, grid, sms, s) != cudaSuccess) return ATTNRES_ERR_CUDA;
    return launch_finalize(b.part, grid, p->R, W, static_cast<uint16_t*>(dq), dq_f32, static_cast<uint16_t*>(dw_o),
                           dw_o_f32, s) == cudaSuccess
               ? ATTNRES_OK
               : ATTNRES_ERR_CUDA;
}

}  // extern "C"
