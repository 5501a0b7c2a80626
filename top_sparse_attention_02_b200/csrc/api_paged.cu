// api_paged.cu -- the C ABI of the paged-cache entry points (declared in
// include/tsa.h): argument checks, workspace layout and stream-ordered launches.
// No allocation, no synchronisation, no exceptions.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "common.cuh"
#include "paged.h"
#include "tsa.h"

namespace {

tsa_status fail(tsa_status st, const char* fmt, ...) {
    char msg[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    tsa::set_error_message(msg);
    return st;
}

tsa_status cuda_fail(cudaError_t e, const char* where) {
    return fail(TSA_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
size_t a256(size_t x) { return (x + 255) & ~(size_t)255; }
constexpr size_t kFlagBytes = 256;
constexpr long long kMaxStride = 1LL << 38;  // elements: what a tensor map's stride can say

#define TSA_TRY(x)                     \
    do {                               \
        tsa_status _st = (x);          \
        if (_st != TSA_OK) return _st; \
    } while (0)

tsa_status check_dtype(int dtype, int d) {
    if (dtype != TSA_BF16 && dtype != TSA_FP16) return fail(TSA_ERR_UNSUPPORTED, "dtype must be TSA_BF16 or TSA_FP16 (got %d)", dtype);
    if (d != tsa::kDHead) return fail(TSA_ERR_UNSUPPORTED, "head dimension must be 128 (got %d)", d);
    return TSA_OK;
}

// the cache's sizes and strides (its pointers are checked by the calls that use them)
tsa_status check_cache(const tsa_paged_cache& c, tsa::Pages* out) {
    TSA_TRY(check_dtype(c.dtype, c.d));
    if (c.B < 0 || c.Hkv <= 0 || c.num_pages < 1 || c.max_pages < 1)
        return fail(TSA_ERR_INVALID_ARG, "cache: need B >= 0, Hkv > 0, num_pages > 0, max_pages > 0 (got B=%d Hkv=%d num_pages=%d max_pages=%d)",
                    c.B, c.Hkv, c.num_pages, c.max_pages);
    if (c.page_size < tsa::kPageRows || c.page_size % tsa::kPageRows != 0)
        return fail(TSA_ERR_UNSUPPORTED, "cache: page_size must be a multiple of %d (got %d)", tsa::kPageRows, c.page_size);
    if ((long long)c.B * c.Hkv > 1 << 22) return fail(TSA_ERR_UNSUPPORTED, "cache: B*Hkv=%lld above %d", (long long)c.B * c.Hkv, 1 << 22);
    // rows must not overlap: by ascending stride, each stride clears what the smaller ones span
    struct Dim {
        long long stride, n;
    } dim[3] = {{c.row_stride, c.page_size}, {c.head_stride, c.Hkv}, {c.page_stride, c.num_pages}};
    for (Dim& x : dim) {
        if (x.n == 1) x.stride = tsa::kDHead;  // never taken
        if (x.stride < tsa::kDHead || x.stride % 8 != 0 || x.stride > kMaxStride)
            return fail(TSA_ERR_INVALID_ARG, "cache: strides must be multiples of 8 elements, at least d (got page %lld, head %lld, row %lld)",
                        (long long)c.page_stride, (long long)c.head_stride, (long long)c.row_stride);
    }
    Dim by[3] = {dim[0], dim[1], dim[2]};
    std::sort(by, by + 3, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
    __int128 span = tsa::kDHead;
    for (const Dim& x : by) {
        if (x.n == 1) continue;
        if (x.stride < span) return fail(TSA_ERR_INVALID_ARG, "cache: rows overlap (page_stride %lld, head_stride %lld, row_stride %lld)",
                                         (long long)c.page_stride, (long long)c.head_stride, (long long)c.row_stride);
        span += (__int128)x.stride * (x.n - 1);
    }
    if (span > ((__int128)1 << 46)) return fail(TSA_ERR_INVALID_ARG, "cache: K spans more than 2^46 elements");
    out->K = c.K;
    out->V = c.V;
    out->table = c.page_table;
    out->row_stride = dim[0].stride;
    out->head_stride = dim[1].stride;
    out->page_stride = dim[2].stride;
    out->num_pages = c.num_pages;
    out->page_size = c.page_size;
    out->width = c.max_pages;
    out->B = c.B;
    out->Hkv = c.Hkv;
    out->half = c.dtype == TSA_FP16;
    return TSA_OK;
}

tsa_status check_cache_pointers(const tsa_paged_cache& c) {
    if (!c.K || !c.V || !c.page_table) return fail(TSA_ERR_INVALID_ARG, "cache: NULL pointer");
    if (!aligned16(c.K) || !aligned16(c.V)) return fail(TSA_ERR_INVALID_ARG, "cache: K and V must be 16-byte aligned");
    return TSA_OK;
}

tsa_status check_group(int Hq, int Hkv) {
    if (Hq <= 0 || Hq % Hkv != 0) return fail(TSA_ERR_INVALID_ARG, "Hq=%d is not a positive multiple of Hkv=%d", Hq, Hkv);
    if (Hq / Hkv > tsa::kMaxGroup)
        return fail(TSA_ERR_UNSUPPORTED, "GQA group Hq/Hkv=%d above %d", Hq / Hkv, tsa::kMaxGroup);
    return TSA_OK;
}

tsa_status check_rotation(const tsa_rotation& r, tsa::Rotation* out) {
    if (r.rot_dim < 0 || r.rot_dim > tsa::kDHead || r.rot_dim % 16 != 0)
        return fail(TSA_ERR_INVALID_ARG, "rot_dim must be a multiple of 16 in [0, 128] (got %d)", r.rot_dim);
    if (r.rot_dim > 0 && (!r.inv_freq || (reinterpret_cast<uintptr_t>(r.inv_freq) & 7u)))
        return fail(TSA_ERR_INVALID_ARG, "inv_freq must be an aligned pointer");
    out->inv_freq = r.inv_freq;
    out->rot_dim = r.rot_dim;
    out->interleaved = r.interleaved != 0;
    return TSA_OK;
}

// heads of 128 elements: readable by 16 bytes; a head or token that is the only one has no stride
tsa_status check_heads(const void* p, long long st, long long sh, int T, int H, const char* what, tsa::Heads* out) {
    if (H == 0 || T == 0) return TSA_OK;
    if (!p) return fail(TSA_ERR_INVALID_ARG, "%s: NULL pointer", what);
    if (!aligned16(p)) return fail(TSA_ERR_INVALID_ARG, "%s must be 16-byte aligned", what);
    if (T == 1) st = 0;
    if (H == 1) sh = 0;
    if (st % 8 != 0 || sh % 8 != 0 || st < 0 || sh < 0 || st > kMaxStride || sh > kMaxStride)
        return fail(TSA_ERR_INVALID_ARG, "%s: strides must be multiples of 8 elements, not negative (got %lld, %lld)", what, st, sh);
    out->p = p;
    out->st = st;
    out->sh = sh;
    return TSA_OK;
}

// an output's heads must not overlap one another
tsa_status check_out(const tsa::Heads& o, int T, int H, const char* what) {
    if (T == 0 || H == 0) return TSA_OK;
    long long lo = o.sh, nlo = H, hi = o.st, nhi = T;
    if (T > 1 && (H == 1 || lo > hi)) std::swap(lo, hi), std::swap(nlo, nhi);
    __int128 span = tsa::kDHead;
    for (int i = 0; i < 2; ++i) {
        const long long s = i ? hi : lo, n = i ? nhi : nlo;
        if (n == 1) continue;
        if (s < span) return fail(TSA_ERR_INVALID_ARG, "%s: heads overlap", what);
        span += (__int128)s * (n - 1);
    }
    return TSA_OK;
}

tsa_status check_ws(const void* ws, size_t ws_bytes, size_t need) {
    if (ws == nullptr) return fail(TSA_ERR_WORKSPACE, "workspace pointer is NULL");
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return fail(TSA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    if (ws_bytes < need) return fail(TSA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
    return TSA_OK;
}

// [flag 256 B][the CTAs' pieces][a shared prefix's partials, and
// those of the sequences' own rows]
struct Layout {
    size_t pieces, parts, total;
};

// Whether the prefix gets its own pass.  It saves reading the prefix's rows again for
// every sequence but one (out of L2, after the first), and costs its set-up and partials to
// write and join.  Measured, us without and with it, page 64, 100 own rows a sequence:
//
//   rows saved, about    20,000     40,000     82,000    160,000    320,000
//    4 x    32/8 heads   9.5 13.4  11.2 14.5  14.5 15.1  20.1 17.6  31.5 23.4
//    8 x    32/8         9.6 12.7  11.0 13.8  13.9 15.5  19.1 16.5  28.6 18.4
//   16 x    64/8        10.1 17.4  11.3 18.0  14.5 18.4  19.6 19.6  29.1 19.6
//   32 x     8/8                   12.4 17.6  14.5 18.0  19.4 17.2  27.8 17.6
//    8 x     8/2         9.2 12.0  10.4 13.0  13.7 13.3  18.4 14.9  28.3 16.8
//   16 x     8/1         9.6 14.1  10.9 13.6  13.7 14.7  18.6 16.9  28.5 17.8
//   64 x    32/8                   14.5 24.7  18.8 24.7  22.3 25.0  31.5 23.8
//    2 x    32/8        10.2 13.7  12.7 14.8  17.2 20.1  26.0 28.3  42.8 45.4
//
// (graph replays; with cold caches the same within 2 us, but for two sequences, where it
// is 24.6 28.7, 41.0 36.9, 69.6 54.3 in the last three columns).  So it pays from 80,000 to
// 160,000 rows on, for 64 sequences and more from 250,000.  The bound is the lower end,
// where tsa.h has it; between the two a call may lose up to 4 us (64 sequences: 6).
bool shares(const tsa::Pages& c, int prefix_len) {
    return prefix_len > 0 && prefix_len <= c.rows_cap() && (c.B - 1LL) * prefix_len * c.Hkv >= 81920;
}

Layout layout(const tsa::Pages& c, int Hq, int prefix_len) {
    Layout L;
    size_t off = kFlagBytes;
    L.pieces = off;
    off += a256((size_t)2 * tsa::paged_ctas() * (Hq / c.Hkv) * tsa::kPartFloats * sizeof(float));
    L.parts = off;
    if (shares(c, prefix_len))
        off += a256((size_t)(tsa::prefix_max_splits(c.Hkv, c.B * (Hq / c.Hkv), prefix_len) + 1) * c.B * Hq *
                    tsa::kPartFloats * sizeof(float));
    L.total = off;
    return L;
}

tsa_status attn(const tsa_paged_attn_args* a, bool prefix, const char* what, void* stream) {
    if (!a) return fail(TSA_ERR_INVALID_ARG, "%s: NULL args", what);
    tsa::Pages c;
    TSA_TRY(check_cache(a->cache, &c));
    TSA_TRY(check_group(a->Hq, c.Hkv));
    if (!std::isfinite(a->scale * tsa::kLog2e) || !(a->scale > 0.f))  // (the kernels' scores are in base 2)
        return fail(TSA_ERR_INVALID_ARG, "%s: scale must be > 0 and scale * log2(e) finite (got %g)", what, (double)a->scale);
    if (a->prefix_len < 0 || (!prefix && a->prefix_len != 0))
        return fail(TSA_ERR_INVALID_ARG, "%s: prefix_len must be %s (got %d)", what, prefix ? ">= 0" : "0", a->prefix_len);
    if (prefix && (a->idx || a->k_per_seq))
        return fail(TSA_ERR_INVALID_ARG, "%s: idx and k_per_seq must be NULL (every row is attended)", what);
    if (a->idx && a->k_max <= 0) return fail(TSA_ERR_INVALID_ARG, "%s: k_max must be > 0 with an index list (got %d)", what, a->k_max);
    if (!a->idx && (a->k_per_seq || a->k_max != 0))
        return fail(TSA_ERR_INVALID_ARG, "%s: k_per_seq and k_max belong to an index list", what);
    if (c.B > 0) {
        TSA_TRY(check_cache_pointers(a->cache));
        if (!a->Q || !a->seq_lens || !a->O) return fail(TSA_ERR_INVALID_ARG, "%s: NULL pointer", what);
        if (!aligned16(a->Q) || !aligned16(a->O)) return fail(TSA_ERR_INVALID_ARG, "%s: Q and O must be 16-byte aligned", what);
        if (a->O == a->Q) return fail(TSA_ERR_INVALID_ARG, "%s: O must not be Q", what);
    }
    if ((long long)c.B * c.Hkv * ((c.rows_cap() + 63LL) / 64 + 4) > INT32_MAX)
        return fail(TSA_ERR_UNSUPPORTED, "%s: B*Hkv*max_pages*page_size above 2^37 rows", what);
    const Layout L = layout(c, a->Hq, a->prefix_len);
    TSA_TRY(check_ws(a->ws, a->ws_bytes, L.total));
    if (a->prefix_len > 1 << 30) return fail(TSA_ERR_UNSUPPORTED, "%s: prefix_len=%d above 2^30", what, a->prefix_len);
    char* w = static_cast<char*>(a->ws);
    unsigned* flag = static_cast<unsigned*>(a->ws);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    tsa::PrefixParts pre;
    if (shares(c, a->prefix_len)) {  // (a prefix above the table's rows: no sequence holds it)
        const cudaError_t e = tsa::launch_prefix(c, a->Q, a->Hq, a->seq_lens, a->prefix_len, a->scale,
                                                 reinterpret_cast<float*>(w + L.parts), &pre, flag, st);
        if (e != cudaSuccess) return cuda_fail(e, "tsa_prefix_attn (shared prefix)");
    }
    const cudaError_t e = tsa::launch_paged_attn(c, a->Q, a->Hq, a->seq_lens, a->idx, a->k_per_seq, a->k_max, a->scale,
                                                 a->O, a->lse, reinterpret_cast<float*>(w + L.pieces),
                                                 pre, flag, st);
    if (e != cudaSuccess) return cuda_fail(e, what);
    return TSA_OK;
}

}  // namespace

extern "C" {

tsa_status tsa_qk_norm_rope(const tsa_qk_args* a, void* stream) {
    if (!a) return fail(TSA_ERR_INVALID_ARG, "tsa_qk_norm_rope: NULL args");
    TSA_TRY(check_dtype(a->dtype, a->d));
    if (a->T < 0 || a->Hq < 0 || a->Hkv < 0 || (long long)a->Hq + a->Hkv > 1 << 20)
        return fail(TSA_ERR_INVALID_ARG, "tsa_qk_norm_rope: need T, Hq, Hkv >= 0 (got T=%d Hq=%d Hkv=%d)", a->T, a->Hq, a->Hkv);
    if (!std::isfinite(a->eps) || a->eps < 0.f)
        return fail(TSA_ERR_INVALID_ARG, "tsa_qk_norm_rope: eps must be finite and >= 0 (got %g)", (double)a->eps);
    tsa::Rotation rot;
    TSA_TRY(check_rotation(a->rot, &rot));
    tsa::Heads q, k, qo, ko;
    TSA_TRY(check_heads(a->q, a->q_stride_t, a->q_stride_h, a->T, a->Hq, "q", &q));
    TSA_TRY(check_heads(a->k, a->k_stride_t, a->k_stride_h, a->T, a->Hkv, "k", &k));
    TSA_TRY(check_heads(a->q_out, a->q_out_stride_t, a->q_out_stride_h, a->T, a->Hq, "q_out", &qo));
    TSA_TRY(check_heads(a->k_out, a->k_out_stride_t, a->k_out_stride_h, a->T, a->Hkv, "k_out", &ko));
    TSA_TRY(check_out(qo, a->T, a->Hq, "q_out"));
    TSA_TRY(check_out(ko, a->T, a->Hkv, "k_out"));
    // an output that begins where its input does is that input, stride by stride
    if ((a->Hq > 0 && qo.p && qo.p == q.p && (qo.st != q.st || qo.sh != q.sh)) ||
        (a->Hkv > 0 && ko.p && ko.p == k.p && (ko.st != k.st || ko.sh != k.sh)))
        return fail(TSA_ERR_INVALID_ARG, "tsa_qk_norm_rope: an output in its input's place must have its strides");
    if (rot.rot_dim > 0 && a->T > 0 && !a->positions) return fail(TSA_ERR_INVALID_ARG, "tsa_qk_norm_rope: positions: NULL pointer");
    if (!aligned16(a->q_weight) || !aligned16(a->k_weight))
        return fail(TSA_ERR_INVALID_ARG, "tsa_qk_norm_rope: weights must be 16-byte aligned");
    const cudaError_t e = tsa::launch_qk_norm_rope(q, k, qo, ko, a->T, a->Hq, a->Hkv, a->dtype == TSA_FP16, a->q_weight,
                                                   a->k_weight, a->eps, a->positions, rot,
                                                   static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "tsa_qk_norm_rope");
    return TSA_OK;
}

tsa_status tsa_paged_append(const tsa_append_args* a, void* stream) {
    if (!a) return fail(TSA_ERR_INVALID_ARG, "tsa_paged_append: NULL args");
    tsa::Pages c;
    TSA_TRY(check_cache(a->cache, &c));
    if (a->T < 0) return fail(TSA_ERR_INVALID_ARG, "tsa_paged_append: T must be >= 0 (got %d)", a->T);
    tsa::Rotation rot;
    TSA_TRY(check_rotation(a->rot, &rot));
    tsa::Heads k, v;
    TSA_TRY(check_heads(a->K, a->k_stride_t, a->k_stride_h, a->T, c.Hkv, "K", &k));
    TSA_TRY(check_heads(a->V, a->v_stride_t, a->v_stride_h, a->T, c.Hkv, "V", &v));
    if (a->T > 0) {
        TSA_TRY(check_cache_pointers(a->cache));
        if (!a->row) return fail(TSA_ERR_INVALID_ARG, "tsa_paged_append: row: NULL pointer");
        if (!a->seq && a->T > c.B)
            return fail(TSA_ERR_INVALID_ARG, "tsa_paged_append: T=%d tokens without seq, but B=%d sequences", a->T, c.B);
    }
    TSA_TRY(check_ws(a->ws, a->ws_bytes, kFlagBytes));
    const cudaError_t e = tsa::launch_paged_append(c, k, v, a->T, a->seq, a->row, a->positions, rot,
                                                   static_cast<unsigned*>(a->ws), static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "tsa_paged_append");
    return TSA_OK;
}

size_t tsa_paged_workspace_size(const tsa_paged_cache* cache, int32_t Hq, int32_t prefix_len) {
    if (!cache) {
        fail(TSA_ERR_INVALID_ARG, "tsa_paged_workspace_size: NULL cache");
        return 0;
    }
    tsa::Pages c;
    if (check_cache(*cache, &c) != TSA_OK) return 0;
    if (Hq == 0 && prefix_len == 0) return kFlagBytes;
    if (check_group(Hq, c.Hkv) != TSA_OK) return 0;
    if (prefix_len < 0) {
        fail(TSA_ERR_INVALID_ARG, "tsa_paged_workspace_size: prefix_len must be >= 0 (got %d)", prefix_len);
        return 0;
    }
    return layout(c, Hq, prefix_len).total;
}

tsa_status tsa_paged_attn(const tsa_paged_attn_args* args, void* stream) { return attn(args, false, "tsa_paged_attn", stream); }

tsa_status tsa_prefix_attn(const tsa_paged_attn_args* args, void* stream) { return attn(args, true, "tsa_prefix_attn", stream); }

}  // extern "C"
