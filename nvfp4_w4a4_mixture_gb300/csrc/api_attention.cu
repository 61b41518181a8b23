// api_attention.cu -- the C ABI of the attention half of a block (include/moe_nvfp4.h): checks on the host, then the launch.
#include <algorithm>
#include <cmath>
#include <utility>

#include "api.cuh"
#include "attention.cuh"

using namespace moe;

namespace {

constexpr int kMaxRequests = 1 << 30;  // so that a search among them and a block of them a thread are counted in 32 bits

moe_status_t check_cache(const moe_kv_cache_t* C, KvCache* c)
{
    if (C->dtype != MOE_DTYPE_BF16 && C->dtype != MOE_DTYPE_E4M3) return fail(MOE_ERR_INVALID_ARG, "cache dtype=%d", C->dtype);
    if (C->D != 64 && C->D != 128 && C->D != 256) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "D=%d: 64, 128 or 256", C->D);
    if (C->n_kv < 1 || C->n_kv > 1024) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "n_kv=%d outside [1, 1024]", C->n_kv);
    if (C->page_size < 1 || C->page_size > 65536 || (C->page_size & (C->page_size - 1)))
        return fail(MOE_ERR_UNSUPPORTED_SHAPE, "page_size=%d: a power of two in [1, 65536]", C->page_size);
    if (C->n_pages < 1) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "n_pages=%d < 1", C->n_pages);
    if (C->dtype == MOE_DTYPE_BF16 && (C->k_scale || C->v_scale)) return fail(MOE_ERR_INVALID_ARG, "k_scale and v_scale go with an E4M3 cache");
    c->k = C->k;
    c->v = C->v;
    c->e4m3 = C->dtype == MOE_DTYPE_E4M3;
    c->n_pages = C->n_pages;
    c->page_log2 = 0;
    while ((1 << c->page_log2) < C->page_size) ++c->page_log2;
    c->n_kv = C->n_kv;
    c->D = C->D;
    c->ld_page = C->ld_page;
    c->ld_slot = C->ld_slot;
    c->ld_head = C->ld_head;
    c->k_scale = C->k_scale;
    c->v_scale = C->v_scale;
    return MOE_OK;
}

// Bytes from the cache's first element to behind its last.
int64_t cache_span(const moe_kv_cache_t* C)
{
    const int es = C->dtype == MOE_DTYPE_E4M3 ? 1 : 2;
    return ((C->n_pages - 1) * C->ld_page + (C->page_size - 1) * C->ld_slot + (C->n_kv - 1) * C->ld_head + C->D) * es;
}

// The cache's dimensions of more than one by their strides, the least first, with the elements from the first to behind the
// last of what lies below each (extent[n]: of the whole).
struct Levels {
    int n;
    int64_t ld[3], count[3], extent[4];
};

Levels levels_of(const moe_kv_cache_t* C)
{
    Levels l{0, {C->ld_page, C->ld_slot, C->ld_head}, {C->n_pages, C->page_size, C->n_kv}, {C->D}};
    for (int i = 0; i < 3; ++i) {
        int at = i;
        for (int j = i + 1; j < 3; ++j)
            if (l.ld[j] < l.ld[at]) at = j;
        std::swap(l.ld[i], l.ld[at]);
        std::swap(l.count[i], l.count[at]);
    }
    for (int i = 0; i < 3; ++i) {
        if (l.count[i] == 1) continue;
        l.ld[l.n] = l.ld[i];
        l.count[l.n] = l.count[i];
        l.extent[l.n + 1] = l.extent[l.n] + (l.count[i] - 1) * l.ld[i];
        ++l.n;
    }
    return l;
}

// Whether some element of the lowest `at` levels and one of the same shape that begins d elements behind it are one: d is a
// difference of their indices times the strides. Of each stride it holds two multiples at the most, since what lies below
// is no longer than the stride.
bool meet(const Levels& l, int at, int64_t d)
{
    if (d <= -l.extent[at] || d >= l.extent[at]) return false;
    if (at == 0) return true;
    const int64_t ld = l.ld[at - 1], down = d >= 0 ? d / ld : -((ld - 1 - d) / ld);
    for (int64_t i = down; i <= down + 1; ++i)
        if (i > -l.count[at - 1] && i < l.count[at - 1] && meet(l, at - 1, d - i * ld)) return true;
    return false;
}

moe_status_t check_cache_memory(const moe_kv_cache_t* C)
{
    const int es = C->dtype == MOE_DTYPE_E4M3 ? 1 : 2;
    if (!C->k || !C->v) return fail(MOE_ERR_INVALID_ARG, "NULL cache pointer");
    if (C->ld_page < 0 || C->ld_slot < 0 || C->ld_head < 0) return fail(MOE_ERR_INVALID_ARG, "negative cache stride");
    if (!aligned(C->k, 16) || !aligned(C->v, 16) || (C->n_pages > 1 && C->ld_page * es % 16) || (C->page_size > 1 && C->ld_slot * es % 16) ||
        (C->n_kv > 1 && C->ld_head * es % 16))
        return fail(MOE_ERR_MISALIGNED, "cache strides %lld, %lld, %lld: every head must start on 16 bytes", (long long)C->ld_page,
                    (long long)C->ld_slot, (long long)C->ld_head);
    // pages, slots and heads do not lie on one another: sorted by stride, each is at least the extent of those below
    const Levels l = levels_of(C);
    for (int i = 0; i < l.n; ++i)
        if (l.ld[i] < l.extent[i]) return fail(MOE_ERR_INVALID_ARG, "cache strides %lld, %lld, %lld: heads overlap", (long long)C->ld_page,
                                               (long long)C->ld_slot, (long long)C->ld_head);
    if ((C->k_scale && !aligned(C->k_scale, 4)) || (C->v_scale && !aligned(C->v_scale, 4)))
        return fail(MOE_ERR_MISALIGNED, "k_scale and v_scale must be 4-byte aligned");
    return MOE_OK;
}

moe_status_t check_requests(const moe_requests_t* R, int page_size, int T, Requests* r)
{
    if (R->S < 1) return fail(MOE_ERR_INVALID_ARG, "S=%d: no request holds the T=%d rows", R->S, T);
    if (R->S > kMaxRequests) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "S=%d: more than 2^30", R->S);
    if (R->max_pages < 1) return fail(MOE_ERR_INVALID_ARG, "max_pages=%d < 1", R->max_pages);
    if (!R->seg_offsets || !R->kv_len || !R->pages) return fail(MOE_ERR_INVALID_ARG, "NULL table pointer");
    if (R->S > 1 && R->ld_pages < R->max_pages)
        return fail(MOE_ERR_INVALID_ARG, "pages: row stride %lld < max_pages=%d", (long long)R->ld_pages, R->max_pages);
    if (!aligned(R->seg_offsets, 4) || !aligned(R->kv_len, 4) || !aligned(R->pages, 4))
        return fail(MOE_ERR_MISALIGNED, "seg_offsets, kv_len and pages must be 4-byte aligned");
    r->S = R->S;
    r->seg_offsets = R->seg_offsets;
    r->kv_len = R->kv_len;
    r->pages = R->pages;
    r->ld_pages = R->S > 1 ? R->ld_pages : 0;
    r->max_len = static_cast<int64_t>(R->max_pages) * page_size;
    return MOE_OK;
}

bool overlaps_tables(const void* out, int64_t ld, int64_t width, int T, const moe_requests_t* R, const moe_kv_cache_t* C)
{
    const int64_t span = cache_span(C);
    return rows_overlap_bytes(out, ld, width, T, R->seg_offsets, 4LL * (R->S + 1LL)) || rows_overlap_bytes(out, ld, width, T, R->kv_len, 4LL * R->S) ||
           rows_overlap_bytes(out, ld, width, T, R->pages, 4 * ((R->S - 1) * R->ld_pages + R->max_pages)) ||
           rows_overlap_bytes(out, ld, width, T, C->k, span) || rows_overlap_bytes(out, ld, width, T, C->v, span) ||
           rows_overlap_bytes(out, ld, width, T, C->k_scale, 4LL * C->n_kv) || rows_overlap_bytes(out, ld, width, T, C->v_scale, 4LL * C->n_kv);
}

}  // namespace

extern "C" {

moe_status_t moe_cache_append(const moe_kv_cache_t* C, const moe_requests_t* R, const moe_rotary_t* P, const uint16_t* q,
                              int64_t ld_q, const uint16_t* k, int64_t ld_k, const uint16_t* v, int64_t ld_v, int T,
                              uint16_t* q_out, int64_t ld_q_out, void* ws, size_t ws_bytes, moe_stream_t stream)
{
    if (!C || !R || !P) return fail(MOE_ERR_INVALID_ARG, "cache, requests or rotary is NULL");
    AppendArgs a{};
    MOE_TRY(check_cache(C, &a.c));
    const int D = C->D;
    if (P->n_q < 0 || P->n_q > 1024) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "n_q=%d outside [0, 1024]", P->n_q);
    if (P->rot < 0 || P->rot > D || P->rot % 16) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "rot=%d not a multiple of 16 in [0, D=%d]", P->rot, D);
    if (!(P->eps >= 0.0f)) return fail(MOE_ERR_INVALID_ARG, "eps=%g: must be >= 0", static_cast<double>(P->eps));
    if (T < 0) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "T=%d < 0", T);
    if (T == 0) return MOE_OK;  // an empty batch: nothing is read or written, the pointers may be NULL
    MOE_TRY(check_cache_memory(C));
    MOE_TRY(check_requests(R, C->page_size, T, &a.r));
    if ((P->rot > 0) != (P->inv_freq != nullptr)) return fail(MOE_ERR_INVALID_ARG, "inv_freq and rot=%d go together", P->rot);
    if ((P->n_q > 0) != (q != nullptr) || (P->n_q > 0) != (q_out != nullptr)) return fail(MOE_ERR_INVALID_ARG, "q, q_out and n_q=%d go together", P->n_q);
    if (P->w_q && !P->n_q) return fail(MOE_ERR_INVALID_ARG, "w_q needs q");
    if (!k || !v) return fail(MOE_ERR_INVALID_ARG, "NULL tensor pointer");
    const int64_t wq = static_cast<int64_t>(P->n_q) * D, wk = static_cast<int64_t>(C->n_kv) * D;
    if (q) MOE_TRY(check_rows("q", q, ld_q, wq, 2, T));
    if (q) MOE_TRY(check_rows("q_out", q_out, ld_q_out, wq, 2, T));
    MOE_TRY(check_rows("k", k, ld_k, wk, 2, T));
    MOE_TRY(check_rows("v", v, ld_v, wk, 2, T));
    if (!aligned(P->inv_freq, 4) || !aligned(P->w_q, 16) || !aligned(P->w_k, 16))
        return fail(MOE_ERR_MISALIGNED, "w_q and w_k must be 16-byte, inv_freq 4-byte aligned");
    if (q) {
        if (!(q_out == q && (T == 1 || ld_q_out == ld_q)) && rows_overlap(q_out, ld_q_out * 2, wq * 2, q, ld_q * 2, wq * 2, T))
            return fail(MOE_ERR_INVALID_ARG, "q_out overlaps q without being q");
        if (rows_overlap(q_out, ld_q_out * 2, wq * 2, k, ld_k * 2, wk * 2, T) || rows_overlap(q_out, ld_q_out * 2, wq * 2, v, ld_v * 2, wk * 2, T) ||
            rows_overlap_bytes(q_out, ld_q_out * 2, wq * 2, T, P->inv_freq, 2LL * P->rot) || rows_overlap_bytes(q_out, ld_q_out * 2, wq * 2, T, P->w_q, 2LL * D) ||
            rows_overlap_bytes(q_out, ld_q_out * 2, wq * 2, T, P->w_k, 2LL * D) || overlaps_tables(q_out, ld_q_out * 2, wq * 2, T, R, C))
            return fail(MOE_ERR_INVALID_ARG, "q_out overlaps another argument");
    }
    const int64_t span = cache_span(C);
    for (const void* cache : {static_cast<const void*>(C->k), static_cast<const void*>(C->v)})
        if (rows_overlap_bytes(q, ld_q * 2, wq * 2, T, cache, span) || rows_overlap_bytes(k, ld_k * 2, wk * 2, T, cache, span) ||
            rows_overlap_bytes(v, ld_v * 2, wk * 2, T, cache, span))
            return fail(MOE_ERR_INVALID_ARG, "the cache overlaps q, k or v");
    const int64_t apart = static_cast<const char*>(C->v) - static_cast<const char*>(C->k);  // (a multiple of 16)
    const Levels l = levels_of(C);
    if (meet(l, l.n, apart / (C->dtype == MOE_DTYPE_E4M3 ? 1 : 2))) return fail(MOE_ERR_INVALID_ARG, "keys and values lie on one another");
    MOE_TRY(check_ws(ws, ws_bytes, sizeof(WsHeader)));
    MOE_TRY(check_device());
    a.T = T;
    a.n_q = P->n_q;
    a.rot = P->rot;
    a.interleaved = P->interleaved != 0;
    a.inv_freq = P->inv_freq;
    a.w_q = P->w_q;
    a.w_k = P->w_k;
    a.eps = P->eps;
    a.w_offset = P->w_offset;
    a.q = q;
    a.k = k;
    a.v = v;
    a.ld_q = ld_q;
    a.ld_k = ld_k;
    a.ld_v = ld_v;
    a.q_out = q_out;
    a.ld_q_out = ld_q_out;
    a.status = &static_cast<WsHeader*>(ws)->status;
    MOE_CUDA(launch_cache_append(a, device_sm_count(), static_cast<cudaStream_t>(stream)), "cache append launch");
    return MOE_OK;
}

static moe_status_t check_attention(int n_q, int n_kv, int max_new)
{
    if (n_q < 1 || n_q % n_kv || n_q / n_kv > 64) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "n_q=%d: a multiple of n_kv=%d, at most 64 times", n_q, n_kv);
    if (max_new < 1 || max_new > 16) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "max_new=%d outside [1, 16]", max_new);
    return MOE_OK;
}

size_t moe_attention_workspace_bytes(int S, int n_q, int n_kv, int D, int max_new)
{
    if (S < 0 || S > kMaxRequests || n_kv < 1 || n_kv > 1024 || (D != 64 && D != 128 && D != 256) || check_attention(n_q, n_kv, max_new) != MOE_OK) return 0;
    return attention_workspace_bytes(S, n_q, n_kv, D, max_new, device_sm_count());
}

moe_status_t moe_paged_attention(const moe_kv_cache_t* C, const moe_requests_t* R, const moe_attention_t* A,
                                 const uint16_t* q, int64_t ld_q, int T, uint16_t* out, int64_t ld_out, float* lse, void* ws,
                                 size_t ws_bytes, moe_stream_t stream)
{
    if (!C || !R || !A) return fail(MOE_ERR_INVALID_ARG, "cache, requests or attention is NULL");
    AttentionArgs a{};
    MOE_TRY(check_cache(C, &a.c));
    MOE_TRY(check_attention(A->n_q, C->n_kv, A->max_new));
    if (A->window < 0) return fail(MOE_ERR_INVALID_ARG, "window=%d < 0", A->window);
    if (!std::isfinite(A->scale)) return fail(MOE_ERR_INVALID_ARG, "scale=%g: must be finite", static_cast<double>(A->scale));
    if (T < 0) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "T=%d < 0", T);
    if (T == 0) return MOE_OK;  // an empty batch: nothing is read or written, the pointers may be NULL
    MOE_TRY(check_cache_memory(C));
    MOE_TRY(check_requests(R, C->page_size, T, &a.r));
    a.r.max_len = std::min<int64_t>(a.r.max_len, 0x7FFFFFFF - 64);  // a unit's positions fit 32 bits
    if (static_cast<int64_t>(T) * A->n_q > 0x7FFFFF00) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "T=%d rows of n_q=%d heads: 2^31 or more", T, A->n_q);
    if (!q || !out) return fail(MOE_ERR_INVALID_ARG, "NULL tensor pointer");
    const int64_t w = static_cast<int64_t>(A->n_q) * C->D;
    MOE_TRY(check_rows("q", q, ld_q, w, 2, T));
    MOE_TRY(check_rows("out", out, ld_out, w, 2, T));
    if (!aligned(lse, 4)) return fail(MOE_ERR_MISALIGNED, "lse must be 4-byte aligned");
    const int64_t lw = 4LL * A->n_q;
    if (!(out == q && (T == 1 || ld_out == ld_q)) && rows_overlap(out, ld_out * 2, w * 2, q, ld_q * 2, w * 2, T))
        return fail(MOE_ERR_INVALID_ARG, "out overlaps q without being q");
    if (overlaps_tables(out, ld_out * 2, w * 2, T, R, C)) return fail(MOE_ERR_INVALID_ARG, "out overlaps the cache or a table");
    if (lse && (rows_overlap(lse, lw, lw, q, ld_q * 2, w * 2, T) || rows_overlap(lse, lw, lw, out, ld_out * 2, w * 2, T) || overlaps_tables(lse, lw, lw, T, R, C)))
        return fail(MOE_ERR_INVALID_ARG, "lse overlaps another argument");
    MOE_TRY(check_ws(ws, ws_bytes, sizeof(WsHeader)));
    if (A->report) MOE_TRY(check_ws(A->report, sizeof(WsHeader), sizeof(WsHeader)));
    if (A->report != ws && rows_overlap_bytes(A->report, sizeof(WsHeader), sizeof(WsHeader), 1, ws, static_cast<int64_t>(ws_bytes)))
        return fail(MOE_ERR_INVALID_ARG, "report lies in ws");
    MOE_TRY(check_device());
    const int sms = device_sm_count();
    MOE_TRY(check_ws(ws, ws_bytes, attention_workspace_bytes(R->S, A->n_q, C->n_kv, C->D, A->max_new, sms)));
    a.T = T;
    a.n_q = A->n_q;
    a.group = A->n_q / C->n_kv;
    a.group_mul = (65536u + a.group - 1) / a.group;
    a.max_new = A->max_new;
    a.window = A->window;
    a.scale = A->scale;
    a.q = q;
    a.ld_q = ld_q;
    a.out = out;
    a.ld_out = ld_out;
    a.lse = lse;
    WsHeader* const header = static_cast<WsHeader*>(A->report ? A->report : ws);
    a.status = &header->status;
    a.hooks = header;
    MOE_CUDA(launch_paged_attention(a, ws, sms, static_cast<cudaStream_t>(stream)), "attention launch");
    return MOE_OK;
}

moe_status_t moe_quantize_fp8(const uint16_t* x, int64_t ld_x, int T, int K, uint8_t* codes, float* scale, moe_stream_t stream)
{
    if (K < 16 || K > 65536 || K % 16) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "K=%d not a multiple of 16 in [16, 65536]", K);
    if (T < 0) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "T=%d < 0", T);
    if (T == 0) return MOE_OK;  // an empty batch: nothing is read or written, the pointers may be NULL
    if (!x || !codes || !scale) return fail(MOE_ERR_INVALID_ARG, "NULL tensor pointer");
    MOE_TRY(check_rows("x", x, ld_x, K, 2, T));
    if (!aligned(codes, 16) || !aligned(scale, 4)) return fail(MOE_ERR_MISALIGNED, "codes must be 16-byte, scale 4-byte aligned");
    const int64_t sw = 4LL * ((K + 127) / 128);
    if (rows_overlap(codes, K, K, x, ld_x * 2, 2LL * K, T) || rows_overlap(scale, sw, sw, x, ld_x * 2, 2LL * K, T) || rows_overlap(codes, K, K, scale, sw, sw, T))
        return fail(MOE_ERR_INVALID_ARG, "x, codes and scale overlap");
    MOE_TRY(check_device());
    MOE_CUDA(launch_quantize_fp8(x, T > 1 ? ld_x : K, T, K, codes, scale, device_sm_count(), static_cast<cudaStream_t>(stream)), "FP8 quantize launch");
    return MOE_OK;
}

moe_status_t moe_gemm_fp8(const uint8_t* a, const float* a_scale, const uint8_t* b, const float* b_scale, int T, int N, int K,
                          void* out, int out_dtype, int64_t ld_out, void* ws, size_t ws_bytes, moe_stream_t stream)
{
    if (K < 16 || K > 65536 || K % 16) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "K=%d not a multiple of 16 in [16, 65536]", K);
    if (N < 8 || N > 1048576 || N % 8) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "N=%d not a multiple of 8 in [8, 1048576]", N);
    if (T < 0) return fail(MOE_ERR_UNSUPPORTED_SHAPE, "T=%d < 0", T);
    if (out_dtype != MOE_DTYPE_BF16 && out_dtype != MOE_DTYPE_F32) return fail(MOE_ERR_INVALID_ARG, "out_dtype=%d", out_dtype);
    if (T == 0) return MOE_OK;  // an empty batch: nothing is read or written, the pointers may be NULL
    if (!a || !a_scale || !b || !b_scale || !out) return fail(MOE_ERR_INVALID_ARG, "NULL tensor pointer");
    const int es = out_dtype == MOE_DTYPE_F32 ? 4 : 2;
    MOE_TRY(check_rows("out", out, ld_out, N, es, T));
    if (!aligned(a, 16) || !aligned(b, 16) || !aligned(a_scale, 4) || !aligned(b_scale, 4))
        return fail(MOE_ERR_MISALIGNED, "a and b must be 16-byte, their scales 4-byte aligned");
    const int64_t kb = (K + 127) / 128, nb = (N + 127) / 128, w = static_cast<int64_t>(N) * es;
    if (rows_overlap_bytes(out, ld_out * es, w, T, a, static_cast<int64_t>(T) * K) || rows_overlap_bytes(out, ld_out * es, w, T, b, static_cast<int64_t>(N) * K) ||
        rows_overlap_bytes(out, ld_out * es, w, T, a_scale, 4LL * T * kb) || rows_overlap_bytes(out, ld_out * es, w, T, b_scale, 4 * nb * kb))
        return fail(MOE_ERR_INVALID_ARG, "out overlaps an input");
    MOE_TRY(check_ws(ws, ws_bytes, sizeof(WsHeader)));
    MOE_TRY(check_device());
    GemmFp8Args g{};
    g.T = T;
    g.N = N;
    g.K = K;
    g.a = a;
    g.b = b;
    g.a_scale = a_scale;
    g.b_scale = b_scale;
    g.out = out;
    g.out_f32 = es == 4;
    g.ld_out = T > 1 ? ld_out : N;
    g.status = &static_cast<WsHeader*>(ws)->status;
    g.hooks = static_cast<const WsHeader*>(ws);
    MOE_CUDA(launch_gemm_fp8(g, device_sm_count(), static_cast<cudaStream_t>(stream)), "FP8 GEMM launch");
    return MOE_OK;
}

}  // extern "C"
