// Host side of the prompt and shared-prompt attention operators (fq_qk_norm_rope,
// fq_attn_prompt, fq_attn_shared): argument checks, then the launches.  Every check runs
// before anything is enqueued.

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "api_util.h"
#include "fq.h"
#include "kernels.h"

using namespace fq;

namespace {

constexpr uint64_t MAX_ROWS = 1ull << 30;     // query or key rows of one call (32-bit row indexes)
constexpr uint64_t MAX_STRIDE = 1ull << 36;   // elements: byte strides stay below the 2^40 of a tensor map
constexpr uint32_t MAX_HEADS = 1024;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

fq_status check_heads(uint32_t Hq, uint32_t Hkv) {
    if (!Hq || !Hkv || Hq % Hkv)
        return fail(FQ_ERR_INVALID_ARGUMENT, "num_attention_heads %u not a positive multiple of num_key_value_heads %u", Hq, Hkv);
    if (Hq > MAX_HEADS) return fail(FQ_ERR_INVALID_ARGUMENT, "more than %u heads", MAX_HEADS);
    const uint32_t G = Hq / Hkv;
    if (G != 1 && G != 2 && G != 4 && G != 8) return fail(FQ_ERR_UNSUPPORTED, "GQA group %u (1, 2, 4 or 8)", G);
    return FQ_OK;
}

// a view of which rows [row0, row0 + n) are used
fq_status check_view(const fq_kv_view& v, uint32_t Hkv, uint64_t row0, uint64_t n, const char* what, uint32_t s) {
    if (row0 + n > v.rows)
        return fail(FQ_ERR_KV_CACHE_OVERFLOW, "%s %u: rows %llu + %llu > %llu", what, s, (unsigned long long)row0,
                    (unsigned long long)n, (unsigned long long)v.rows);
    if (n == 0) return FQ_OK;
    if (!v.k || !v.v) return fail(FQ_ERR_INVALID_ARGUMENT, "%s %u: null k or v", what, s);
    if (!aligned16(v.k) || !aligned16(v.v)) return fail(FQ_ERR_INVALID_ARGUMENT, "%s %u: k or v not 16-byte aligned", what, s);
    if (v.row_stride % 8 || v.head_stride % 8 || v.row_stride < HEAD_DIM || v.row_stride > MAX_STRIDE ||
        (Hkv > 1 && v.head_stride < HEAD_DIM) || v.head_stride > MAX_STRIDE)
        return fail(FQ_ERR_INVALID_ARGUMENT, "%s %u: strides (%llu, %llu) (multiples of 8 elements, at least %d)", what, s,
                    (unsigned long long)v.row_stride, (unsigned long long)v.head_stride, HEAD_DIM);
    if (row0 + n > MAX_ROWS) return fail(FQ_ERR_INVALID_ARGUMENT, "%s %u: more than 2^30 rows", what, s);
    return FQ_OK;
}

fq_status row_stride(uint64_t given, uint64_t width, uint64_t multiple, const char* what, int64_t* out) {
    const uint64_t r = given ? given : width;
    if (r < width || r % multiple || r > MAX_STRIDE)
        return fail(FQ_ERR_INVALID_ARGUMENT, "%s row stride %llu (at least %llu, a multiple of %llu)", what,
                    (unsigned long long)r, (unsigned long long)width, (unsigned long long)multiple);
    *out = (int64_t)r;
    return FQ_OK;
}

fq_status check_count(uint32_t n_seq) {
    if (n_seq == 0) return fail(FQ_ERR_INVALID_SEQUENCE_LENGTH, "empty batch");
    if (n_seq > (uint32_t)MAX_SEQ) return fail(FQ_ERR_INVALID_ARGUMENT, "%u sequences exceed %d", n_seq, MAX_SEQ);
    return FQ_OK;
}

KvRows rows_of(const fq_kv_view& v) {
    KvRows r;
    r.k = (uint16_t*)v.k;
    r.v = (uint16_t*)v.v;
    r.row_stride = (int64_t)v.row_stride;
    r.head_stride = (int64_t)v.head_stride;
    return r;
}

// the checks that both attentions share, and the common part of their arguments
fq_status attn_common(const void* q, uint64_t q_stride, uint32_t Hq, uint32_t Hkv, float scale, void* out,
                      uint64_t out_stride, fq_dtype out_dtype, uint64_t q_rows, void* ws, size_t ws_bytes, size_t need,
                      AttnIo& io) {
    if (out_dtype != FQ_BF16 && out_dtype != FQ_F32) return fail(FQ_ERR_UNSUPPORTED, "out dtype must be BF16 or F32");
    if (!std::isfinite(scale)) return fail(FQ_ERR_INVALID_ARGUMENT, "scale is not finite");
    if (q_rows > MAX_ROWS) return fail(FQ_ERR_INVALID_ARGUMENT, "more than 2^30 query rows");
    const uint64_t width = (uint64_t)Hq * HEAD_DIM;
    TRY(row_stride(q_stride, width, 8, "q", &io.q_stride));
    TRY(row_stride(out_stride, width, out_dtype == FQ_BF16 ? 8 : 4, "out", &io.out_stride));
    if (q_rows) {
        if (!q || !out) return fail(FQ_ERR_INVALID_ARGUMENT, "null q or out");
        if (!aligned16(q) || !aligned16(out)) return fail(FQ_ERR_INVALID_ARGUMENT, "q or out not 16-byte aligned");
        if (need > ws_bytes || (need && (!ws || !aligned16(ws))))
            return fail(FQ_ERR_INVALID_ARGUMENT, "workspace of %zu bytes, 16-byte aligned, needed (%zu given)", need, ws_bytes);
    }
    io.q = (const uint16_t*)q;
    io.out = out;
    io.out_f32 = out_dtype == FQ_F32;
    io.Hq = (int)Hq;
    io.Hkv = (int)Hkv;
    io.scale = scale;
    return FQ_OK;
}

}  // namespace

extern "C" {

fq_status fq_qk_norm_rope(const float* qkv, uint64_t qkv_stride, uint32_t n_seq, const uint32_t* len,
                          const uint32_t* pos0, const fq_kv_view* views, uint32_t n_views, const uint32_t* kv_row0,
                          uint32_t num_attention_heads, uint32_t num_key_value_heads, const float* q_norm,
                          const float* k_norm, float eps, const float* rope, uint32_t rope_rows, void* q_out,
                          uint64_t q_stride, void* stream) {
    const uint32_t Hq = num_attention_heads, Hkv = num_key_value_heads;
    TRY(check_heads(Hq, Hkv));
    TRY(check_count(n_seq));
    if (!len || !pos0 || !views || !kv_row0) return fail(FQ_ERR_INVALID_ARGUMENT, "null argument");
    if (n_views != 1 && n_views != n_seq) return fail(FQ_ERR_INVALID_ARGUMENT, "%u views for %u sequences", n_views, n_seq);
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(FQ_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
    QkRowsArgs a;
    TRY(row_stride(qkv_stride, (uint64_t)(Hq + 2 * Hkv) * HEAD_DIM, 4, "qkv", &a.qkv_stride));
    TRY(row_stride(q_stride, (uint64_t)Hq * HEAD_DIM, 8, "q", &a.q_stride));
    uint64_t rows = 0;
    for (uint32_t s = 0; s < n_seq; ++s) {
        const fq_kv_view& v = views[n_views == 1 ? 0 : s];
        a.row0[s] = (int32_t)rows;
        a.pos0[s] = (int32_t)pos0[s];
        a.kv_row0[s] = (int32_t)kv_row0[s];
        a.kv[s] = rows_of(v);
        if ((uint64_t)pos0[s] + len[s] > rope_rows)
            return fail(FQ_ERR_INVALID_SEQUENCE_LENGTH, "sequence %u: positions %u + %u > %u table rows", s, pos0[s], len[s], rope_rows);
        TRY(check_view(v, Hkv, kv_row0[s], len[s], "view", s));
        rows += len[s];
        if (rows > MAX_ROWS) return fail(FQ_ERR_INVALID_ARGUMENT, "more than 2^30 rows");
        for (uint32_t t = 0; t < s && len[s]; ++t)   // two sequences that write the same rows race
            if (len[t] && (a.kv[t].k == a.kv[s].k || a.kv[t].v == a.kv[s].v) &&
                kv_row0[t] < (uint64_t)kv_row0[s] + len[s] && kv_row0[s] < (uint64_t)kv_row0[t] + len[t])
                return fail(FQ_ERR_INVALID_ARGUMENT, "sequences %u and %u write the same rows", t, s);
    }
    if (rows == 0) return FQ_OK;
    if (!qkv || !q_norm || !k_norm || !rope || !q_out) return fail(FQ_ERR_INVALID_ARGUMENT, "null argument");
    if (!aligned16(qkv) || !aligned16(q_norm) || !aligned16(k_norm) || !aligned16(rope) || !aligned16(q_out))
        return fail(FQ_ERR_INVALID_ARGUMENT, "qkv, gains, rope and q_out must be 16-byte aligned");
    a.qkv = qkv;
    a.q_norm = q_norm;
    a.k_norm = k_norm;
    a.rope = (const float2*)rope;
    a.eps = eps;
    a.Hq = (int)Hq;
    a.Hkv = (int)Hkv;
    a.n_seq = (int)n_seq;
    a.rows = (int)rows;
    a.q_out = (uint16_t*)q_out;
    launch_qk_rows(a, (cudaStream_t)stream);
    CK(cudaGetLastError());
    return FQ_OK;
}

fq_status fq_attn_prompt_workspace(uint32_t n_seq, const uint32_t* q_len, const uint32_t* k_len,
                                   uint32_t num_attention_heads, uint32_t num_key_value_heads, size_t* bytes) {
    TRY(check_heads(num_attention_heads, num_key_value_heads));
    TRY(check_count(n_seq));
    if (!q_len || !k_len || !bytes) return fail(FQ_ERR_INVALID_ARGUMENT, "null argument");
    *bytes = 0;
    return FQ_OK;
}

fq_status fq_attn_prompt(const void* q, uint64_t q_stride, const fq_kv_view* views, uint32_t n_views, uint32_t n_seq,
                         const uint32_t* q_len, const uint32_t* kv_row0, const uint32_t* k_len,
                         uint32_t num_attention_heads, uint32_t num_key_value_heads, float scale, void* out,
                         uint64_t out_stride, fq_dtype out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    const uint32_t Hq = num_attention_heads, Hkv = num_key_value_heads;
    TRY(check_heads(Hq, Hkv));
    TRY(check_count(n_seq));
    if (!q_len || !k_len || !views) return fail(FQ_ERR_INVALID_ARGUMENT, "null argument");
    if (n_views != 1 && n_views != n_seq) return fail(FQ_ERR_INVALID_ARGUMENT, "%u views for %u sequences", n_views, n_seq);
    PromptArgs a;
    a.n_seq = (int)n_seq;
    uint64_t qr = 0, kr = 0;
    for (uint32_t s = 0; s < n_seq; ++s) {
        const fq_kv_view& v = views[n_views == 1 ? 0 : s];
        const uint64_t r0 = kv_row0 ? kv_row0[s] : n_views == 1 ? kr : 0;
        TRY(check_view(v, Hkv, r0, k_len[s], "sequence", s));
        if (q_len[s] > MAX_ROWS) return fail(FQ_ERR_INVALID_ARGUMENT, "more than 2^30 query rows");
        a.seq[s] = PromptSeq{(int32_t)qr, (int32_t)q_len[s], (int32_t)r0, (int32_t)k_len[s]};
        a.kv[s] = rows_of(v);
        qr += q_len[s];
        kr += k_len[s];
        if (qr > MAX_ROWS || kr > (uint64_t)MAX_SEQ * MAX_ROWS) return fail(FQ_ERR_INVALID_ARGUMENT, "more than 2^30 query rows");
    }
    TRY(attn_common(q, q_stride, Hq, Hkv, scale, out, out_stride, out_dtype, qr, workspace, workspace_bytes, 0, a.io));
    if (qr == 0) return FQ_OK;
    a.q_rows = (int)qr;
    launch_prompt(a, (cudaStream_t)stream);
    CK(cudaGetLastError());
    return FQ_OK;
}

fq_status fq_attn_shared_workspace(uint32_t n_seq, uint32_t prefix_len, const uint32_t* tail_len,
                                   uint32_t num_attention_heads, uint32_t num_key_value_heads, size_t* bytes) {
    TRY(check_heads(num_attention_heads, num_key_value_heads));
    TRY(check_count(n_seq));
    if (!tail_len || !bytes) return fail(FQ_ERR_INVALID_ARGUMENT, "null argument");
    *bytes = 0;
    return FQ_OK;
}

fq_status fq_attn_shared(const void* q, uint64_t q_stride, uint32_t n_seq, const fq_kv_view* prefix,
                         uint32_t prefix_len, const fq_kv_view* tails, const uint32_t* tail_len,
                         uint32_t num_attention_heads, uint32_t num_key_value_heads, float scale, void* out,
                         uint64_t out_stride, fq_dtype out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    const uint32_t Hq = num_attention_heads, Hkv = num_key_value_heads;
    TRY(check_heads(Hq, Hkv));
    TRY(check_count(n_seq));
    if (!tail_len) return fail(FQ_ERR_INVALID_ARGUMENT, "null argument");
    SharedArgs a;
    if (prefix_len) {
        if (!prefix) return fail(FQ_ERR_INVALID_ARGUMENT, "null prefix");
        TRY(check_view(*prefix, Hkv, 0, prefix_len, "prefix", 0));
        a.prefix = rows_of(*prefix);
    }
    a.prefix_len = (int)prefix_len;
    for (uint32_t s = 0; s < n_seq; ++s) {
        a.tail_len[s] = (int32_t)tail_len[s];
        if (!tail_len[s]) continue;
        if (!tails) return fail(FQ_ERR_INVALID_ARGUMENT, "null tails");
        TRY(check_view(tails[s], Hkv, 0, tail_len[s], "tail", s));
        a.tail[s] = rows_of(tails[s]);
    }
    TRY(attn_common(q, q_stride, Hq, Hkv, scale, out, out_stride, out_dtype, n_seq, workspace, workspace_bytes, 0, a.io));
    a.n_seq = (int)n_seq;
    launch_shared(a, (cudaStream_t)stream);
    CK(cudaGetLastError());
    return FQ_OK;
}

}  // extern "C"
