// Host side of the operators on windows, pages and caches made shorter (fq_attn_window, fq_attn_paged,
// fq_qk_norm_rope_paged): argument checks, then the launches.  The checks and the work lists
// are those of attn_host.h.

#include <mutex>

#include "attn_host.h"

using namespace fq;

namespace {

constexpr int MAX_DEVICES = 64;
struct Device {
    std::mutex mu;
    uint32_t* bad = nullptr;    // (set once the kernels are prepared)
};
Device g_devices[MAX_DEVICES];

fq_status prepare_device(uint32_t** waits, uint32_t** bad) {
    int dev = 0;
    TRY(attn_device(&dev, waits));
    Device& d = g_devices[dev];
    std::lock_guard<std::mutex> lk(d.mu);
    if (!d.bad) {
        uint32_t* w = nullptr;
        CK(attn_window_tiles_prepare());
        CK(attn_window_rows_prepare());
        CK(attn_page_word(&w));
        attn_set_page_word(dev, w);
        d.bad = w;
    }
    *bad = d.bad;
    return FQ_OK;
}

AttnMask mask_of(uint32_t window, uint32_t sinks) {
    AttnMask m;
    if (window && window < (uint32_t)m.window) m.window = (int32_t)window;
    m.sinks = (int32_t)std::min<uint64_t>(sinks, MAX_ROWS);
    return m;
}

// a pool and the table of n_seq sequences with the given rows (0: none are used)
fq_status check_pages(const fq_kv_pages* pages, const int32_t* table, uint64_t table_stride, uint32_t n_seq, const uint64_t* rows,
                      uint32_t Hkv, KvPages& p) {
    if (!pages) return fail(FQ_ERR_INVALID_ARGUMENT, "null pages");
    const fq_kv_pages& g = *pages;
    if (g.page_rows < 16 || g.page_rows > 256 || (g.page_rows & (g.page_rows - 1)))
        return fail(FQ_ERR_INVALID_ARGUMENT, "pages of %u rows (16, 32, 64, 128 or 256)", g.page_rows);
    if (g.n_pages > 0x7FFFFFFFu) return fail(FQ_ERR_INVALID_ARGUMENT, "2^31 pages or more");
    if (table_stride > MAX_STRIDE) return fail(FQ_ERR_INVALID_ARGUMENT, "table stride above 2^36");
    while (1u << p.shift < g.page_rows) ++p.shift;
    uint64_t most = 0;
    for (uint32_t s = 0; s < n_seq; ++s) {
        most = std::max(most, rows[s]);
        if (rows[s] > MAX_ROWS) return fail(FQ_ERR_INVALID_ARGUMENT, "more than 2^30 rows");
        if ((rows[s] + g.page_rows - 1) / g.page_rows > table_stride)
            return fail(FQ_ERR_KV_CACHE_OVERFLOW, "sequence %u: %llu rows need more than the table's %llu pages of %u", s,
                        (unsigned long long)rows[s], (unsigned long long)table_stride, g.page_rows);
    }
    p.n_pages = (int32_t)g.n_pages;
    p.table = table;
    p.table_stride = (int64_t)table_stride;
    if (most == 0) return FQ_OK;
    if (!table || (reinterpret_cast<uintptr_t>(table) & 3)) return fail(FQ_ERR_INVALID_ARGUMENT, "null or misaligned page table");
    if (!g.n_pages) return fail(FQ_ERR_KV_CACHE_OVERFLOW, "a pool without pages");
    if (!g.k || !g.v) return fail(FQ_ERR_INVALID_ARGUMENT, "pages: null k or v");
    if (!aligned16(g.k) || !aligned16(g.v)) return fail(FQ_ERR_INVALID_ARGUMENT, "pages: k or v not 16-byte aligned");
    auto bad = [](uint64_t stride) { return stride % 8 || stride < HEAD_DIM || stride > MAX_STRIDE; };
    if (bad(g.row_stride) || (Hkv > 1 && bad(g.head_stride)) || (g.n_pages > 1 && bad(g.page_stride)))
        return fail(FQ_ERR_INVALID_ARGUMENT, "pages: strides (%llu, %llu, %llu) (multiples of 8 elements, %d to 2^36)",
                    (unsigned long long)g.page_stride, (unsigned long long)g.row_stride, (unsigned long long)g.head_stride, HEAD_DIM);
    if ((g.n_pages - 1.) * (double)g.page_stride + (double)g.page_rows * (double)g.row_stride + (Hkv - 1.) * (double)g.head_stride > 0x1p47)
        return fail(FQ_ERR_INVALID_ARGUMENT, "pages beyond 2^47 elements");
    p.k = (uint16_t*)g.k;
    p.v = (uint16_t*)g.v;
    p.row_stride = (int64_t)g.row_stride;
    p.head_stride = Hkv > 1 ? (int64_t)g.head_stride : HEAD_DIM;
    p.page_stride = g.n_pages > 1 ? (int64_t)g.page_stride : (int64_t)g.row_stride;
    return FQ_OK;
}

// What the calls over views and over pages share.
struct Call {
    AttnIo io;
    AttnMask mask;
    Partials part;
    AttnSeq seq[MAX_SEQ];
    int n_seq = 0, q_rows = 0;
    ViewUse use[MAX_SEQ];   // of views
    int n_views = 0;
    KvPages pages;
    uint32_t *waits = nullptr;
};

template <class Args>
fq_status run_tiles_t(const Plan& p, const Call& c, const AttnSeq* seq, const ViewUse* views, int n_views, cudaStream_t s) {
    Args* a = new (std::nothrow) Args;
    if (!a) return fail(FQ_ERR_OUT_OF_MEMORY, "host memory");
    auto run = [&]() -> fq_status {
        const AttnIo& io = c.io;
        a->io = io;
        a->c = std::fabs(score_factor(io.scale));
        a->negate = io.scale < 0.f;
        a->g_shift = 0;
        while (io.Hkv << a->g_shift < io.Hq) ++a->g_shift;
        a->inv_hkv = (uint32_t)(((1ull << 31) + io.Hkv - 1) / io.Hkv);
        a->waits.record = c.waits;
        a->part = c.part;
        a->mask = c.mask;
        a->pages = c.pages;
        std::copy(seq, seq + c.n_seq, a->seq);
        const uint64_t G = io.Hq / io.Hkv;
        const uint64_t dims[4] = {(uint64_t)HEAD_DIM, G, (uint64_t)io.Hkv, (uint64_t)c.q_rows};
        const uint64_t strides[4] = {2, HEAD_DIM * 2, G * HEAD_DIM * 2, (uint64_t)io.q_stride * 2};
        const uint32_t box[4] = {64, (uint32_t)G, 1, (uint32_t)(TILE_ROWS / G)};
        if (!encode_bf16_tiles(a->map_q, io.q, 4, dims, strides, box)) return fail(FQ_ERR_CUDA, "tensor map of q refused");
        if constexpr (Args::PAGED) {
            const KvPages& g = c.pages;
            const uint64_t pd[4] = {(uint64_t)HEAD_DIM, 1ull << g.shift, (uint64_t)io.Hkv, (uint64_t)g.n_pages};
            const uint64_t ps[4] = {2, (uint64_t)g.row_stride * 2, (uint64_t)g.head_stride * 2, (uint64_t)g.page_stride * 2};
            const uint32_t pb[4] = {64, (uint32_t)std::min(TILE_ROWS, 1 << g.shift), 1, 1};
            if (!encode_bf16_tiles(a->map_k[0], g.k, 4, pd, ps, pb) || !encode_bf16_tiles(a->map_v[0], g.v, 4, pd, ps, pb))
                return fail(FQ_ERR_CUDA, "tensor map of the pages refused");
        } else {
            for (int v = 0; v < n_views; ++v)
                if (views[v].used) {
                    TRY(encode_rows(a->map_k[v], a->map_v[v], views[v].rows, views[v].used, io.Hkv));
                    a->kv[v] = views[v].rows;
                }
        }
        constexpr size_t NE = Args::ENTRIES;
        for (size_t e0 = 0; e0 < p.tiles.size(); e0 += NE) {
            a->n_entries = (int)std::min(NE, p.tiles.size() - e0);
            std::copy(p.tiles.begin() + e0, p.tiles.begin() + e0 + a->n_entries, a->e);
            launch_tiles(*a, s);
            CK(cudaGetLastError());
        }
        return FQ_OK;
    };
    const fq_status st = run();
    delete a;
    return st;
}

fq_status run_tiles(const Plan& p, const Call& c, bool paged, cudaStream_t s) {
    if (p.tiles.empty()) return FQ_OK;
    const size_t n = p.tiles.size();
    if (paged) return n <= PagedArgsS::ENTRIES ? run_tiles_t<PagedArgsS>(p, c, c.seq, nullptr, 0, s) : run_tiles_t<PagedArgsL>(p, c, c.seq, nullptr, 0, s);
    auto one_view = [&](const AttnSeq* seq, const ViewUse* use) {
        return n <= WindowArgs1S::ENTRIES ? run_tiles_t<WindowArgs1S>(p, c, seq, use, 1, s) : run_tiles_t<WindowArgs1>(p, c, seq, use, 1, s);
    };
    if (c.n_views == 1) return one_view(c.seq, c.use);
    // maps for the views that the units read
    AttnSeq own[MAX_SEQ];
    ViewUse used[MAX_SEQ];
    std::copy(c.seq, c.seq + c.n_seq, own);
    bool read[MAX_SEQS] = {};
    for (const TileEntry& e : p.tiles) read[e.info & 127] = true;
    int n_views = 0;
    for (int i = 0; i < c.n_seq; ++i)
        if (read[i]) {
            used[n_views] = c.use[c.seq[i].view];
            own[i].view = n_views++;
        }
    if (n_views == 1) return one_view(own, used);
    return run_tiles_t<WindowArgsN>(p, c, own, used, n_views, s);
}

template <bool PAGED>
fq_status run_groups(const Plan& p, const Call& c, cudaStream_t s) {
    if (p.groups.empty()) return FQ_OK;
    WindowRowsArgs<PAGED> a;
    a.io = c.io;
    a.part = c.part;
    a.mask = c.mask;
    a.pages = c.pages;
    a.n_items = p.items;
    a.c = score_factor(c.io.scale);
    for (size_t g = 0; g < p.groups.size(); ++g) {
        a.g[g] = p.groups[g];
        if (PAGED) {
            a.kv[g].k = c.pages.k;
            a.kv[g].v = c.pages.v;
            a.kv[g].row_stride = c.pages.row_stride;
            a.kv[g].head_stride = c.pages.head_stride;
        } else {
            a.kv[g] = c.use[c.seq[p.groups[g].seq].view].rows;
        }
        for (int i = 0; i < chunks(p, g); ++i) a.group[p.groups[g].item0 + i] = (uint8_t)g;
    }
    launch_attn_window_rows(a, !p.tiles.empty(), s);
    CK(cudaGetLastError());
    return FQ_OK;
}

// After the checks of K and V: plan, the other checks, launches.
fq_status run_window(Call& c, bool paged, const void* q, uint64_t q_stride, uint64_t q_rows, const uint32_t* k_len, uint32_t Hq,
                     uint32_t Hkv, float scale, void* out, uint64_t out_stride, fq_dtype out_dtype, float* lse, void* workspace,
                     size_t workspace_bytes, void* stream) {
    try {
        Plan p;
        plan_prompt(p, (uint32_t)c.n_seq, c.seq, Hq / Hkv, Hkv, c.mask);
        TRY(attn_common(q, q_stride, Hq, Hkv, scale, out, out_stride, out_dtype, q_rows, *std::max_element(k_len, k_len + c.n_seq),
                        workspace, workspace_bytes, p.bytes(Hkv), c.io));
        if (reinterpret_cast<uintptr_t>(lse) & 3) return fail(FQ_ERR_INVALID_ARGUMENT, "lse not 4-byte aligned");
        if (q_rows == 0) return FQ_OK;
        c.io.lse = lse;
        c.q_rows = (int)q_rows;
        c.part = p.at(workspace, Hkv);
        TRY(prepare_device(&c.waits, &c.pages.bad));
        cudaStream_t s = (cudaStream_t)stream;
        TRY(run_tiles(p, c, paged, s));
        TRY(paged ? run_groups<true>(p, c, s) : run_groups<false>(p, c, s));
        return run_join(p, c.io, c.part, s);
    } catch (const std::bad_alloc&) {
        return fail(FQ_ERR_OUT_OF_MEMORY, "host memory");
    }
}

}  // namespace

extern "C" {

fq_status fq_attn_window(const void* q, uint64_t q_stride, const fq_kv_view* views, uint32_t n_views, uint32_t n_seq,
                         const uint32_t* q_len, const uint32_t* kv_row0, const uint32_t* k_len,
                         uint32_t num_attention_heads, uint32_t num_key_value_heads, uint32_t window, uint32_t sinks,
                         float scale, void* out, uint64_t out_stride, fq_dtype out_dtype, float* lse, void* workspace,
                         size_t workspace_bytes, void* stream) {
    const uint32_t Hq = num_attention_heads, Hkv = num_key_value_heads;
    TRY(check_heads(Hq, Hkv));
    TRY(check_count(n_seq));
    if (!q_len || !k_len || !views) return fail(FQ_ERR_INVALID_ARGUMENT, "null argument");
    if (n_views != 1 && n_views != n_seq) return fail(FQ_ERR_INVALID_ARGUMENT, "%u views for %u sequences", n_views, n_seq);
    Call c;
    uint64_t q_rows = 0;
    TRY(prompt_sequences(n_seq, q_len, kv_row0, k_len, views, n_views, Hkv, c.seq, c.use, &q_rows));
    c.n_seq = (int)n_seq;
    c.n_views = (int)n_views;
    c.mask = mask_of(window, sinks);
    return run_window(c, false, q, q_stride, q_rows, k_len, Hq, Hkv, scale, out, out_stride, out_dtype, lse, workspace,
                      workspace_bytes, stream);
}

fq_status fq_attn_window_workspace(uint32_t n_seq, const uint32_t* q_len, const uint32_t* k_len,
                                   uint32_t num_attention_heads, uint32_t num_key_value_heads, uint32_t window,
                                   uint32_t sinks, size_t* bytes) {
    TRY(check_heads(num_attention_heads, num_key_value_heads));
    TRY(check_count(n_seq));
    if (!q_len || !k_len || !bytes) return fail(FQ_ERR_INVALID_ARGUMENT, "null argument");
    AttnSeq seq[MAX_SEQ];
    uint64_t q_rows;
    TRY(prompt_sequences(n_seq, q_len, nullptr, k_len, nullptr, 0, num_key_value_heads, seq, nullptr, &q_rows));
    try {
        Plan p;
        plan_prompt(p, n_seq, seq, num_attention_heads / num_key_value_heads, num_key_value_heads, mask_of(window, sinks));
        *bytes = p.bytes(num_key_value_heads);
    } catch (const std::bad_alloc&) {
        return fail(FQ_ERR_OUT_OF_MEMORY, "host memory");
    }
    return FQ_OK;
}

fq_status fq_attn_paged(const void* q, uint64_t q_stride, const fq_kv_pages* pages, const int32_t* page_table,
                        uint64_t table_stride, uint32_t n_seq, const uint32_t* q_len, const uint32_t* k_len,
                        uint32_t num_attention_heads, uint32_t num_key_value_heads, uint32_t window, uint32_t sinks,
                        float scale, void* out, uint64_t out_stride, fq_dtype out_dtype, float* lse, void* workspace,
                        size_t workspace_bytes, void* stream) {
    const uint32_t Hq = num_attention_heads, Hkv = num_key_value_heads;
    TRY(check_heads(Hq, Hkv));
    TRY(check_count(n_seq));
    if (!q_len || !k_len) return fail(FQ_ERR_INVALID_ARGUMENT, "null argument");
    Call c;
    uint64_t q_rows = 0, rows[MAX_SEQ];
    TRY(prompt_sequences(n_seq, q_len, nullptr, k_len, nullptr, 1, Hkv, c.seq, nullptr, &q_rows));
    for (uint32_t s = 0; s < n_seq; ++s) rows[s] = k_len[s];
    TRY(check_pages(pages, page_table, table_stride, n_seq, rows, Hkv, c.pages));
    c.n_seq = (int)n_seq;
    c.mask = mask_of(window, sinks);
    return run_window(c, true, q, q_stride, q_rows, k_len, Hq, Hkv, scale, out, out_stride, out_dtype, lse, workspace,
                      workspace_bytes, stream);
}

fq_status fq_qk_norm_rope_paged(const float* qkv, uint64_t qkv_stride, uint32_t n_seq, const uint32_t* len,
                                const uint32_t* pos0, const fq_kv_pages* pages, const int32_t* page_table,
                                uint64_t table_stride, const uint32_t* kv_row0, uint32_t num_attention_heads,
                                uint32_t num_key_value_heads, const float* q_norm, const float* k_norm, float eps,
                                const float* rope, uint32_t rope_rows, void* q_out, uint64_t q_stride, void* stream) {
    const uint32_t Hq = num_attention_heads, Hkv = num_key_value_heads;
    TRY(check_heads(Hq, Hkv));
    TRY(check_count(n_seq));
    if (!len || !pos0 || !kv_row0) return fail(FQ_ERR_INVALID_ARGUMENT, "null argument");
    QkPagedArgs a;
    uint64_t rows = 0, ends[MAX_SEQ];
    for (uint32_t s = 0; s < n_seq; ++s) ends[s] = len[s] ? (uint64_t)kv_row0[s] + len[s] : 0;
    TRY(check_pages(pages, page_table, table_stride, n_seq, ends, Hkv, a.pages));
    TRY(qk_rows_common(
        qkv, qkv_stride, n_seq, len, pos0, kv_row0, Hq, Hkv, q_norm, k_norm, eps, rope, rope_rows, q_out, q_stride, a, &rows,
        [](uint32_t) { return FQ_OK; }));
    if (rows == 0) return FQ_OK;
    uint32_t* waits;
    TRY(prepare_device(&waits, &a.pages.bad));
    launch_qk_paged(a, (cudaStream_t)stream);
    CK(cudaGetLastError());
    return FQ_OK;
}

}  // extern "C"
