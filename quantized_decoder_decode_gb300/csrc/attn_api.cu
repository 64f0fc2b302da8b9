// Host side of the prompt and shared-prompt attention operators (fq_qk_norm_rope,
// fq_attn_prompt, fq_attn_shared): argument checks, then the launches.  Every check runs
// before anything is enqueued.

#include <atomic>
#include <mutex>

#include "attn_host.h"

using namespace fq;

namespace {

// Sequences 0 .. n_seq - 1: the tails (row groups), n_seq: all query rows over the prefix (tiles, or a
// row group when they are few).
void plan_shared(Plan& p, uint32_t n_seq, const AttnSeq* seq, uint32_t G, uint32_t Hkv) {
    const int tpt = TILE_ROWS / (int)G;
    const AttnSeq& all = seq[n_seq];
    const bool tiled = all.k_len && n_seq * G > (uint32_t)SMALL_ROWS, rows = all.k_len && !tiled;
    std::vector<Unit> units;
    if (tiled) add_units(units, all, (int)n_seq, (int)G, false);
    if (rows) add_group(p, all, (int)n_seq);
    bool tails = false;
    for (uint32_t s = 0; s < n_seq; ++s)
        if (seq[s].k_len) {
            add_group(p, seq[s], (int)s);
            tails = true;
        }
    const bool partial = all.k_len && tails;   // both: joined
    choose(p.even, units, seq, (int)G, (int)Hkv, partial, (float)all.k_len * Hkv * (HEAD_DIM * 4e-6f));
    emit(p, units, partial);
    plan_groups(p, Hkv, partial);
    // where the partial results of each sequence are
    std::vector<JoinEntry> e(n_seq);
    for (uint32_t s = 0; s < n_seq; ++s)
        e[s] = JoinEntry{(int)s, 1, (int)std::min<int64_t>((int64_t)all.k_len + seq[s].k_len, SEES_ALL), SEES_ALL,
                         0, 0, 0, 0, 0, 0, 0, 0, 0};
    for (const Unit& u : units)
        for (int i = 0; u.slot >= 0 && i < u.n_tok; ++i) {
            JoinEntry& j = e[u.tok0 + i];
            j.a0 = u.slot + i / tpt;
            j.nA = u.splits;
            j.a_step = u.single ? 1 : 2;
            j.a_row = i % tpt * (int)G;
        }
    for (size_t g = 0; g < p.groups.size(); ++g) {
        const RowGroup& r = p.groups[g];
        if (r.slot0 < 0) continue;
        if (p.groups[g].seq < (int)n_seq) {
            e[p.groups[g].seq].c0 = r.slot0;
            e[p.groups[g].seq].nC = chunks(p, g);
            continue;
        }
        for (uint32_t i = 0; i < n_seq; ++i) {
            e[i].b0 = r.slot0;
            e[i].nB = chunks(p, g);
            e[i].b_row = (int)(i * G);
        }
    }
    // (units and groups finish the others themselves; the join writes the zeros of those without a key)
    for (const JoinEntry& j : e)
        if (j.nA || j.nB || j.nC || j.k_len == 0) p.join.push_back(j);
}

// ---------------------------------------------------------------- launches

// The record of give-ups of one device that belongs to no model.  It only ever counts up, so that no check can
// take one away from another thread: every thread compares it with what it was at its own last check, and
// starts from the last value that any check has read.
struct Device {
    std::mutex mu;
    uint32_t* word = nullptr;          // (set once the kernels are prepared)
    std::atomic<uint32_t> read{0};
    std::atomic<uint32_t*> pages{nullptr};   // counts table entries without a page, in the same way
    std::atomic<uint32_t> pages_read{0};
};
constexpr int MAX_DEVICES = 64;
Device g_devices[MAX_DEVICES];
struct Seen {
    bool any = false;
    uint32_t count = 0, pages = 0;
};
thread_local Seen t_seen[MAX_DEVICES];

fq_status prepare_device(Device** out, Seen** seen) {
    int dev = 0;
    CK(cudaGetDevice(&dev));
    if (dev >= MAX_DEVICES) return fail(FQ_ERR_UNSUPPORTED, "device %d of %d at most", dev, MAX_DEVICES);
    Device& d = g_devices[dev];
    Seen& s = t_seen[dev];
    if (!s.any) s = Seen{true, d.read.load(), d.pages_read.load()};
    std::lock_guard<std::mutex> lk(d.mu);
    if (!d.word) {
        uint32_t* w = nullptr;
        CK(attn_tiles_prepare());
        CK(attn_rows_prepare());
        CK(attn_wait_word(&w));
        d.word = w;
    }
    *out = &d;
    *seen = &s;
    return FQ_OK;
}

template <class Args>
fq_status run_tiles_t(const Plan& p, const AttnIo& io, const AttnWaits& waits, const Partials& part, const AttnSeq* seq,
                      int n_seq, int q_rows, const ViewUse* views, int n_views, cudaStream_t s) {
    Device* dev;
    Seen* seen;
    TRY(prepare_device(&dev, &seen));
    Args* a = new (std::nothrow) Args;
    if (!a) return fail(FQ_ERR_OUT_OF_MEMORY, "host memory");
    auto run = [&]() -> fq_status {
        a->io = io;
        a->c = std::fabs(score_factor(io.scale));
        a->negate = io.scale < 0.f;
        a->g_shift = 0;
        while (io.Hkv << a->g_shift < io.Hq) ++a->g_shift;
        a->inv_hkv = (uint32_t)(((1ull << 31) + io.Hkv - 1) / io.Hkv);
        a->waits = waits;
        if (!waits.record) a->waits.record = dev->word;
        a->part = part;
        std::copy(seq, seq + n_seq, a->seq);
        const uint64_t G = io.Hq / io.Hkv;
        const uint64_t qs = (uint64_t)io.q_stride * 2;
        const uint64_t dims[4] = {(uint64_t)HEAD_DIM, G, (uint64_t)io.Hkv, (uint64_t)q_rows};
        const uint64_t strides[4] = {2, HEAD_DIM * 2, G * HEAD_DIM * 2, qs};
        const uint32_t box[4] = {64, (uint32_t)G, 1, (uint32_t)(TILE_ROWS / G)};
        if (!encode_bf16_tiles(a->map_q, io.q, 4, dims, strides, box)) return fail(FQ_ERR_CUDA, "tensor map of q refused");
        for (int v = 0; v < n_views; ++v)
            if (views[v].used) TRY(encode_rows(a->map_k[v], a->map_v[v], views[v].rows, views[v].used, io.Hkv));
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

fq_status run_tiles(const Plan& p, const AttnIo& io, const AttnWaits& waits, const Partials& part, const AttnSeq* seq,
                    int n_seq, int q_rows, const ViewUse* views, int n_views, cudaStream_t s) {
    if (p.tiles.empty()) return FQ_OK;
    const size_t n = p.tiles.size();
    // maps for the views that the units read
    AttnSeq own[MAX_SEQS];
    ViewUse used[MAX_SEQS];
    if (n_views > 1) {
        std::copy(seq, seq + n_seq, own);
        bool read[MAX_SEQS] = {};
        for (const TileEntry& e : p.tiles) read[e.info & 127] = true;
        n_views = 0;
        for (int i = 0; i < n_seq; ++i)
            if (read[i]) {
                used[n_views] = views[seq[i].view];
                own[i].view = n_views++;
            }
        seq = own;
        views = used;
    }
    auto run = n_views == 1 ? (n <= TileArgs1S::ENTRIES ? run_tiles_t<TileArgs1S> : run_tiles_t<TileArgs1>)
                            : (n <= TileArgsNS::ENTRIES && n_views <= TileArgsNS::VIEWS ? run_tiles_t<TileArgsNS> : run_tiles_t<TileArgsN>);
    return run(p, io, waits, part, seq, n_seq, q_rows, views, n_views, s);
}

// The row groups; rows[i]: the rows of view i.
fq_status run_groups(const Plan& p, const AttnIo& io, const Partials& part, const AttnSeq* seq, const ViewUse* views,
                     cudaStream_t s) {
    if (p.groups.empty()) return FQ_OK;
    Device* dev;
    Seen* seen;
    TRY(prepare_device(&dev, &seen));
    RowsArgs a;
    a.io = io;
    a.part = part;
    a.n_items = p.items;
    a.c = score_factor(io.scale);
    for (size_t g = 0; g < p.groups.size(); ++g) {
        a.g[g] = p.groups[g];
        a.kv[g] = views[seq[p.groups[g].seq].view].rows;
        for (int i = 0; i < chunks(p, g); ++i) a.group[p.groups[g].item0 + i] = (uint8_t)g;
    }
    launch_attn_rows(a, !p.tiles.empty(), s);
    CK(cudaGetLastError());
    return FQ_OK;
}

// The sequences of a shared call: the tails, then all query rows over the prefix.
fq_status shared_sequences(uint32_t n_seq, uint32_t prefix_len, const uint32_t* tail_len, AttnSeq* seq) {
    if (prefix_len > MAX_ROWS) return fail(FQ_ERR_INVALID_ARGUMENT, "more than 2^30 rows");
    int32_t view = 1;
    for (uint32_t s = 0; s < n_seq; ++s) {
        if (tail_len[s] > MAX_ROWS) return fail(FQ_ERR_INVALID_ARGUMENT, "more than 2^30 rows");
        seq[s] = AttnSeq{(int32_t)s, 1, 0, (int32_t)tail_len[s], SEES_ALL, tail_len[s] ? view++ : 0};
    }
    seq[n_seq] = AttnSeq{0, (int32_t)n_seq, 0, (int32_t)prefix_len, SEES_ALL, 0};
    return FQ_OK;
}

}  // namespace

namespace fq {

fq_status attn_prompt(const AttnWaits& waits, const void* q, uint64_t q_stride, const fq_kv_view* views, uint32_t n_views,
                      uint32_t n_seq, const uint32_t* q_len, const uint32_t* kv_row0, const uint32_t* k_len, uint32_t Hq,
                      uint32_t Hkv, float scale, void* out, uint64_t out_stride, fq_dtype out_dtype, void* workspace,
                      size_t workspace_bytes, void* stream) {
    TRY(check_heads(Hq, Hkv));
    TRY(check_count(n_seq));
    if (!q_len || !k_len || !views) return fail(FQ_ERR_INVALID_ARGUMENT, "null argument");
    if (n_views != 1 && n_views != n_seq) return fail(FQ_ERR_INVALID_ARGUMENT, "%u views for %u sequences", n_views, n_seq);
    AttnSeq seq[MAX_SEQ];
    ViewUse use[MAX_SEQ];
    uint64_t q_rows = 0;
    TRY(prompt_sequences(n_seq, q_len, kv_row0, k_len, views, n_views, Hkv, seq, use, &q_rows));
    try {
        Plan p;
        plan_prompt(p, n_seq, seq, Hq / Hkv, Hkv);
        AttnIo io;
        TRY(attn_common(q, q_stride, Hq, Hkv, scale, out, out_stride, out_dtype, q_rows, *std::max_element(k_len, k_len + n_seq),
                        workspace, workspace_bytes, p.bytes(Hkv), io));
        if (q_rows == 0) return FQ_OK;
        const Partials part = p.at(workspace, Hkv);
        cudaStream_t s = (cudaStream_t)stream;
        TRY(run_tiles(p, io, waits, part, seq, (int)n_seq, (int)q_rows, use, (int)n_views, s));
        TRY(run_groups(p, io, part, seq, use, s));
        return run_join(p, io, part, s);
    } catch (const std::bad_alloc&) {
        return fail(FQ_ERR_OUT_OF_MEMORY, "host memory");
    }
}

fq_status attn_shared(const AttnWaits& waits, const void* q, uint64_t q_stride, uint32_t n_seq, const fq_kv_view* prefix,
                      uint32_t prefix_len, const fq_kv_view* tails, const uint32_t* tail_len, uint32_t Hq, uint32_t Hkv,
                      float scale, void* out, uint64_t out_stride, fq_dtype out_dtype, void* workspace,
                      size_t workspace_bytes, void* stream) {
    TRY(check_heads(Hq, Hkv));
    TRY(check_count(n_seq));
    if (!tail_len) return fail(FQ_ERR_INVALID_ARGUMENT, "null argument");
    ViewUse use[MAX_SEQS];
    int n_views = 1;   // the prefix is view 0
    if (prefix_len) {
        if (!prefix) return fail(FQ_ERR_INVALID_ARGUMENT, "null prefix");
        TRY(check_view(*prefix, Hkv, 0, prefix_len, "prefix", 0));
        use[0].rows = rows_of(*prefix);
        use[0].used = prefix_len;
    }
    for (uint32_t s = 0; s < n_seq; ++s) {
        if (!tail_len[s]) continue;
        if (!tails) return fail(FQ_ERR_INVALID_ARGUMENT, "null tails");
        TRY(check_view(tails[s], Hkv, 0, tail_len[s], "tail", s));
        use[n_views].rows = rows_of(tails[s]);
        use[n_views++].used = tail_len[s];
    }
    AttnSeq seq[MAX_SEQS];
    TRY(shared_sequences(n_seq, prefix_len, tail_len, seq));
    try {
        Plan p;
        plan_shared(p, n_seq, seq, Hq / Hkv, Hkv);
        AttnIo io;
        TRY(attn_common(q, q_stride, Hq, Hkv, scale, out, out_stride, out_dtype, n_seq,
                        (uint64_t)prefix_len + *std::max_element(tail_len, tail_len + n_seq), workspace, workspace_bytes,
                        p.bytes(Hkv), io));
        const Partials part = p.at(workspace, Hkv);
        cudaStream_t s = (cudaStream_t)stream;
        TRY(run_tiles(p, io, waits, part, seq, (int)n_seq + 1, (int)n_seq, use, 1, s));
        TRY(run_groups(p, io, part, seq, use, s));
        return run_join(p, io, part, s);
    } catch (const std::bad_alloc&) {
        return fail(FQ_ERR_OUT_OF_MEMORY, "host memory");
    }
}

fq_status attn_device(int* dev, uint32_t** waits) {
    Device* d;
    Seen* seen;
    TRY(prepare_device(&d, &seen));
    *dev = (int)(d - g_devices);
    *waits = d->word;
    return FQ_OK;
}

void attn_set_page_word(int dev, uint32_t* word) { g_devices[dev].pages.store(word); }

fq_status attn_prompt_whole(const AttnWaits& waits, const void* q, const fq_kv_view* view, uint32_t q_len, uint32_t k_len,
                            uint32_t Hq, uint32_t Hkv, void* out, void* stream) {
    TRY(check_heads(Hq, Hkv));
    if (!view) return fail(FQ_ERR_INVALID_ARGUMENT, "null argument");
    if (q_len == 0) return fail(FQ_ERR_INVALID_SEQUENCE_LENGTH, "no query rows");
    AttnSeq seq[1];
    ViewUse use[1];
    uint64_t q_rows = 0;
    TRY(prompt_sequences(1, &q_len, nullptr, &k_len, view, 1, Hkv, seq, use, &q_rows));
    AttnIo io;
    TRY(attn_common(q, 0, Hq, Hkv, 1.f / std::sqrt((float)HEAD_DIM), out, 0, FQ_BF16, q_rows, k_len, nullptr, 0, 0, io));
    try {
        Plan p;
        std::vector<Unit> units;
        add_units(units, seq[0], 0, (int)(Hq / Hkv), false);
        emit(p, units, false);
        return run_tiles(p, io, waits, Partials(), seq, 1, (int)q_rows, use, 1, (cudaStream_t)stream);
    } catch (const std::bad_alloc&) {
        return fail(FQ_ERR_OUT_OF_MEMORY, "host memory");
    }
}

}  // namespace fq

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
    QkRowsArgs a;
    uint64_t rows = 0;
    TRY(qk_rows_common(qkv, qkv_stride, n_seq, len, pos0, kv_row0, Hq, Hkv, q_norm, k_norm, eps, rope, rope_rows, q_out, q_stride, a, &rows,
                       [&](uint32_t s) {
                           const fq_kv_view& v = views[n_views == 1 ? 0 : s];
                           a.kv[s] = rows_of(v);
                           return check_view(v, Hkv, kv_row0[s], len[s], "view", s);
                       }));
    if (rows == 0) return FQ_OK;
    TRY(check_apart(n_seq, len, views, n_views, kv_row0, Hkv));
    launch_qk_rows(a, (cudaStream_t)stream);
    CK(cudaGetLastError());
    return FQ_OK;
}

fq_status fq_attn_prompt_workspace(uint32_t n_seq, const uint32_t* q_len, const uint32_t* k_len,
                                   uint32_t num_attention_heads, uint32_t num_key_value_heads, size_t* bytes) {
    TRY(check_heads(num_attention_heads, num_key_value_heads));
    TRY(check_count(n_seq));
    if (!q_len || !k_len || !bytes) return fail(FQ_ERR_INVALID_ARGUMENT, "null argument");
    AttnSeq seq[MAX_SEQ];
    uint64_t q_rows;
    TRY(prompt_sequences(n_seq, q_len, nullptr, k_len, nullptr, 0, num_key_value_heads, seq, nullptr, &q_rows));
    try {
        Plan p;
        plan_prompt(p, n_seq, seq, num_attention_heads / num_key_value_heads, num_key_value_heads);
        *bytes = p.bytes(num_key_value_heads);
    } catch (const std::bad_alloc&) {
        return fail(FQ_ERR_OUT_OF_MEMORY, "host memory");
    }
    return FQ_OK;
}

fq_status fq_attn_shared_workspace(uint32_t n_seq, uint32_t prefix_len, const uint32_t* tail_len,
                                   uint32_t num_attention_heads, uint32_t num_key_value_heads, size_t* bytes) {
    TRY(check_heads(num_attention_heads, num_key_value_heads));
    TRY(check_count(n_seq));
    if (!tail_len || !bytes) return fail(FQ_ERR_INVALID_ARGUMENT, "null argument");
    AttnSeq seq[MAX_SEQS];
    TRY(shared_sequences(n_seq, prefix_len, tail_len, seq));
    try {
        Plan p;
        plan_shared(p, n_seq, seq, num_attention_heads / num_key_value_heads, num_key_value_heads);
        *bytes = p.bytes(num_key_value_heads);
    } catch (const std::bad_alloc&) {
        return fail(FQ_ERR_OUT_OF_MEMORY, "host memory");
    }
    return FQ_OK;
}

fq_status fq_attn_prompt(const void* q, uint64_t q_stride, const fq_kv_view* views, uint32_t n_views, uint32_t n_seq,
                         const uint32_t* q_len, const uint32_t* kv_row0, const uint32_t* k_len,
                         uint32_t num_attention_heads, uint32_t num_key_value_heads, float scale, void* out,
                         uint64_t out_stride, fq_dtype out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    return attn_prompt(AttnWaits(), q, q_stride, views, n_views, n_seq, q_len, kv_row0, k_len, num_attention_heads,
                       num_key_value_heads, scale, out, out_stride, out_dtype, workspace, workspace_bytes, stream);
}

fq_status fq_attn_shared(const void* q, uint64_t q_stride, uint32_t n_seq, const fq_kv_view* prefix,
                         uint32_t prefix_len, const fq_kv_view* tails, const uint32_t* tail_len,
                         uint32_t num_attention_heads, uint32_t num_key_value_heads, float scale, void* out,
                         uint64_t out_stride, fq_dtype out_dtype, void* workspace, size_t workspace_bytes, void* stream) {
    return attn_shared(AttnWaits(), q, q_stride, n_seq, prefix, prefix_len, tails, tail_len, num_attention_heads,
                       num_key_value_heads, scale, out, out_stride, out_dtype, workspace, workspace_bytes, stream);
}

fq_status fq_attn_check(void* stream) {
    Device* dev;
    Seen* seen;
    TRY(prepare_device(&dev, &seen));
    cudaStream_t s = (cudaStream_t)stream;
    uint32_t n = 0;
    CK(cudaMemcpyAsync(&n, dev->word, sizeof n, cudaMemcpyDeviceToHost, s));
    CK(cudaStreamSynchronize(s));
    const uint32_t before = seen->count;
    seen->count = n;
    dev->read.store(n);
    if (n != before)
        return fail(FQ_ERR_DEVICE_TIMEOUT, "a bounded device wait of an attention operator gave up (in %u thread blocks)", n - before);
    if (uint32_t* pages = dev->pages.load()) {
        CK(cudaMemcpyAsync(&n, pages, sizeof n, cudaMemcpyDeviceToHost, s));
        CK(cudaStreamSynchronize(s));
        const uint32_t bad = n - seen->pages;
        seen->pages = n;
        dev->pages_read.store(n);
        if (bad) return fail(FQ_ERR_INVALID_ARGUMENT, "a page table named pages outside the pool (met %u times)", bad);
    }
    return FQ_OK;
}

}  // extern "C"
