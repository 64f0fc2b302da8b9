// Host side of the operators on windows, pages and caches made shorter (fq_attn_window, fq_attn_paged,
// fq_qk_norm_rope_paged, fq_attn_key_weights, fq_kv_evict): argument checks, then the launches.  The checks and the work lists
// are those of attn_host.h.

#include <mutex>

#include "attn_host.h"
#include "cache_plan.h"

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
        CK(key_weights_prepare());
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
        if ((rows[s] + g.page_rows - 1) / g.page_rows > table_stride)
            return fail(FQ_ERR_KV_CACHE_OVERFLOW, "sequence %u: %llu rows need more than the table's %llu pages of %u", s,
                        (unsigned long long)rows[s], (unsigned long long)table_stride, g.page_rows);
        if (rows[s] > MAX_ROWS) return fail(FQ_ERR_INVALID_ARGUMENT, "more than 2^30 rows");
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

// Rows of a pool that share elements would be written twice in one call, or one over the other.  Pages, rows, heads and the
// way from K to V in the order of their strides: where each stride is at least as long as what the ones below it span (any
// nest of them; every layout that keeps K and V alike), no two rows meet.  Else the pages are looked at for every
// difference of rows and heads: 0.2 ms for 256 rows of 8 heads, 20 ms at most.
bool pool_rows_meet(const KvPages& p, int64_t Hkv) {
    const int64_t R = 1ll << p.shift, N = p.n_pages;
    const int64_t to_v = (int64_t)(reinterpret_cast<uintptr_t>(p.v) / 2) - (int64_t)(reinterpret_cast<uintptr_t>(p.k) / 2);
    struct Dim {
        int64_t stride, n;
    } d[4] = {{p.row_stride, R}, {p.head_stride, Hkv}, {p.page_stride, N}, {std::llabs(to_v), 2}};
    std::sort(d, d + 4, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
    int64_t span = HEAD_DIM;
    bool nest = true;
    for (const Dim& x : d) {
        if (x.n == 1) continue;
        nest = nest && x.stride >= span;
        span += (x.n - 1) * x.stride;
    }
    if (nest) return false;
    for (int64_t r = 1 - R; r < R; ++r)
        for (int64_t h = 1 - Hkv; h < Hkv; ++h) {
            const int64_t c = r * p.row_stride + h * p.head_stride;
            if (rows_near(c, p.page_stride, N, N, r == 0 && h == 0) || rows_near(to_v + c, p.page_stride, N, N, false)) return true;
        }
    return false;
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
            // (without rows no pool is asked for, and none is read)
            if (g.k && (!encode_bf16_tiles(a->map_k[0], g.k, 4, pd, ps, pb) || !encode_bf16_tiles(a->map_v[0], g.v, 4, pd, ps, pb)))
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
        a.pos[g] = p.pos[g];
    }
    a.n_groups = (int)p.groups.size();
    a.share = p.share;
    for (int i = 0, g = 0; i < p.items; ++i) {   // the first group that ends behind the part's beginning
        while (g + 1 < a.n_groups && a.pos[g + 1] <= i * a.share) ++g;
        a.group[i] = (uint8_t)g;
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
        p.even = true;
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

// ---------------------------------------------------------------- gathered weights

constexpr int KW_MAX_RUN = 4096;    // blocks of an entry, at most (no wait for a unit's end comes near its limit)
constexpr size_t KW_MAX_ENTRIES = 1 << 22;   // of a call
// What a thread block's part of the line is, at least, with keys that stay (512 tokens, 32 / 8 heads 11.1 us; 10: 12.9) and without.
constexpr int KW_MIN_SHARE = 6, KW_MIN_ROWS_SHARE = 3;
// What cutting entries costs: the units that begin with a cut, and the launch that joins their sums (100 tokens over 500 keys,
// 16 / 8 heads: 14 us cut, 7.6 whole).
constexpr int KW_CUT = 8;

int kw_grid(int64_t line, bool keys) {
    const int64_t least = keys ? KW_MIN_SHARE : KW_MIN_ROWS_SHARE;
    return (int)std::min<int64_t>(ATTN_SMS, (line + least - 1) / least);
}
int kw_cost(const KwEntry& e) { return kw_start(e.info & (KW_ROWS | KW_NONE)) + e.len; }
bool kw_keys(const KwEntry& e) { return !(e.info & (KW_ROWS | KW_NONE)); }

struct KwPlan {
    std::vector<KwEntry> e;         // those with the same keys KW_MAX_RUN query blocks apart
    int64_t line = 0;               // of a kv head
    bool keys = false;
    size_t bytes(uint32_t Hkv) const {   // (a launch of a part of the entries has as many thread blocks at most)
        const int grid = keys ? kw_grid(line * Hkv, true) : 0;
        return grid > 1 ? (size_t)grid * 2 * KW_KEY_TILES * TILE_ROWS * 4 : 0;
    }
};

// Up to 96 packed query rows (a block) stay while the keys pass by; of more, the query blocks pass by keys that stay.  20 tokens
// over 16000 keys, 32 / 8 heads (80 rows): 12.9 us, 15.9 with keys that stay; 48 tokens (192 rows): 20.5 and 17.5.
fq_status plan_key_weights(KwPlan& p, uint32_t n_seq, const AttnSeq* seq, uint32_t G, const AttnMask& m) {
    auto none = [&](int s, int j0, int j1) {
        for (const int most = KW_MAX_RUN * KW_REST; j0 < j1; j0 += most) {
            const int end = std::min(j1, j0 + most);
            p.e.push_back(KwEntry{s | KW_NONE, j0, end, 0, ceil_div(end - j0, KW_REST), 0});
        }
    };
    bool sorted = true;
    for (uint32_t i = 0; i < n_seq; ++i) {
        const AttnSeq& q = seq[i];
        if (q.k_len == 0) continue;
        const int s = (int)i, all = ceil_div(q.k_len, TILE_ROWS), blocks = ceil_div((int64_t)q.q_len * G, KW_BLOCK);
        const KeyTiles t = key_tiles(m, q.k_len, q.off, 0, q.q_len);
        if (t.n == 0) {
            none(s, 0, all);
            continue;
        }
        none(s, t.sinks, t.first);
        const int ends[2][2] = {{0, t.sinks}, {t.first, all}};
        for (auto& e : ends) {
            if (blocks <= 1) {
                for (int j = e[0]; j < e[1]; j += KW_MAX_RUN)
                    p.e.push_back(KwEntry{s | KW_ROWS, j, 0, 0, std::min(e[1] - j, KW_MAX_RUN), 0});
                continue;
            }
            for (int j = e[0]; j < e[1]; j += KW_KEY_TILES) {
                const int j1 = std::min(e[1], j + KW_KEY_TILES);
                // the tokens that see one of these keys
                const int64_t k0 = (int64_t)j * TILE_ROWS, k1 = std::min<int64_t>(q.k_len, (int64_t)j1 * TILE_ROWS) - 1;
                const int64_t first = std::max<int64_t>(0, k0 - q.off + 1);
                const int64_t last = k0 < m.sinks ? q.q_len - 1 : std::min<int64_t>(q.q_len - 1, k1 + m.window - q.off);
                if (last < first) {
                    none(s, j, j1);
                    continue;
                }
                const int b0 = (int)(first * G / KW_BLOCK), b1 = (int)((last * G + G - 1) / KW_BLOCK) + 1;
                int more = 0;
                for (int b = b0; b < b1; more = KW_MORE) {
                    const int end = std::min(b1, (b / KW_MAX_RUN + 1) * KW_MAX_RUN);
                    p.e.push_back(KwEntry{s | KW_KEYS | more, j, j1, b, end - b, 0});
                    sorted = sorted && end <= KW_MAX_RUN;
                    b = end;
                }
                p.keys = true;
                if (p.e.size() > KW_MAX_ENTRIES)
                    return fail(FQ_ERR_INVALID_ARGUMENT, "more than 2^22 units of work: fewer rows in a call");
            }
        }
    }
    for (const KwEntry& e : p.e) p.line += kw_cost(e);
    if (!sorted) std::stable_sort(p.e.begin(), p.e.end(), [](const KwEntry& a, const KwEntry& b) { return a.b0 / KW_MAX_RUN < b.b0 / KW_MAX_RUN; });
    return FQ_OK;
}

// What a call reads and writes of gathered weights: of sequence s and kv head h, the floats at lo + h * stride and behind.
struct WeightRows {
    int64_t lo = 0, stride = 0, n = 0;   // in floats; n of each head
};
// Do two sequences' weights share floats?
bool weights_meet(const WeightRows& a, const WeightRows& b, int64_t Hkv) {
    if (!a.n || !b.n) return false;
    const int64_t ea = a.lo + (Hkv - 1) * a.stride + a.n, eb = b.lo + (Hkv - 1) * b.stride + b.n;
    if (ea <= b.lo || eb <= a.lo) return false;
    if (Hkv == 1) return true;
    if (a.stride != b.stride) {   // heads in the order of their floats (each array's do not overlap)
        for (int64_t h = 0, g = 0; h < Hkv && g < Hkv;) {
            const int64_t x = a.lo + h * a.stride, y = b.lo + g * b.stride;
            if (x + a.n <= y) ++h;
            else if (y + b.n <= x) ++g;
            else return true;
        }
        return false;
    }
    const int64_t d = b.lo - a.lo;   // heads h of b and g of a meet where d + (h - g) stride is between -b.n and a.n
    const int64_t below = d >= 0 ? d / a.stride : -((-d + a.stride - 1) / a.stride);
    for (int64_t x = below; x <= below + 1; ++x) {
        const int64_t at = d - x * a.stride;
        if (x > -Hkv && x < Hkv && at < a.n && at + b.n > 0) return true;
    }
    return false;
}
fq_status check_weights(const fq_key_weights& w, uint32_t Hkv, uint64_t row0, uint64_t n, const char* what, uint32_t s, WeightRows& r) {
    if (n == 0) return FQ_OK;
    if (!w.w || (reinterpret_cast<uintptr_t>(w.w) & 3)) return fail(FQ_ERR_INVALID_ARGUMENT, "%s %u: null or misaligned weights", what, s);
    if (Hkv > 1 && (w.head_stride < row0 + n || w.head_stride > MAX_STRIDE))
        return fail(FQ_ERR_INVALID_ARGUMENT, "%s %u: head stride %llu (at least the rows used, %llu, at most 2^36)", what, s,
                    (unsigned long long)w.head_stride, (unsigned long long)(row0 + n));
    r.lo = (int64_t)(reinterpret_cast<uintptr_t>(w.w) / 4) + (int64_t)row0;
    r.stride = Hkv > 1 ? (int64_t)w.head_stride : 0;
    r.n = (int64_t)n;
    return FQ_OK;
}
fq_status check_weights_apart(const WeightRows* r, uint32_t n_seq, uint32_t Hkv) {
    // rows of one array (the rule): apart in one head, and all of them inside a head's stride
    WeightRows o[MAX_SEQ];
    int n = 0;
    bool same = true;
    for (uint32_t i = 0; i < n_seq; ++i)
        if (r[i].n) {
            o[n] = r[i];
            same = same && o[n].stride == o[0].stride;
            ++n;
        }
    if (n < 2) return FQ_OK;
    std::sort(o, o + n, [](const WeightRows& a, const WeightRows& b) { return a.lo < b.lo; });
    bool apart = same && (Hkv == 1 || o[n - 1].lo + o[n - 1].n - o[0].lo <= o[0].stride);
    for (int i = 0; i + 1 < n; ++i) apart = apart && o[i].lo + o[i].n <= o[i + 1].lo;
    if (apart) return FQ_OK;
    for (uint32_t i = 0; i < n_seq; ++i)
        for (uint32_t j = i + 1; j < n_seq; ++j)
            if (weights_meet(r[i], r[j], Hkv)) return fail(FQ_ERR_INVALID_ARGUMENT, "sequences %u and %u write the same weights", i, j);
    return FQ_OK;
}

// What a call adds to is read beside the sums that other thread blocks write: `before` and `after` of a sequence are the same
// weights, or lie apart; those of two sequences lie apart.
fq_status check_weights_read(const WeightRows* read, const WeightRows* written, uint32_t n_seq, uint32_t Hkv) {
    bool place = true;
    int64_t lo[2] = {INT64_MAX, INT64_MAX}, hi[2] = {INT64_MIN, INT64_MIN};
    auto same = [&](uint32_t i) { return read[i].lo == written[i].lo && read[i].stride == written[i].stride; };
    for (uint32_t i = 0; i < n_seq; ++i) {
        if (!read[i].n) continue;
        place = place && same(i);
        for (int k = 0; k < 2; ++k) {
            const WeightRows& r = k ? written[i] : read[i];
            lo[k] = std::min(lo[k], r.lo);
            hi[k] = std::max(hi[k], r.lo + (Hkv - 1) * r.stride + r.n);
        }
    }
    if (place || hi[0] <= lo[1] || hi[1] <= lo[0]) return FQ_OK;   // (in place: written weights lie apart)
    for (uint32_t i = 0; i < n_seq; ++i)
        for (uint32_t j = 0; j < n_seq; ++j)
            if (!(i == j && same(i)) && weights_meet(read[i], written[j], Hkv))
                return fail(FQ_ERR_INVALID_ARGUMENT, "sequence %u writes weights that sequence %u adds to", j, i);
    return FQ_OK;
}

template <class Args>
fq_status run_key_weights_t(const KwPlan& p, const AttnIo& io, const float* lse, const AttnMask& mask, uint32_t* waits, float* part,
                            const AttnSeq* seq, int n_seq, int q_rows, const ViewUse* views, const KeyWeights* w, int n_views,
                            cudaStream_t s) {
    Args* a = new (std::nothrow) Args;
    if (!a) return fail(FQ_ERR_OUT_OF_MEMORY, "host memory");
    auto run = [&]() -> fq_status {
        a->lse = lse;
        a->Hq = io.Hq;
        a->Hkv = io.Hkv;
        a->g_shift = 0;
        while (io.Hkv << a->g_shift < io.Hq) ++a->g_shift;
        a->c = score_factor(io.scale);
        a->mask = mask;
        a->waits.record = waits;
        a->part = part;
        std::copy(seq, seq + n_seq, a->seq);
        const uint64_t G = io.Hq / io.Hkv;
        const uint64_t dims[4] = {(uint64_t)HEAD_DIM, G, (uint64_t)io.Hkv, (uint64_t)q_rows};
        const uint64_t strides[4] = {2, HEAD_DIM * 2, G * HEAD_DIM * 2, (uint64_t)io.q_stride * 2};
        const uint32_t box[4] = {64, (uint32_t)G, 1, (uint32_t)(KW_BLOCK / G)};
        if (q_rows && !encode_bf16_tiles(a->map_q, io.q, 4, dims, strides, box)) return fail(FQ_ERR_CUDA, "tensor map of q refused");
        for (int v = 0; v < n_views; ++v) {
            a->w[v] = w[v];
            if (!views[v].used) continue;
            const uint64_t rs = (uint64_t)views[v].rows.row_stride * 2, hs = io.Hkv > 1 ? (uint64_t)views[v].rows.head_stride * 2 : rs;
            const uint64_t kd[3] = {(uint64_t)HEAD_DIM, views[v].used, (uint64_t)io.Hkv}, ks[3] = {2, rs, hs};
            const uint32_t kb[3] = {64, (uint32_t)TILE_ROWS, 1};
            if (!encode_bf16_tiles(a->map_k[v], views[v].rows.k, 3, kd, ks, kb)) return fail(FQ_ERR_CUDA, "tensor map of K refused");
        }
        constexpr size_t NE = Args::ENTRIES;
        for (size_t e0 = 0; e0 < p.e.size();) {
            bool keys = false, cuts = false;
            int longest = 0;
            a->total = a->n_entries = 0;
            for (; (size_t)a->n_entries < NE && e0 < p.e.size() && p.e[e0].b0 / KW_MAX_RUN == p.e[e0 - a->n_entries].b0 / KW_MAX_RUN; ++e0) {
                KwEntry& e = a->e[a->n_entries++];
                e = p.e[e0];
                e.pos = a->total;
                a->total += kw_cost(e);
                longest = std::max(longest, kw_cost(e));
                keys = keys || kw_keys(e);
                cuts = cuts || (kw_keys(e) && e.len > KW_WHOLE);
            }
            const int64_t line = (int64_t)a->total * io.Hkv;
            int grid = kw_grid(line, keys);
            a->share = (line + grid - 1) / grid;
            grid = (int)((line + a->share - 1) / a->share);
            const bool whole = keys && (int64_t)a->n_entries * io.Hkv <= ATTN_SMS && longest <= a->share + KW_CUT;
            if (whole) {   // a thread block each
                for (int i = 0; i < a->n_entries; ++i) a->e[i].pos = i * longest;
                a->share = longest;
                a->total = a->n_entries * longest;
                grid = a->n_entries * io.Hkv;
            }
            launch_key_weights(*a, grid, s);
            CK(cudaGetLastError());
            if (!cuts || whole || grid == 1) continue;
            launch_key_weights_join(*a, s);
            CK(cudaGetLastError());
        }
        return FQ_OK;
    };
    const fq_status st = run();
    delete a;
    return st;
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
        p.even = true;
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
    if (pool_rows_meet(a.pages, Hkv)) return fail(FQ_ERR_INVALID_ARGUMENT, "pages, rows or heads of the pool, or its K and V, share elements");
    uint32_t* waits;
    TRY(prepare_device(&waits, &a.pages.bad));
    launch_qk_paged(a, (cudaStream_t)stream);
    CK(cudaGetLastError());
    return FQ_OK;
}

fq_status fq_attn_key_weights_workspace(uint32_t n_seq, const uint32_t* q_len, const uint32_t* k_len,
                                        uint32_t num_attention_heads, uint32_t num_key_value_heads, uint32_t window,
                                        uint32_t sinks, size_t* bytes) {
    TRY(check_heads(num_attention_heads, num_key_value_heads));
    TRY(check_count(n_seq));
    if (!q_len || !k_len || !bytes) return fail(FQ_ERR_INVALID_ARGUMENT, "null argument");
    AttnSeq seq[MAX_SEQ];
    uint64_t q_rows;
    TRY(prompt_sequences(n_seq, q_len, nullptr, k_len, nullptr, 0, num_key_value_heads, seq, nullptr, &q_rows));
    try {
        KwPlan p;
        TRY(plan_key_weights(p, n_seq, seq, num_attention_heads / num_key_value_heads, mask_of(window, sinks)));
        *bytes = p.bytes(num_key_value_heads);
    } catch (const std::bad_alloc&) {
        return fail(FQ_ERR_OUT_OF_MEMORY, "host memory");
    }
    return FQ_OK;
}

fq_status fq_attn_key_weights(const void* q, uint64_t q_stride, const float* lse, const fq_kv_view* views, uint32_t n_views,
                              uint32_t n_seq, const uint32_t* q_len, const uint32_t* kv_row0, const uint32_t* k_len,
                              uint32_t num_attention_heads, uint32_t num_key_value_heads, uint32_t window, uint32_t sinks,
                              float scale, const fq_key_weights* before, const fq_key_weights* after, void* workspace,
                              size_t workspace_bytes, void* stream) {
    const uint32_t Hq = num_attention_heads, Hkv = num_key_value_heads;
    TRY(check_heads(Hq, Hkv));
    TRY(check_count(n_seq));
    if (!q_len || !k_len || !views || !after) return fail(FQ_ERR_INVALID_ARGUMENT, "null argument");
    if (n_views != 1 && n_views != n_seq) return fail(FQ_ERR_INVALID_ARGUMENT, "%u views for %u sequences", n_views, n_seq);
    AttnSeq seq[MAX_SEQ];
    ViewUse use[MAX_SEQ];
    fq_kv_view keys[MAX_SEQ];   // V is not looked at
    for (uint32_t v = 0; v < n_views; ++v) {
        keys[v] = views[v];
        keys[v].v = views[v].k;
    }
    uint64_t q_rows = 0;
    TRY(prompt_sequences(n_seq, q_len, kv_row0, k_len, keys, n_views, Hkv, seq, use, &q_rows));
    KeyWeights w[MAX_SEQ];
    WeightRows written[MAX_SEQ], read[MAX_SEQ];
    for (uint32_t s = 0; s < n_seq; ++s) {
        const uint32_t v = n_views == 1 ? 0 : s;
        TRY(check_weights(after[v], Hkv, (uint64_t)seq[s].k_row0, k_len[s], "after", s, written[s]));
        w[v].after = after[v].w;
        w[v].after_stride = written[s].stride;
        if (!before || !k_len[s]) continue;
        TRY(check_weights(before[v], Hkv, (uint64_t)seq[s].k_row0, k_len[s], "before", s, read[s]));
        w[v].before = before[v].w;
        w[v].before_stride = read[s].stride;
    }
    // (strides come from sequences with keys)
    for (uint32_t s = 0; s < n_seq; ++s)
        if (written[s].n) w[n_views == 1 ? 0 : s].after_stride = written[s].stride;
    TRY(check_weights_apart(written, n_seq, Hkv));
    if (before) TRY(check_weights_read(read, written, n_seq, Hkv));
    AttnMask mask = mask_of(window, sinks);
    try {
        KwPlan p;
        TRY(plan_key_weights(p, n_seq, seq, Hq / Hkv, mask));
        AttnIo io;
        // (no output of the rows' shape: q stands in for it)
        TRY(attn_common(q, q_stride, Hq, Hkv, scale, (void*)q, 0, FQ_BF16, q_rows, 0, workspace, workspace_bytes, p.bytes(Hkv), io));
        if (q_rows && (!lse || (reinterpret_cast<uintptr_t>(lse) & 3))) return fail(FQ_ERR_INVALID_ARGUMENT, "null or misaligned lse");
        if (p.e.empty()) return FQ_OK;
        uint32_t *waits, *bad;
        TRY(prepare_device(&waits, &bad));
        cudaStream_t s = (cudaStream_t)stream;
        const size_t n = p.e.size();
        auto run = n_views > 1 ? run_key_weights_t<KwArgsN>
                               : n <= KwArgs1S::ENTRIES ? run_key_weights_t<KwArgs1S>
                                                        : n <= KwArgs1M::ENTRIES ? run_key_weights_t<KwArgs1M> : run_key_weights_t<KwArgs1>;
        return run(p, io, lse, mask, waits, (float*)workspace, seq, (int)n_seq, (int)q_rows, use, w, (int)n_views, s);
    } catch (const std::bad_alloc&) {
        return fail(FQ_ERR_OUT_OF_MEMORY, "host memory");
    }
}

fq_status fq_kv_evict(const fq_kv_view* from, uint32_t n_from, const fq_key_weights* weights, uint32_t n_seq,
                      const uint32_t* kv_row0, const uint32_t* k_len, const uint32_t* keep, uint32_t sinks, uint32_t recent,
                      uint32_t num_key_value_heads, const fq_kv_view* to, uint32_t n_to, const fq_key_weights* to_weights,
                      const uint32_t* to_row0, int32_t* kept, void* stream) {
    const uint32_t Hkv = num_key_value_heads;
    TRY(check_count(n_seq));
    if (!Hkv || Hkv > MAX_HEADS) return fail(FQ_ERR_INVALID_ARGUMENT, "%u kv heads (1 to %u)", Hkv, MAX_HEADS);
    if (!from || !weights || !k_len || !keep || !to) return fail(FQ_ERR_INVALID_ARGUMENT, "null argument");
    if ((n_from != 1 && n_from != n_seq) || (n_to != 1 && n_to != n_seq))
        return fail(FQ_ERR_INVALID_ARGUMENT, "%u and %u views for %u sequences", n_from, n_to, n_seq);
    EvictArgs a;
    a.n_seq = (int)n_seq;
    a.Hkv = (int)Hkv;
    a.sinks = (int32_t)std::min<uint64_t>(sinks, MAX_ROWS);
    a.recent = (int32_t)std::min<uint64_t>(recent, MAX_ROWS);
    a.kept = kept;
    uint64_t r0 = 0, d0 = 0;
    int64_t total = 0, blocks = 0;
    uint32_t longest = 0, n[MAX_SEQ], to_rows[MAX_SEQ];
    WeightRows written[MAX_SEQ], read[MAX_SEQ];
    Span reads[2 * MAX_SEQ], writes[2 * MAX_SEQ];
    int n_reads = 0, n_writes = 0;
    for (uint32_t s = 0; s < n_seq; ++s) {
        if (k_len[s] > MAX_ROWS) return fail(FQ_ERR_INVALID_ARGUMENT, "more than 2^30 rows");
        n[s] = std::min(k_len[s], keep[s]);
        if (n[s] < k_len[s] && (uint64_t)sinks + recent > keep[s])
            return fail(FQ_ERR_INVALID_ARGUMENT, "sequence %u: %u rows do not hold %u first and %u recent ones", s, keep[s], sinks, recent);
        const uint32_t v = n_from == 1 ? 0 : s, t = n_to == 1 ? 0 : s;
        const uint64_t row = kv_row0 ? kv_row0[s] : n_from == 1 ? r0 : 0, at = to_row0 ? to_row0[s] : n_to == 1 ? d0 : 0;
        TRY(check_view(from[v], Hkv, row, k_len[s], "sequence", s));
        TRY(check_view(to[t], Hkv, at, n[s], "destination", s));
        TRY(check_weights(weights[v], Hkv, row, k_len[s], "sequence", s, read[s]));
        EvictSeq& e = a.s[s];
        e = EvictSeq{};
        e.len = (int32_t)k_len[s];
        e.n = (int32_t)n[s];
        e.kept0 = total;
        e.block0 = (int32_t)blocks;
        to_rows[s] = (uint32_t)at;
        if (n[s]) {
            if (to_weights) TRY(check_weights(to_weights[t], Hkv, at, n[s], "destination", s, written[s]));
            auto rows_at = [&](const fq_kv_view& g, uint64_t r) {
                KvRows x = rows_of(g);
                x.k += r * g.row_stride;
                x.v += r * g.row_stride;
                if (Hkv == 1) x.head_stride = 0;
                return x;
            };
            e.w = weights[v].w + row;
            e.w_stride = read[s].stride;
            e.w_to = to_weights ? to_weights[t].w + at : nullptr;
            e.w_to_stride = written[s].stride;
            e.from = rows_at(from[v], row);
            e.to = rows_at(to[t], at);
            reads[n_reads++] = span_of(from[v].k, from[v], (uint32_t)row, k_len[s], Hkv, s);
            reads[n_reads++] = span_of(from[v].v, from[v], (uint32_t)row, k_len[s], Hkv, s);
        }
        longest = std::max(longest, n[s] < k_len[s] ? k_len[s] : 0);
        total += (int64_t)n[s] * Hkv;
        blocks += (int64_t)ceil_div(n[s], EVICT_ROWS) * Hkv;
        if (blocks > 0x7FFFFFFF) return fail(FQ_ERR_INVALID_ARGUMENT, "2^36 rows of heads or more stay");
        r0 += k_len[s];
        d0 += n[s];
    }
    if (total == 0) return FQ_OK;
    if (!kept || (reinterpret_cast<uintptr_t>(kept) & 3)) return fail(FQ_ERR_INVALID_ARGUMENT, "null or misaligned kept");
    TRY(check_apart(n_seq, n, to, n_to, to_rows, Hkv));
    TRY(check_weights_apart(written, n_seq, Hkv));
    // A row (or weight) that is written while another block still has to read it: looked for where what is read and what is
    // written lie among one another at all.
    struct Extent {
        int64_t lo = INT64_MAX, hi = INT64_MIN;
        void add(int64_t l, int64_t h) {
            lo = std::min(lo, l);
            hi = std::max(hi, h);
        }
        bool meets(const Extent& e) const { return lo < e.hi && e.lo < hi; }
    } rows_read, rows_written, weights_read, weights_written;
    for (uint32_t s = 0; s < n_seq; ++s) {
        if (!n[s]) continue;
        const fq_kv_view& t = to[n_to == 1 ? 0 : s];
        for (void* p : {t.k, t.v}) writes[n_writes++] = span_of(p, t, to_rows[s], n[s], Hkv, s);
        for (int i : {1, 2}) {
            rows_read.add(reads[n_writes - i].lo, reads[n_writes - i].hi);
            rows_written.add(writes[n_writes - i].lo, writes[n_writes - i].hi);
        }
        const WeightRows &r = read[s], &w = written[s];
        weights_read.add(r.lo, r.lo + (Hkv - 1) * r.stride + r.n);
        if (w.n) weights_written.add(w.lo, w.lo + (Hkv - 1) * w.stride + w.n);
    }
    int64_t steps = 1 << 20;
    for (int j = 0; j < n_writes && rows_read.meets(rows_written); ++j)
        for (int i = 0; i < n_reads; ++i)
            if (rows_meet(reads[i], writes[j], Hkv, false, steps))
                return fail(FQ_ERR_INVALID_ARGUMENT, "sequence %u moves to rows that sequence %u is read from", writes[j].seq, reads[i].seq);
    for (uint32_t j = 0; j < n_seq && weights_read.meets(weights_written); ++j)
        for (uint32_t i = 0; i < n_seq; ++i)
            if (n[i] && weights_meet(read[i], written[j], Hkv))
                return fail(FQ_ERR_INVALID_ARGUMENT, "weights of sequence %u move to where those of sequence %u are read", j, i);
    launch_evict(a, (int)longest, (int)blocks, (cudaStream_t)stream);
    CK(cudaGetLastError());
    return FQ_OK;
}

}  // extern "C"
