// Host side of the prompt and shared-prompt attention operators (fq_qk_norm_rope,
// fq_attn_prompt, fq_attn_shared): argument checks, then the launches.  Every check runs
// before anything is enqueued.

#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <mutex>
#include <new>
#include <vector>

#include "api_util.h"
#include "attn_plan.h"
#include "fq.h"

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

// ---------------------------------------------------------------- work lists

// Times of attn_tiles.cu in microseconds (measured at head_dim 128 on one GB300) that the choices
// below weigh: a key tile of a pair of query tiles and of a single one, a unit's own cost (loads
// before its first scores, outputs), what a unit with partial results costs more, and joining
// them: a launch and the reads.
constexpr float T_PAIR = 1.45f, T_SINGLE = 0.85f, T_UNIT = 4.f, T_PARTIAL = 0.7f, T_JOIN = 3.f, T_JOIN_MB = 0.4f;
// .. and of attn_rows.cu: a CTA's own cost, and megabytes of keys and values per SM
constexpr float T_ROWS = 4.f, T_ROWS_MB = 26.f;
// Keys per chunk of attn_rows.cu at least
constexpr int64_t ROWS_CHUNK = 128;

struct Plan {
    std::vector<TileEntry> tiles;     // longest first
    std::vector<RowGroup> groups;
    std::vector<int> group_view;      // sequence whose view a group reads (-1: the prefix)
    std::vector<JoinEntry> join;
    int64_t tile_slots = 0, row_slots = 0;
    int row_items = 0;

    size_t tile_bytes(uint32_t Hkv) const { return (size_t)tile_slots * Hkv * TILE_ROWS * HEAD_DIM * 4; }
    size_t row_bytes(uint32_t Hkv) const { return (size_t)row_slots * Hkv * ROWS_MAX * HEAD_DIM * 4; }
    size_t bytes(uint32_t Hkv) const {   // values, then (m, l) pairs: 2 of every 128 + 2 floats
        return (tile_bytes(Hkv) + row_bytes(Hkv)) / HEAD_DIM * (HEAD_DIM + 2);
    }
    Partials at(void* ws, uint32_t Hkv) const {
        Partials p;
        char* b = (char*)ws;
        p.a_o = (float*)b;
        p.b_o = (float*)(b += tile_bytes(Hkv));
        p.a_ml = (float2*)(b += row_bytes(Hkv));
        p.b_ml = (float2*)(b + tile_bytes(Hkv) / HEAD_DIM * 2);
        return p;
    }
    int add_slots(int64_t& n, int64_t k) {
        n += k;
        return (int)(n - k);
    }
};

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// chunk the keys of the groups so that their CTAs fill the GPU about once
void plan_groups(Plan& p, uint32_t Hkv, bool partial) {
    auto ctas = [&](int64_t per) {
        int64_t n = 0;
        for (auto& g : p.groups) n += std::max(1, ceil_div(g.k_len, per));
        return n * Hkv;
    };
    int64_t keys = 0, longest = 0;
    for (auto& g : p.groups) {
        keys += g.k_len;
        longest = std::max<int64_t>(longest, g.k_len);
    }
    // the shortest chunks that still give one wave of CTAs
    int64_t per = std::max(ROWS_CHUNK, (keys * Hkv + ROWS_CTAS - 1) / ROWS_CTAS / 64 * 64);
    while (per < longest && ctas(per) > ROWS_CTAS) per += std::max<int64_t>(64, per / 32 / 64 * 64);
    for (auto& g : p.groups) {
        const int splits = std::max(1, ceil_div(g.k_len, per));
        g.chunk = std::max(64, ceil_div(ceil_div(g.k_len, splits), 64) * 64);
        const int n = std::max(1, ceil_div(g.k_len, g.chunk));
        g.item0 = p.row_items;
        p.row_items += n;
        g.slot0 = partial || n > 1 ? p.add_slots(p.row_slots, n) : -1;
    }
}

int splits_of(const Plan& p, size_t g) {
    return (g + 1 < p.groups.size() ? p.groups[g + 1].item0 : p.row_items) - p.groups[g].item0;
}

struct Tiles {
    int tok0, n_tok, nt;   // tokens and key tiles of a unit
    int seq;
    bool single;
};

// Units of sequence s: pairs of query tiles, or single ones.
void add_units(std::vector<Tiles>& units, const PromptSeq& q, int s, int tpt, bool singles) {
    const bool single = singles || q.q_len <= tpt;
    const int step = single ? tpt : 2 * tpt;
    for (int t = 0; t < q.q_len; t += step) {
        const int n_tok = std::min(step, q.q_len - t);
        units.push_back(Tiles{t, n_tok, ceil_div(std::max(0, std::min(q.k_len, t + n_tok - 1 + q.off)), TILE_ROWS), s, single});
    }
}

// Estimated time of the units with at most `cap` key tiles each (longer ones split): the longest
// unit, or as many average ones as the fullest CTA gets.
float estimate(const std::vector<Tiles>& units, int cap, int G, int Hkv) {
    float total = 0.f, longest = 0.f, joined_mb = 0.f;
    int64_t n = 0;
    for (const Tiles& u : units) {
        const int S = std::max(1, ceil_div(u.nt, cap));
        const float one = (u.single ? T_SINGLE : T_PAIR) * ceil_div(u.nt, S) + T_UNIT + (S > 1 ? T_PARTIAL : 0.f);
        total += S * one * Hkv;
        longest = std::max(longest, one);
        n += (int64_t)S * Hkv;
        if (S > 1) joined_mb += S * (float)u.n_tok * G * Hkv * (HEAD_DIM * 4e-6f);
    }
    const float even = total / n * ceil_div(n, ATTN_SMS);
    // many units per CTA even out
    return std::max(longest, n > 4 * ATTN_SMS ? total / ATTN_SMS : even) + (joined_mb > 0.f ? T_JOIN + T_JOIN_MB * joined_mb : 0.f);
}

void plan_prompt(Plan& p, uint32_t n_seq, const PromptSeq* seq, uint32_t G, uint32_t Hkv) {
    const int tpt = TILE_ROWS / (int)G;
    // Sequences of a few rows go to attn_rows.cu, but for short ones beside others that need tiles:
    // a unit more costs less than a launch more (1024 keys: 11 us of one CTA).
    bool tiled = false;
    for (uint32_t s = 0; s < n_seq; ++s) tiled |= (int64_t)seq[s].q_len * G > ROWS_MAX;
    std::vector<Tiles> units, other;
    for (uint32_t s = 0; s < n_seq; ++s) {
        const PromptSeq& q = seq[s];
        if (q.q_len == 0) continue;
        if ((int64_t)q.q_len * G > ROWS_MAX || (tiled && q.k_len <= 1024)) {
            add_units(units, q, (int)s, tpt, false);
            continue;
        }
        p.groups.push_back(RowGroup{q.q_row0, q.q_len, q.k_row0, q.k_len, q.off, 0, 0, -1});
        p.group_view.push_back((int)s);
    }
    plan_groups(p, Hkv, false);
    for (size_t g = 0; g < p.groups.size(); ++g) {
        const RowGroup& r = p.groups[g];
        if (r.slot0 >= 0)
            p.join.push_back(JoinEntry{r.q_row0, r.n_tok, r.k_len, r.off, 0, 0, 0, 0, r.slot0, splits_of(p, g), 0, 0, 0});
    }
    if (units.empty()) return;
    // Pairs of query tiles share their K and V tiles, single ones give shorter units, and units may
    // be split along the keys: with few units per SM the estimate chooses (2048 tokens, 16 / 8
    // heads: single tiles 19 us, pairs 27, split pairs 33).
    int longest = 0;
    for (const Tiles& u : units) longest = std::max(longest, u.nt);
    int cap = std::max(1, longest);
    if ((int64_t)units.size() * Hkv < 3 * ATTN_SMS) {
        for (const Tiles& u : units)
            if (u.tok0 == 0) add_units(other, seq[u.seq], u.seq, tpt, true);
        float best = 0.f;
        bool singles = false;
        for (int mode = 0; mode < 2; ++mode)
            for (int k = 1; k <= 24 && (k == 1 || longest / k >= 4); ++k) {
                const int c = std::max(1, ceil_div(longest, k));
                const float t = estimate(mode ? other : units, c, (int)G, (int)Hkv);
                if ((mode == 0 && k == 1) || t < best) {
                    best = t;
                    cap = c;
                    singles = mode == 1;
                }
            }
        if (singles) units.swap(other);
    }
    for (const Tiles& u : units) {
        const int S = std::max(1, ceil_div(u.nt, cap));
        const uint32_t info = (uint32_t)u.seq | (u.single ? TILE_SINGLE : 0u);
        if (S == 1) {
            p.tiles.push_back(TileEntry{u.tok0, info, 0, u.nt});
            continue;
        }
        const int blocks = u.single ? 1 : 2;
        const int slot = p.add_slots(p.tile_slots, (int64_t)S * blocks);
        for (int i = 0; i < S; ++i)
            p.tiles.push_back(TileEntry{u.tok0, info | (uint32_t)(slot + i * blocks + 1) << 8, (int)((int64_t)u.nt * i / S),
                                        (int)((int64_t)u.nt * (i + 1) / S)});
        const PromptSeq& q = seq[u.seq];
        for (int b = 0; b < blocks && b * tpt < u.n_tok; ++b)
            p.join.push_back(JoinEntry{q.q_row0 + u.tok0 + b * tpt, std::min(tpt, u.n_tok - b * tpt), q.k_len,
                                       q.off + u.tok0 + b * tpt, slot + b, S, blocks, 0, 0, 0, 0, 0, 0});
    }
    std::stable_sort(p.tiles.begin(), p.tiles.end(), [](const TileEntry& a, const TileEntry& b) {
        const float ca = (a.j1 - a.j0) * (a.info & TILE_SINGLE ? T_SINGLE : T_PAIR);
        return ca > (b.j1 - b.j0) * (b.info & TILE_SINGLE ? T_SINGLE : T_PAIR);
    });
}

// Splits of a shared prefix of nt key tiles (rows packed query rows, `units` units per kv head)
// while row groups with `tail_mb` of keys and values run on the SMs that the units leave.
int prefix_splits(int nt, int units, int rows, bool single, float tail_mb, int Hkv) {
    int best_S = 1;
    float best = 0.f;
    for (int S = 1; S <= nt; ++S) {
        const int ctas = units * Hkv * S;
        const float tiles = ((single ? T_SINGLE : T_PAIR) * ceil_div(nt, S) + T_UNIT + T_PARTIAL) * ceil_div(ctas, ATTN_SMS);
        float t = tiles;
        if (tail_mb > 0.f) {
            const int free = ATTN_SMS - std::min(ctas, ATTN_SMS);
            const float alone = T_ROWS + T_ROWS_MB * tail_mb / ATTN_SMS;
            t = tiles + alone;
            if (free > 0) t = std::min(t, std::max(tiles, T_ROWS + T_ROWS_MB * tail_mb / free));
        }
        t += T_JOIN + T_JOIN_MB * (S + (tail_mb > 0.f ? 1 : 0)) * rows * Hkv * (HEAD_DIM * 4e-6f);
        if (S == 1 || t < best) {
            best = t;
            best_S = S;
        }
        if (ctas >= 2 * ATTN_SMS) break;
    }
    return best_S;
}

void plan_shared(Plan& p, uint32_t n_seq, uint32_t prefix_len, const uint32_t* tail_len, uint32_t G, uint32_t Hkv) {
    const int tpt = TILE_ROWS / (int)G;
    const int P = (int)prefix_len;
    const bool tiled = P > 0 && n_seq * G > (uint32_t)ROWS_MAX;
    if (P > 0 && !tiled) {   // few rows: the prefix is a row group of all sequences
        p.groups.push_back(RowGroup{0, (int)n_seq, 0, P, SEES_ALL, 0, 0, -1});
        p.group_view.push_back(-1);
    }
    std::vector<int> tail_group(n_seq, -1);
    for (uint32_t s = 0; s < n_seq; ++s)
        if (tail_len[s]) {
            tail_group[s] = (int)p.groups.size();
            p.groups.push_back(RowGroup{(int)s, 1, 0, (int)tail_len[s], SEES_ALL, 0, 0, -1});
            p.group_view.push_back((int)s);
        }
    const bool tails = p.groups.size() > (P > 0 && !tiled ? 1u : 0u);
    plan_groups(p, Hkv, tiled || (P > 0 && tails));
    // the prefix as tiles: units (pairs of query tiles) x splits of the keys
    int S = 1, blocks = 1, units = 0, slot = 0;
    const bool single = (int)n_seq <= tpt;
    if (tiled) {
        units = ceil_div(n_seq, 2 * tpt);
        blocks = single ? 1 : 2;
        const int nt = ceil_div(P, TILE_ROWS);
        float mb = 0.f;
        for (uint32_t s = 0; s < n_seq; ++s) mb += (float)tail_len[s] * Hkv * (HEAD_DIM * 4e-6f);
        S = prefix_splits(nt, units, (int)(n_seq * G), single, mb, (int)Hkv);
        const bool partial = S > 1 || tails;
        if (partial) slot = p.add_slots(p.tile_slots, (int64_t)S * blocks * units);
        for (int u = 0; u < units; ++u)
            for (int i = 0; i < S; ++i)
                p.tiles.push_back(TileEntry{u * 2 * tpt,
                                            (single ? TILE_SINGLE : 0u) |
                                                (partial ? (uint32_t)(slot + (u * S + i) * blocks + 1) << 8 : 0u),
                                            (int)((int64_t)nt * i / S), (int)((int64_t)nt * (i + 1) / S)});
        if (!partial) return;
    } else if (!(P > 0 && tails)) {
        // finished by the row groups themselves, but for split groups and sequences without keys
        for (uint32_t s = 0; s < n_seq; ++s) {
            const int g = P > 0 ? 0 : tail_group[s];
            if (g >= 0 && p.groups[g].slot0 < 0) continue;
            JoinEntry e{(int)s, 1, g < 0 ? 0 : p.groups[g].k_len, SEES_ALL, 0, 0, 0, 0, 0, 0, 0, 0, 0};
            if (g >= 0) {
                e.b0 = p.groups[g].slot0;
                e.nB = splits_of(p, g);
                e.b_row = P > 0 ? (int)(s * G) : 0;
            }
            p.join.push_back(e);
        }
        return;
    }
    for (uint32_t s = 0; s < n_seq; ++s) {
        const int64_t keys = (int64_t)P + tail_len[s];
        JoinEntry e{(int)s, 1, (int)std::min<int64_t>(keys, SEES_ALL), SEES_ALL, 0, 0, 0, 0, 0, 0, 0, 0, 0};
        if (tiled) {
            const int b = (int)s / tpt;
            e.a0 = slot + (b / blocks) * S * blocks + b % blocks;
            e.nA = S;
            e.a_step = blocks;
            e.a_row = (int)(s % tpt) * (int)G;
        } else {
            e.b0 = p.groups[0].slot0;
            e.nB = splits_of(p, 0);
            e.b_row = (int)(s * G);
        }
        if (tail_group[s] >= 0) {
            e.c0 = p.groups[tail_group[s]].slot0;
            e.nC = splits_of(p, tail_group[s]);
        }
        p.join.push_back(e);
    }
}

// ---------------------------------------------------------------- launches

fq_status prepare_device() {
    static std::mutex mu;
    static bool done[64] = {};
    int dev = 0;
    CK(cudaGetDevice(&dev));
    std::lock_guard<std::mutex> lk(mu);
    if (dev < 64 && done[dev]) return FQ_OK;
    CK(attn_tiles_prepare());
    if (dev < 64) done[dev] = true;
    return FQ_OK;
}

fq_status encode_rows(void* map_k, void* map_v, const KvRows& r, uint64_t rows, int Hkv) {
    const uint64_t rs = (uint64_t)r.row_stride * 2, hs = Hkv > 1 ? (uint64_t)r.head_stride * 2 : rs;
    const uint64_t dims[3] = {(uint64_t)HEAD_DIM, rows, (uint64_t)Hkv}, strides[3] = {2, rs, hs};
    const uint32_t box[3] = {64, (uint32_t)TILE_ROWS, 1};
    if (!encode_bf16_tiles(map_k, r.k, 3, dims, strides, box) || !encode_bf16_tiles(map_v, r.v, 3, dims, strides, box))
        return fail(FQ_ERR_CUDA, "tensor map of K or V refused");
    return FQ_OK;
}

// views[s]: the rows of sequence s (views[0] for all when one is given), used: rows it is read up to
template <class Args>
fq_status run_tiles(const Plan& p, const AttnIo& io, const Partials& part, const PromptSeq* seq, int n_seq, int q_rows,
                    const KvRows* views, int n_views, const uint64_t* used, cudaStream_t s) {
    TRY(prepare_device());
    Args* a = new (std::nothrow) Args;
    if (!a) return fail(FQ_ERR_OUT_OF_MEMORY, "host memory");
    auto run = [&]() -> fq_status {
        a->io = io;
        a->c = std::max(std::fabs(io.scale) * 1.4426950408889634f, FLT_MIN);   // (a scale of 0: equal weights)
        a->negate = io.scale < 0.f;
        a->part = part;
        std::copy(seq, seq + n_seq, a->seq);
        const uint64_t G = io.Hq / io.Hkv;
        const uint64_t qs = (uint64_t)io.q_stride * 2;
        const uint64_t dims[4] = {(uint64_t)HEAD_DIM, G, (uint64_t)io.Hkv, (uint64_t)q_rows};
        const uint64_t strides[4] = {2, HEAD_DIM * 2, G * HEAD_DIM * 2, qs};
        const uint32_t box[4] = {64, (uint32_t)G, 1, (uint32_t)(TILE_ROWS / G)};
        if (!encode_bf16_tiles(a->map_q, io.q, 4, dims, strides, box)) return fail(FQ_ERR_CUDA, "tensor map of q refused");
        for (int v = 0; v < n_views; ++v)
            if (used[v]) TRY(encode_rows(a->map_k[v], a->map_v[v], views[v], used[v], io.Hkv));
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

fq_status run_one_view(const Plan& p, const AttnIo& io, const Partials& part, const PromptSeq* seq, int n_seq, int q_rows,
                       const KvRows* view, const uint64_t* used, cudaStream_t s) {
    return p.tiles.size() <= (size_t)TileArgsS::ENTRIES ? run_tiles<TileArgsS>(p, io, part, seq, n_seq, q_rows, view, 1, used, s)
                                                        : run_tiles<TileArgs1>(p, io, part, seq, n_seq, q_rows, view, 1, used, s);
}

fq_status run_groups(const Plan& p, const AttnIo& io, const Partials& part, const KvRows* views, const KvRows* prefix,
                     cudaStream_t s) {
    if (p.groups.empty()) return FQ_OK;
    RowsArgs a;
    a.io = io;
    a.c = io.scale * 1.4426950408889634f;
    a.part = part;
    a.n_groups = (int)p.groups.size();
    a.n_items = p.row_items;
    for (size_t g = 0; g < p.groups.size(); ++g) {
        a.g[g] = p.groups[g];
        std::fill(a.group + p.groups[g].item0, a.group + p.groups[g].item0 + splits_of(p, g), (uint8_t)g);
        a.kv[g] = p.group_view[g] < 0 ? *prefix : views[p.group_view[g]];
    }
    launch_attn_rows(a, !p.tiles.empty(), s);
    CK(cudaGetLastError());
    return FQ_OK;
}

template <class Args>
fq_status run_join_t(const Plan& p, const AttnIo& io, const Partials& part, cudaStream_t s) {
    Args a;
    a.io = io;
    a.part = part;
    for (size_t e0 = 0; e0 < p.join.size(); e0 += Args::ENTRIES) {
        a.n_entries = (int)std::min<size_t>(Args::ENTRIES, p.join.size() - e0);
        a.max_tok = 0;
        for (int i = 0; i < a.n_entries; ++i) {
            a.e[i] = p.join[e0 + i];
            a.max_tok = std::max(a.max_tok, a.e[i].n_tok);
        }
        // (a second launch waits for the first, which waits for the partial results)
        launch_attn_join(a, s);
        CK(cudaGetLastError());
    }
    return FQ_OK;
}

fq_status run_join(const Plan& p, const AttnIo& io, const Partials& part, cudaStream_t s) {
    if (p.join.empty()) return FQ_OK;
    return p.join.size() <= (size_t)JoinArgsS::ENTRIES ? run_join_t<JoinArgsS>(p, io, part, s) : run_join_t<JoinArgsL>(p, io, part, s);
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
        if (need > ws_bytes || (need && (!ws || (reinterpret_cast<uintptr_t>(ws) & 31))))
            return fail(FQ_ERR_INVALID_ARGUMENT, "workspace of %zu bytes, 32-byte aligned, needed (%zu given)", need, ws_bytes);
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

// Row ranges of the sequences of a prompt call; views may be null (lengths only).
static fq_status prompt_sequences(uint32_t n_seq, const uint32_t* q_len, const uint32_t* kv_row0, const uint32_t* k_len,
                                  const fq_kv_view* views, uint32_t n_views, uint32_t Hkv, PromptSeq* seq, KvRows* kv,
                                  uint64_t* used, uint64_t* q_rows) {
    uint64_t qr = 0, kr = 0;
    for (uint32_t s = 0; s < n_seq; ++s) {
        if (q_len[s] > MAX_ROWS || k_len[s] > MAX_ROWS) return fail(FQ_ERR_INVALID_ARGUMENT, "more than 2^30 rows");
        uint64_t r0 = 0;
        if (views) {
            const uint32_t w = n_views == 1 ? 0 : s;
            r0 = kv_row0 ? kv_row0[s] : n_views == 1 ? kr : 0;
            TRY(check_view(views[w], Hkv, r0, k_len[s], "sequence", s));
            kv[s] = rows_of(views[w]);
            if (s == w) used[w] = 0;
            if (k_len[s]) used[w] = std::max(used[w], r0 + k_len[s]);
        }
        seq[s] = PromptSeq{(int32_t)qr, (int32_t)q_len[s], (int32_t)r0, (int32_t)k_len[s],
                           (int32_t)k_len[s] - (int32_t)q_len[s] + 1};
        qr += q_len[s];
        kr += k_len[s];
        if (qr > MAX_ROWS) return fail(FQ_ERR_INVALID_ARGUMENT, "more than 2^30 query rows");
    }
    *q_rows = qr;
    return FQ_OK;
}

fq_status fq_attn_prompt_workspace(uint32_t n_seq, const uint32_t* q_len, const uint32_t* k_len,
                                   uint32_t num_attention_heads, uint32_t num_key_value_heads, size_t* bytes) {
    TRY(check_heads(num_attention_heads, num_key_value_heads));
    TRY(check_count(n_seq));
    if (!q_len || !k_len || !bytes) return fail(FQ_ERR_INVALID_ARGUMENT, "null argument");
    PromptSeq seq[MAX_SEQ];
    uint64_t q_rows;
    TRY(prompt_sequences(n_seq, q_len, nullptr, k_len, nullptr, 0, num_key_value_heads, seq, nullptr, nullptr, &q_rows));
    try {
        Plan p;
        plan_prompt(p, n_seq, seq, num_attention_heads / num_key_value_heads, num_key_value_heads);
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
    const uint32_t Hq = num_attention_heads, Hkv = num_key_value_heads;
    TRY(check_heads(Hq, Hkv));
    TRY(check_count(n_seq));
    if (!q_len || !k_len || !views) return fail(FQ_ERR_INVALID_ARGUMENT, "null argument");
    if (n_views != 1 && n_views != n_seq) return fail(FQ_ERR_INVALID_ARGUMENT, "%u views for %u sequences", n_views, n_seq);
    PromptSeq seq[MAX_SEQ];
    KvRows kv[MAX_SEQ];
    uint64_t used[MAX_SEQ], q_rows = 0;
    TRY(prompt_sequences(n_seq, q_len, kv_row0, k_len, views, n_views, Hkv, seq, kv, used, &q_rows));
    try {
        Plan p;
        plan_prompt(p, n_seq, seq, Hq / Hkv, Hkv);
        AttnIo io;
        TRY(attn_common(q, q_stride, Hq, Hkv, scale, out, out_stride, out_dtype, q_rows, workspace, workspace_bytes,
                        p.bytes(Hkv), io));
        if (q_rows == 0) return FQ_OK;
        const Partials part = p.at(workspace, Hkv);
        cudaStream_t s = (cudaStream_t)stream;
        if (!p.tiles.empty())
            TRY(n_views == 1 ? run_one_view(p, io, part, seq, (int)n_seq, (int)q_rows, kv, used, s)
                             : run_tiles<TileArgsN>(p, io, part, seq, (int)n_seq, (int)q_rows, kv, (int)n_views, used, s));
        TRY(run_groups(p, io, part, kv, nullptr, s));
        return run_join(p, io, part, s);
    } catch (const std::bad_alloc&) {
        return fail(FQ_ERR_OUT_OF_MEMORY, "host memory");
    }
}

fq_status fq_attn_shared_workspace(uint32_t n_seq, uint32_t prefix_len, const uint32_t* tail_len,
                                   uint32_t num_attention_heads, uint32_t num_key_value_heads, size_t* bytes) {
    TRY(check_heads(num_attention_heads, num_key_value_heads));
    TRY(check_count(n_seq));
    if (!tail_len || !bytes) return fail(FQ_ERR_INVALID_ARGUMENT, "null argument");
    if (prefix_len > MAX_ROWS) return fail(FQ_ERR_INVALID_ARGUMENT, "more than 2^30 rows");
    for (uint32_t s = 0; s < n_seq; ++s)
        if (tail_len[s] > MAX_ROWS) return fail(FQ_ERR_INVALID_ARGUMENT, "more than 2^30 rows");
    try {
        Plan p;
        plan_shared(p, n_seq, prefix_len, tail_len, num_attention_heads / num_key_value_heads, num_key_value_heads);
        *bytes = p.bytes(num_key_value_heads);
    } catch (const std::bad_alloc&) {
        return fail(FQ_ERR_OUT_OF_MEMORY, "host memory");
    }
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
    KvRows first, kv[MAX_SEQ];
    if (prefix_len) {
        if (!prefix) return fail(FQ_ERR_INVALID_ARGUMENT, "null prefix");
        TRY(check_view(*prefix, Hkv, 0, prefix_len, "prefix", 0));
        first = rows_of(*prefix);
    }
    for (uint32_t s = 0; s < n_seq; ++s) {
        if (!tail_len[s]) continue;
        if (!tails) return fail(FQ_ERR_INVALID_ARGUMENT, "null tails");
        TRY(check_view(tails[s], Hkv, 0, tail_len[s], "tail", s));
        kv[s] = rows_of(tails[s]);
    }
    try {
        Plan p;
        plan_shared(p, n_seq, prefix_len, tail_len, Hq / Hkv, Hkv);
        AttnIo io;
        TRY(attn_common(q, q_stride, Hq, Hkv, scale, out, out_stride, out_dtype, n_seq, workspace, workspace_bytes,
                        p.bytes(Hkv), io));
        const Partials part = p.at(workspace, Hkv);
        cudaStream_t s = (cudaStream_t)stream;
        if (!p.tiles.empty()) {
            const PromptSeq all{0, (int32_t)n_seq, 0, (int32_t)prefix_len, SEES_ALL};
            const uint64_t used = prefix_len;
            TRY(run_one_view(p, io, part, &all, 1, (int)n_seq, &first, &used, s));
        }
        TRY(run_groups(p, io, part, kv, &first, s));
        return run_join(p, io, part, s);
    } catch (const std::bad_alloc&) {
        return fail(FQ_ERR_OUT_OF_MEMORY, "host memory");
    }
}

fq_status fq_attn_check(void* stream) {
    uint32_t n = 0;
    CK(attn_wait_record(&n, (cudaStream_t)stream));
    if (n) return fail(FQ_ERR_DEVICE_TIMEOUT, "a bounded device wait of an attention operator gave up (%u waits)", n);
    return FQ_OK;
}

}  // extern "C"
