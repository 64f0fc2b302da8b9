// Host side of the attention operators: argument checks and work lists that their entry points share
// (attn_api.cu, attn_cache_api.cu).  Every check runs before anything is enqueued.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdlib>
#include <new>
#include <vector>

#include "api_util.h"
#include "attn_plan.h"
#include "fq.h"

namespace fq {
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
    auto bad = [](uint64_t stride) { return stride % 8 || stride < HEAD_DIM || stride > MAX_STRIDE; };
    if (bad(v.row_stride) || (Hkv > 1 && bad(v.head_stride)))
        return fail(FQ_ERR_INVALID_ARGUMENT, "%s %u: strides (%llu, %llu) (multiples of 8 elements, %d to 2^36)", what, s,
                    (unsigned long long)v.row_stride, (unsigned long long)v.head_stride, HEAD_DIM);
    if (row0 + n > MAX_ROWS) return fail(FQ_ERR_INVALID_ARGUMENT, "%s %u: more than 2^30 rows", what, s);
    if ((double)(row0 + n) * (double)v.row_stride + (Hkv - 1.) * (double)v.head_stride > 0x1p47)
        return fail(FQ_ERR_INVALID_ARGUMENT, "%s %u: rows beyond 2^47 elements", what, s);
    return FQ_OK;
}

// The K or V rows that one sequence writes: element d of row r and head h is at lo + r * rs + h * hs + d.
struct Span {
    int64_t lo, hi, rs, hs, n;   // in elements; hi: behind the last
    uint32_t seq;
};
Span span_of(const void* p, const fq_kv_view& v, uint32_t row0, uint32_t n, uint32_t Hkv, uint32_t s) {
    const int64_t rs = (int64_t)v.row_stride, hs = Hkv > 1 ? (int64_t)v.head_stride : 0;
    const int64_t lo = (int64_t)(reinterpret_cast<uintptr_t>(p) / 2) + (int64_t)row0 * rs;
    return Span{lo, lo + (n - 1) * rs + (Hkv - 1) * hs + HEAD_DIM, rs, hs, n, s};
}

// Is there a row difference d in [-(n2 - 1), n1 - 1] with |c + d * rs| < HEAD_DIM?  (rs >= HEAD_DIM: one of the two
// that bring it to both sides of zero)
bool rows_near(int64_t c, int64_t rs, int64_t n1, int64_t n2, bool not_zero) {
    const int64_t below = c > 0 ? -((c + rs - 1) / rs) : -c / rs;
    for (int64_t d = below; d <= below + 1; ++d)
        if (d > -n2 && d < n1 && !(not_zero && d == 0) && std::llabs(c + d * rs) < HEAD_DIM) return true;
    return false;
}
// Do two of the spans' rows share elements (self: two different rows or heads of one span)?  `steps` is what the
// call's check may still take, some 10 ms in all; beyond that the
// answer is yes.
bool rows_meet(const Span& a, const Span& b, int64_t Hkv, bool self, int64_t& steps) {
    if (a.hi <= b.lo || b.hi <= a.lo) return false;
    const int64_t c = a.lo - b.lo;
    if (a.rs == b.rs && a.hs == b.hs) {
        // rows of one layout: heads far apart (a cache layer), or all heads of a row before the next row
        if (std::max(std::llabs(c - (b.n - 1) * a.rs), std::llabs(c + (a.n - 1) * a.rs)) <= a.hs - HEAD_DIM ||
            (c % a.rs == 0 && a.rs >= Hkv * a.hs))
            return rows_near(c, a.rs, a.n, b.n, self);
        if ((steps -= 2 * Hkv) < 0) return true;
        for (int64_t dh = 1 - Hkv; dh < Hkv; ++dh)
            if (rows_near(c + dh * a.hs, a.rs, a.n, b.n, self && dh == 0)) return true;
        return false;
    }
    // other strides: head by head where their extents overlap, row by row
    const int64_t la = (a.n - 1) * a.rs + HEAD_DIM, lb = (b.n - 1) * b.rs + HEAD_DIM;
    for (int64_t h = 0; h < Hkv; ++h)
        for (int64_t g = 0; g < Hkv; ++g) {
            const int64_t d = c + h * a.hs - g * b.hs;
            if (d + la <= 0 || d >= lb) {
                if (--steps < 0) return true;
                continue;
            }
            if ((steps -= a.n) < 0) return true;
            for (int64_t r = 0; r < a.n; ++r)
                if (rows_near(d + r * a.rs, b.rs, 1, b.n, false)) return true;
        }
    return false;
}

// Rows that are written twice in one call would race.
fq_status check_apart(uint32_t n_seq, const uint32_t* len, const fq_kv_view* views, uint32_t n_views, const uint32_t* row0,
                      uint32_t Hkv) {
    auto refuse = [](uint32_t a, uint32_t b) {
        return fail(FQ_ERR_INVALID_ARGUMENT, "sequences %u and %u write the same rows", std::min(a, b), std::max(a, b));
    };
    int64_t steps = 1 << 20;
    if (n_views == 1) {   // where all rows of the view are apart, only row ranges count
        struct Range {
            uint64_t r0, r1;
            uint32_t seq;
        } r[MAX_SEQ];
        int n = 0;
        for (uint32_t i = 0; i < n_seq; ++i)
            if (len[i]) r[n++] = Range{row0[i], (uint64_t)row0[i] + len[i], i};
        std::sort(r, r + n, [](const Range& a, const Range& b) { return a.r0 < b.r0; });
        for (int i = 0; i + 1 < n; ++i)
            if (r[i].r1 > r[i + 1].r0) return refuse(r[i].seq, r[i + 1].seq);
        const uint32_t first = (uint32_t)r[0].r0, rows = (uint32_t)(r[n - 1].r1 - r[0].r0);
        const Span k = span_of(views->k, *views, first, rows, Hkv, 0), v = span_of(views->v, *views, first, rows, Hkv, 0);
        if (!rows_meet(k, k, Hkv, true, steps) && !rows_meet(k, v, Hkv, false, steps)) return FQ_OK;
    }
    Span s[2 * MAX_SEQ];
    int n = 0;
    for (uint32_t i = 0; i < n_seq; ++i) {
        if (len[i] == 0) continue;
        const fq_kv_view& v = views[n_views == 1 ? 0 : i];
        s[n++] = span_of(v.k, v, row0[i], len[i], Hkv, i);
        s[n++] = span_of(v.v, v, row0[i], len[i], Hkv, i);
        if (rows_meet(s[n - 1], s[n - 1], Hkv, true, steps))
            return fail(FQ_ERR_INVALID_ARGUMENT, "sequence %u: rows or heads of its view overlap", i);
    }
    std::sort(s, s + n, [](const Span& a, const Span& b) { return a.lo < b.lo; });
    for (int i = 0; i < n; ++i)
        for (int j = i + 1; j < n && s[j].lo < s[i].hi; ++j)
            if (rows_meet(s[i], s[j], Hkv, false, steps)) return refuse(s[i].seq, s[j].seq);
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

// Times of attn_tiles.cuh in microseconds (measured at head_dim 128 on one GB300) that the choices
// below weigh: a key tile of a pair of query tiles and of a single one, a unit's own cost (what of
// its loads, joins and outputs nothing hides), what partial results cost more, and
// joining them (a launch, the reads); and reading K and V rows from memory.  (The choices are not
// sensitive to them: T_UNIT of 1.7 or 3.5, T_SINGLE of .78 or .92, T_JOIN of 5 give the same times;
// T_JOIN_MB of .2 splits too often: 64 sequences behind a shared prefix 38.5 -> 40.7 us.)
constexpr float T_PAIR = 1.45f, T_SINGLE = 0.85f, T_UNIT = 2.5f, T_PARTIAL = 0.5f, T_JOIN = 3.f,
                T_JOIN_MB = 0.4f, T_READ_MB = 0.16f;
constexpr int MIN_SPLIT = 4;   // key tiles of a split unit, at least
constexpr int64_t ROWS_CHUNK = 128;   // keys per chunk of attn_rows.cu, at least

struct Plan {
    std::vector<TileEntry> tiles;     // longest first
    std::vector<RowGroup> groups;
    std::vector<JoinEntry> join;
    int64_t a_slots = 0, b_slots = 0;   // partial blocks of 128 and of 8 rows
    int items = 0;                      // chunks of the groups; parts of their line
    std::vector<int64_t> pos;           // on the line: of the groups
    std::vector<int> parts;             // .. items that have a part of them
    int64_t share = 0;                  // .. an item's part
    bool even = false;                  // work in equal parts: groups on a line, long units beside many short ones cut as well

    size_t a_bytes(uint32_t Hkv) const { return (size_t)a_slots * Hkv * TILE_ROWS * HEAD_DIM * 4; }
    size_t b_bytes(uint32_t Hkv) const { return (size_t)b_slots * Hkv * SMALL_ROWS * HEAD_DIM * 4; }
    size_t bytes(uint32_t Hkv) const {   // values, then (m, l) pairs: 2 of every 128 + 2 floats
        return (a_bytes(Hkv) + b_bytes(Hkv)) / HEAD_DIM * (HEAD_DIM + 2);
    }
    Partials at(void* ws, uint32_t Hkv) const {
        Partials p;
        char* b = (char*)ws;
        p.a_o = (float*)b;
        p.b_o = (float*)(b += a_bytes(Hkv));
        p.a_ml = (float2*)(b += b_bytes(Hkv));
        p.b_ml = (float2*)(b + a_bytes(Hkv) / HEAD_DIM * 2);
        return p;
    }
};

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

struct Unit {
    int seq, tok0, n_tok, nt;   // tokens and key tiles
    bool single, small;
    int splits;                 // chosen
    int slot;                   // first partial block, or -1
    float cost(int S, bool partial) const {
        return (single ? T_SINGLE : T_PAIR) * ceil_div(nt, S) + T_UNIT + (partial ? T_PARTIAL : 0.f);
    }
};

// Units of sequence s: pairs of query tiles, or single ones.
void add_units(std::vector<Unit>& units, const AttnSeq& q, int s, int G, bool singles, const AttnMask& m = AttnMask()) {
    const int tpt = TILE_ROWS / G;
    const bool single = singles || q.q_len <= tpt;
    const int step = single ? tpt : 2 * tpt;
    for (int t = 0; t < q.q_len; t += step) {
        const int n_tok = std::min(step, q.q_len - t);
        const int nt = key_tiles(m, q.k_len, q.off, t, n_tok).n;
        units.push_back(Unit{s, t, n_tok, nt, single, q.q_len * (int64_t)G <= SMALL_ROWS, 1, -1});
    }
}

// Estimated time of the units with at most `cap` key tiles each (longer ones are split): the fullest CTA
// as the kernel deals them out, and the join.  Gives up (returns `best`) once it cannot be below that.
float estimate(const std::vector<Unit>& units, int cap, int G, int Hkv, bool partial, float best) {
    float total = 0.f, longest = 0.f, joined_mb = 0.f;
    struct Run { float cost; int n; };
    Run run[256];
    int n_runs = 0;
    int64_t n = 0;
    for (const Unit& u : units) {
        const int S = std::max(1, ceil_div(u.nt, cap));
        const float one = u.cost(S, partial || S > 1);
        total += S * one * Hkv;
        longest = std::max(longest, one);
        n += (int64_t)S * Hkv;
        if (partial || S > 1) joined_mb += S * (float)u.n_tok * G * Hkv * (HEAD_DIM * 4e-6f);
        if (n_runs && run[n_runs - 1].cost == one) run[n_runs - 1].n += S * Hkv;
        else if (n_runs < 256) run[n_runs++] = Run{one, S * Hkv};
    }
    const float join = joined_mb > 0.f ? T_JOIN + T_JOIN_MB * joined_mb : 0.f;
    float t = std::max(longest, total / ATTN_SMS) + join;
    if (t >= best || n <= ATTN_SMS || n > 6 * ATTN_SMS || n_runs == 256) return t;
    std::sort(run, run + n_runs, [](const Run& a, const Run& b) { return a.cost > b.cost; });
    float sum[ATTN_SMS] = {};
    int i = 0, dir = 1, c = 0;
    for (int k = 0; k < n_runs; ++k)
        for (int e = 0; e < run[k].n; ++e, ++i) {
            sum[c] += run[k].cost;
            if (c + dir < 0 || c + dir >= ATTN_SMS) dir = -dir;   // forth and back
            else c += dir;
        }
    return std::max(t, *std::max_element(sum, sum + ATTN_SMS) + join);
}

// Pairs of query tiles share their K and V tiles, single ones give shorter units, and units may be
// split along the keys.  Where there are few units per SM an estimate chooses:
//   2048 tokens, 16 / 8 heads            single tiles 23.8 us, pairs 32.6
//   333 tokens behind 7000, 32 / 4       pairs in three parts 45.2, single tiles in parts 48.3, whole
//                                        single tiles 54.3, whole pairs 91.3
//   10 prompts of 1 to 1187, 32 / 8      pairs 50.4, single tiles 50.8 (many units: pairs)
// From 456 units on (three per SM) pairs are taken whole.  That was measured with units of 1 to 10 key tiles
// alone; a long sequence beside many short ones loses by it (200 rows behind 30000, 32 / 8: beside 40 prompts of
// 20 tokens, split, 100 us; beside 60, whole, 315; floor 51).
// kv_mb: keys and values read from memory, which bounds what splitting can give.
//   ... which is why `even` cuts units that are longer than twice an SM's share into pieces of that share.
void choose(bool even, std::vector<Unit>& units, const AttnSeq* seq, int G, int Hkv, bool partial, float kv_mb, const AttnMask& m = AttnMask()) {
    if (units.empty()) return;
    int longest = 1;
    for (const Unit& u : units) longest = std::max(longest, u.nt);
    int cap = longest;
    if ((int64_t)units.size() * Hkv < 3 * ATTN_SMS) {
        std::vector<Unit> other;
        bool pairs = false, singles = false;
        for (const Unit& u : units) {
            if (u.tok0 == 0) add_units(other, seq[u.seq], u.seq, G, true, m);
            pairs |= !u.single;
        }
        const float floor = T_READ_MB * kv_mb;
        float best = 1e30f;
        for (int mode = 0; mode < (pairs ? 2 : 1); ++mode)
            for (int k = 1; k <= 64 && (k == 1 || longest >= MIN_SPLIT * k); k += k < 8 ? 1 : k / 4) {
                const int c = std::max(1, ceil_div(longest, k));
                const float t = std::max(floor, estimate(mode ? other : units, c, G, Hkv, partial, best));
                if (t < best) {
                    best = t;
                    cap = c;
                    singles = mode == 1;
                }
            }
        if (singles) units.swap(other);
    } else if (even) {
        int64_t all = 0;
        for (const Unit& u : units) all += (int64_t)u.nt * Hkv;
        const int share = (int)std::max<int64_t>(MIN_SPLIT, all / ATTN_SMS);
        if (longest > 2 * share) cap = share;
    }
    for (Unit& u : units) u.splits = std::max(1, ceil_div(u.nt, cap));
}

// Entries of the units, longest first; partial results where a unit is split or `partial` says so.
void emit(Plan& p, std::vector<Unit>& units, bool partial) {
    for (Unit& u : units) {
        uint32_t info = (uint32_t)u.seq | (u.single ? TILE_SINGLE : 0u) | (u.small ? TILE_SMALL : 0u);
        const int blocks = u.single ? 1 : 2;
        if (partial || u.splits > 1) {
            int64_t& n = u.small ? p.b_slots : p.a_slots;
            u.slot = (int)n;
            n += (int64_t)u.splits * blocks;
        }
        for (int i = 0; i < u.splits; ++i)
            p.tiles.push_back(TileEntry{u.tok0, info | (u.slot >= 0 ? (uint32_t)(u.slot + i * blocks + 1) << TILE_SLOT_SHIFT : 0u),
                                        (int)((int64_t)u.nt * i / u.splits), (int)((int64_t)u.nt * (i + 1) / u.splits)});
    }
    auto cost = [](const TileEntry& e) { return (e.j1 - e.j0) * (e.info & TILE_SINGLE ? T_SINGLE : T_PAIR); };
    std::stable_sort(p.tiles.begin(), p.tiles.end(), [&](const TileEntry& a, const TileEntry& b) { return cost(a) > cost(b); });
}

void add_group(Plan& p, const AttnSeq& q, int s, const AttnMask& m = AttnMask()) {
    p.groups.push_back(RowGroup{q.q_row0, q.q_len, q.k_row0, q.k_len, q.off, s, 0, 0, -1, key_span(m, q.k_len, q.off, q.q_len).n});
}

// An item's part of the line, at least, beside tiles, which leave fewer SMs (seven tokens and a chunk of 333 25.9 us, 27.0 with the 192
// of rows alone).
constexpr int64_t ROWS_BESIDE = 288;

// Lays the groups on a line and cuts it into equal parts, whose CTAs run all at once.
void plan_line(Plan& p, uint32_t Hkv, bool tiled) {
    int64_t line = 0;
    for (auto& g : p.groups) {
        p.pos.push_back(line);
        line += rows_line(g.keys);
    }
    const int64_t items = std::max<int64_t>(1, ROWS_CTAS / Hkv);
    p.share = std::max<int64_t>(tiled ? ROWS_BESIDE : ROWS_CHUNK + ROWS_START, (line + items - 1) / items);
    p.items = ceil_div(line, p.share);
    for (size_t i = 0; i < p.groups.size(); ++i) {
        RowGroup& g = p.groups[i];
        const int64_t first = p.pos[i] + ROWS_START;
        int last;
        rows_items(p.share, first, g.keys, g.item0, last);
        p.parts.push_back(last - g.item0 + 1);
        if (p.parts[i] > 1) {
            g.slot0 = (int)p.b_slots;
            p.b_slots += p.parts[i];
        }
    }
}

// Chunks the keys of the groups: the shortest chunks whose CTAs still run all at once, the longest chunks
// first (behind tiles, CTAs start as SMs become free).  Chosen at 16 sequences, 32 / 8 heads, 512 to 4096 keys (38 us
// cold, floor 22; 48: 96, floor 67; 64: 114, floor 89); where the sequences alone fill a wave the longest is hardly
// split any more (55 over 500 keys and one over 30000: 268 us, floor 35; 63 and one: 513), unlike on a line.
void plan_groups(Plan& p, uint32_t Hkv, bool partial) {
    auto ctas = [&](int64_t per) {
        int64_t n = 0;
        for (auto& g : p.groups) n += std::max(1, ceil_div(g.keys, per));
        return n * Hkv;
    };
    int64_t keys = 0, longest = 0;
    for (auto& g : p.groups) {
        keys += g.keys;
        longest = std::max<int64_t>(longest, g.keys);
    }
    int64_t per = std::max(ROWS_CHUNK, (keys * Hkv + ROWS_CTAS - 1) / ROWS_CTAS / 64 * 64);
    while (per < longest && ctas(per) > ROWS_CTAS) per += std::max<int64_t>(64, per / 32 / 64 * 64);
    for (auto& g : p.groups) {
        const int splits = std::max(1, ceil_div(g.keys, per));
        g.chunk = std::max(64, ceil_div(ceil_div(g.keys, splits), 64) * 64);
    }
    // longest chunks first
    std::stable_sort(p.groups.begin(), p.groups.end(), [](const RowGroup& a, const RowGroup& b) {
        return std::min(a.chunk, a.keys) > std::min(b.chunk, b.keys);
    });
    for (auto& g : p.groups) {
        const int n = std::max(1, ceil_div(g.keys, g.chunk));
        g.item0 = p.items;
        p.items += n;
        if (partial || n > 1) {
            g.slot0 = (int)p.b_slots;
            p.b_slots += n;
        }
    }
}
int chunks(const Plan& p, size_t g) {
    if (p.even) return p.parts[g];
    return (g + 1 < p.groups.size() ? p.groups[g + 1].item0 : p.items) - p.groups[g].item0;
}

void plan_prompt(Plan& p, uint32_t n_seq, const AttnSeq* seq, uint32_t G, uint32_t Hkv, const AttnMask& m = AttnMask()) {
    const int tpt = TILE_ROWS / (int)G;
    // Few rows go to attn_rows.cu (16 tokens over 512 to 4097 keys: 30.8 us, as units of tiles 37.1), but
    // for short sequences beside others that need tiles, where a unit more costs less than a launch more
    // (one token beside nine prompts: 50.5 us, with a launch of its own 51.2; the limit of 1024 keys is not
    // measured).
    bool tiled = false;
    for (uint32_t s = 0; s < n_seq; ++s) tiled |= (int64_t)seq[s].q_len * G > SMALL_ROWS;
    std::vector<Unit> units;
    float kv_mb = 0.f;
    for (uint32_t s = 0; s < n_seq; ++s) {
        if (seq[s].q_len == 0) continue;
        if ((int64_t)seq[s].q_len * G > SMALL_ROWS || (tiled && seq[s].k_len <= 1024)) {
            add_units(units, seq[s], (int)s, (int)G, false, m);
            kv_mb += (float)key_span(m, seq[s].k_len, seq[s].off, seq[s].q_len).n * Hkv * (HEAD_DIM * 4e-6f);
        } else {
            add_group(p, seq[s], (int)s, m);
        }
    }
    if (p.even) plan_line(p, Hkv, tiled);
    else plan_groups(p, Hkv, false);
    for (size_t g = 0; g < p.groups.size(); ++g) {
        const RowGroup& r = p.groups[g];
        if (r.slot0 >= 0) p.join.push_back(JoinEntry{r.q_row0, r.n_tok, r.k_len, r.off, 0, 0, 0, 0, r.slot0, chunks(p, g), 0, 0, 0});
    }
    choose(p.even, units, seq, (int)G, (int)Hkv, false, kv_mb, m);
    emit(p, units, false);
    for (const Unit& u : units) {
        if (u.slot < 0) continue;
        const AttnSeq& q = seq[u.seq];
        const int blocks = u.single ? 1 : 2;
        for (int b = 0; b < blocks && b * tpt < u.n_tok; ++b) {
            JoinEntry e{q.q_row0 + u.tok0 + b * tpt, std::min(tpt, u.n_tok - b * tpt), q.k_len, q.off + u.tok0 + b * tpt,
                        0, 0, 0, 0, 0, 0, 0, 0, 0};
            if (u.small) {
                e.b0 = u.slot;
                e.nB = u.splits;
            } else {
                e.a0 = u.slot + b;
                e.nA = u.splits;
                e.a_step = blocks;
            }
            p.join.push_back(e);
        }
    }
}

fq_status encode_rows(void* map_k, void* map_v, const KvRows& r, uint64_t rows, int Hkv) {
    const uint64_t rs = (uint64_t)r.row_stride * 2, hs = Hkv > 1 ? (uint64_t)r.head_stride * 2 : rs;
    const uint64_t dims[3] = {(uint64_t)HEAD_DIM, rows, (uint64_t)Hkv}, strides[3] = {2, rs, hs};
    const uint32_t box[3] = {64, (uint32_t)TILE_ROWS, 1};
    if (!encode_bf16_tiles(map_k, r.k, 3, dims, strides, box) || !encode_bf16_tiles(map_v, r.v, 3, dims, strides, box))
        return fail(FQ_ERR_CUDA, "tensor map of K or V refused");
    return FQ_OK;
}

// scale log2(e).  For a scale of 0 the smallest number: scores that are finite weigh the same, and a masked one
// (-inf) still weighs nothing.
float score_factor(float scale) {
    return std::copysign(std::max(std::fabs(scale) * 1.4426950408889634f, FLT_TRUE_MIN), scale);
}

struct ViewUse {
    KvRows rows;
    uint64_t used = 0;   // rows it is read up to
};

template <class Args>
fq_status run_join_t(const Plan& p, const AttnIo& io, const Partials& part, cudaStream_t s) {
    Args a;
    a.io = io;
    a.part = part;
    for (size_t e0 = 0; e0 < p.join.size(); e0 += Args::ENTRIES) {
        a.n_entries = (int)std::min<size_t>(Args::ENTRIES, p.join.size() - e0);
        a.max_tok = a.max_parts = 0;
        for (int i = 0; i < a.n_entries; ++i) {
            a.e[i] = p.join[e0 + i];
            a.max_tok = std::max(a.max_tok, a.e[i].n_tok);
            a.max_parts = std::max(a.max_parts, a.e[i].nA + a.e[i].nB + a.e[i].nC);
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
                      uint64_t out_stride, fq_dtype out_dtype, uint64_t q_rows, uint64_t max_keys, void* ws, size_t ws_bytes,
                      size_t need, AttnIo& io) {
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
    io.lift = 9.f;   // 2^8 above the reference maximum, and a bit for roundings
    while (max_keys > 1) {
        io.lift += 1.f;
        max_keys = (max_keys + 1) / 2;
    }
    return FQ_OK;
}

// Row ranges of the sequences of a prompt call; views may be null (lengths only).
fq_status prompt_sequences(uint32_t n_seq, const uint32_t* q_len, const uint32_t* kv_row0, const uint32_t* k_len,
                                  const fq_kv_view* views, uint32_t n_views, uint32_t Hkv, AttnSeq* seq, ViewUse* use,
                                  uint64_t* q_rows) {
    uint64_t qr = 0, kr = 0;
    for (uint32_t s = 0; s < n_seq; ++s) {
        if (q_len[s] > MAX_ROWS || k_len[s] > MAX_ROWS) return fail(FQ_ERR_INVALID_ARGUMENT, "more than 2^30 rows");
        uint64_t r0 = 0;
        const uint32_t w = n_views == 1 ? 0 : s;
        if (views) {
            r0 = kv_row0 ? kv_row0[s] : n_views == 1 ? kr : 0;
            TRY(check_view(views[w], Hkv, r0, k_len[s], "sequence", s));
            use[w].rows = rows_of(views[w]);
            if (k_len[s]) use[w].used = std::max(use[w].used, r0 + k_len[s]);
        }
        seq[s] = AttnSeq{(int32_t)qr, (int32_t)q_len[s], (int32_t)r0, (int32_t)k_len[s],
                         (int32_t)k_len[s] - (int32_t)q_len[s] + 1, (int32_t)w};
        qr += q_len[s];
        kr += k_len[s];
        if (qr > MAX_ROWS) return fail(FQ_ERR_INVALID_ARGUMENT, "more than 2^30 query rows");
    }
    *q_rows = qr;
    return FQ_OK;
}

// Checks and the common part of the arguments of QK-norm and rope; cache(s): the check of where sequence s's rows go.
template <class Cache>
fq_status qk_rows_common(const float* qkv, uint64_t qkv_stride, uint32_t n_seq, const uint32_t* len, const uint32_t* pos0,
                         const uint32_t* kv_row0, uint32_t Hq, uint32_t Hkv, const float* q_norm, const float* k_norm, float eps,
                         const float* rope, uint32_t rope_rows, void* q_out, uint64_t q_stride, QkRowsBase& a, uint64_t* n_rows,
                         Cache cache) {
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(FQ_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
    TRY(row_stride(qkv_stride, (uint64_t)(Hq + 2 * Hkv) * HEAD_DIM, 4, "qkv", &a.qkv_stride));
    TRY(row_stride(q_stride, (uint64_t)Hq * HEAD_DIM, 8, "q", &a.q_stride));
    uint64_t rows = 0;
    for (uint32_t s = 0; s < n_seq; ++s) {
        a.row0[s] = (int32_t)rows;
        a.pos0[s] = (int32_t)pos0[s];
        a.kv_row0[s] = (int32_t)kv_row0[s];
        if ((uint64_t)pos0[s] + len[s] > rope_rows)
            return fail(FQ_ERR_INVALID_SEQUENCE_LENGTH, "sequence %u: positions %u + %u > %u table rows", s, pos0[s], len[s], rope_rows);
        TRY(cache(s));
        rows += len[s];
        if (rows > MAX_ROWS) return fail(FQ_ERR_INVALID_ARGUMENT, "more than 2^30 rows");
    }
    *n_rows = rows;
    if (rows == 0) return FQ_OK;
    if (rows * (Hq + 2 * Hkv) >= 1ull << 32) return fail(FQ_ERR_INVALID_ARGUMENT, "2^32 heads of rows or more");
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
    return FQ_OK;
}

}  // namespace
}  // namespace fq
