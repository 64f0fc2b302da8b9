// Arguments of the prompt and shared-prompt attention operators' kernels, and their work lists, made on the host
// (attn_host.h) and passed by value to attn_tiles.cuh, attn_rows.cu and attn_join.cu.
//
// "Packed rows": a kv head's query rows are (token, head of its group) with the head running
// fastest, so G heads x tokens fill the 128 rows of a matrix product.
#pragma once

#include "fq.h"
#include "kernels.h"

namespace fq {

struct KvRows {                   // element d of row r of kv head h: [r * row_stride + h * head_stride + d]
    uint16_t *k = nullptr, *v = nullptr;
    int64_t row_stride = 0, head_stride = 0;
};

// K and V rows in pages: element d of row r of kv head h of page p is at [p * page_stride + r * row_stride +
// h * head_stride + d].  Row r of sequence s is row r % page_rows of page table[s * table_stride + r / page_rows].
struct KvPages {
    uint16_t *k = nullptr, *v = nullptr;
    int64_t page_stride = 0, row_stride = 0, head_stride = 0;
    const int32_t* table = nullptr;
    int64_t table_stride = 0;
    int32_t n_pages = 0, shift = 0;        // rows of a page: 2^shift, 16 to 256
    uint32_t* bad = nullptr;               // counts CTAs that met a table entry outside [0, n_pages): no row is read or written for it
};

// QK-norm + rope of packed rows, q -> q_out, k and v -> cache rows (qk_rows.cu)
struct QkRowsBase {
    const float* qkv;             // [rows][(Hq + 2 Hkv) * 128]
    int64_t qkv_stride;
    const float *q_norm, *k_norm; // [128]
    const float2* rope;           // [positions][64] (cos, sin)
    float eps;
    int Hq, Hkv, n_seq, rows;
    uint16_t* q_out;              // bf16 [rows][Hq * 128]
    int64_t q_stride;
    int32_t row0[MAX_SEQ], pos0[MAX_SEQ], kv_row0[MAX_SEQ];   // per sequence: first row, position, cache row
};
struct QkRowsArgs : QkRowsBase {
    static constexpr bool PAGED = false;
    KvRows kv[MAX_SEQ];
};
struct QkPagedArgs : QkRowsBase {
    static constexpr bool PAGED = true;
    KvPages pages;
};
void launch_qk_rows(const QkRowsArgs& a, cudaStream_t s);
void launch_qk_paged(const QkPagedArgs& a, cudaStream_t s);

struct AttnIo {
    const uint16_t* q;            // bf16 [rows][Hq][128]
    int64_t q_stride;
    void* out;                    // bf16 or f32 [rows][Hq][128]
    int64_t out_stride;
    int out_f32;
    int Hq, Hkv;
    float scale;
    float* lse = nullptr;         // f32 [rows][Hq]: log of the row's sum of exponentials, or null
    float lift;                   // softmax weights are held as 2^-lift of the usual ones: their sum over a row's keys
                                  // stays below 1, and sums of weight x value below the largest value
};
// tensor map over bf16 values of rank 3 or 4 (strides[0] is not read), 128-byte swizzle, zero
// fill outside
bool encode_bf16_tiles(void* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides_bytes,
                       const uint32_t* box);

constexpr int ATTN_SMS = 152;         // SMs that the work lists are made for
constexpr int TILE_ROWS = 128;        // packed rows of a query tile = keys of a key tile
constexpr int SMALL_ROWS = 8;         // packed rows of a row group, of the small partial results
constexpr int32_t SEES_ALL = 1 << 30; // AttnSeq::off of rows that see every key
constexpr int MAX_SEQS = MAX_SEQ + 1; // the sequences of a call, or tails and a prefix

// Query rows and the key rows of a view that they attend to: row i (token) sees keys
// [0, min(k_len, i + off)), off = k_len - q_len + 1 for causal sequences.
struct AttnSeq {
    int32_t q_row0, q_len, k_row0, k_len, off, view;
};

// What a row sees of the keys up to its own: the last `window` of them, and the first `sinks` of the sequence.
struct AttnMask {
    int32_t window = 1 << 30, sinks = 0;   // (no sequence has more than 2^30 keys)
};

// The key tiles that token rows [tok, tok + n_tok) of a sequence look at: [0, sinks) and [first, ..), n in all.
// They are counted through: tile number v is key tile at(v).
struct KeyTiles {
    int32_t sinks = 0, first = 0, n = 0;
    FQ_HD int32_t at(int32_t v) const { return v < sinks ? v : v - sinks + first; }
    // tiles up to the one with the last of `keys` keys (which the window of the first row reaches)
    FQ_HD int32_t up_to(int32_t keys) const {
        const int32_t end = (keys + TILE_ROWS - 1) / TILE_ROWS;
        return keys <= 0 ? 0 : sinks + (end > first ? end - first : 0);
    }
};
FQ_HD inline KeyTiles key_tiles(const AttnMask& m, int32_t k_len, int32_t off, int32_t tok, int32_t n_tok) {
    KeyTiles t;
    const int32_t end = tok + n_tok - 1 + off, last = end < k_len ? end : k_len;   // keys below `last` are seen by some row
    if (n_tok <= 0 || last <= 0) return t;
    const int32_t lo = tok + off - m.window;
    t.first = lo > 0 ? lo / TILE_ROWS : 0;
    const int32_t s = m.sinks < last ? m.sinks : last, st = (s + TILE_ROWS - 1) / TILE_ROWS;
    t.sinks = st < t.first ? st : t.first;
    t.n = t.up_to(last);
    return t;
}

// The same for a row group of attn_rows.cu, in keys: [0, sinks) and from sinks + gap on, n in all; both edges
// are multiples of 16 keys (a block of that kernel, which no page ends in).
struct KeySpan {
    int32_t sinks = 0, gap = 0, n = 0;
    FQ_HD int32_t at(int32_t v) const { return v < sinks ? v : v + gap; }
};
FQ_HD inline KeySpan key_span(const AttnMask& m, int32_t k_len, int32_t off, int32_t n_tok) {
    KeySpan s;
    const int32_t end = n_tok - 1 + off, last = end < k_len ? end : k_len;
    if (n_tok <= 0 || last <= 0) return s;
    const int32_t lo = off - m.window, first = lo > 0 ? lo & ~15 : 0;
    const int32_t k = ((m.sinks < last ? m.sinks : last) + 15) & ~15;
    s.sinks = k < first ? k : first;
    s.gap = first - s.sinks;
    s.n = last - s.gap;
    return s;
}

// One unit of attn_tiles.cuh per kv head: two query tiles (pair) over the same keys, or one tile
// whose key tiles alternate between the two softmax warpgroups.
struct TileEntry {
    int32_t tok0;         // first token (of its sequence)
    uint32_t info;        // sequence | flags | (slot + 1) << 9; slot: first partial block (a pair has
                          // slot and slot + 1), 0 = finished outputs
    int32_t j0, j1;       // key tiles [j0, j1) (clipped to what the rows see)
};
constexpr uint32_t TILE_SINGLE = 1u << 7, TILE_SMALL = 1u << 8;   // SMALL: partial results of 8 rows
constexpr int TILE_SLOT_SHIFT = 9;

// A row group of attn_rows.cu: up to SMALL_ROWS packed rows over keys [0, k_len) in chunks, one CTA per
// chunk and kv head.
struct RowGroup {
    int32_t q_row0, n_tok, k_row0, k_len, off;
    int32_t seq;          // (for the host)
    int32_t item0;        // first work item (chunk) of the group
    int32_t chunk;        // keys per item, a multiple of 64
    int32_t slot0;        // first partial block, or -1: one item that writes finished outputs
    int32_t keys;         // that some row looks at (KeySpan::n)
};

// Rows whose output is joined from partial results: nA blocks of 128 rows from slot a0 (a0 +
// a_step, ..; row of token t: a_row + t * G), nB and nC blocks of 8 rows from slots b0 and c0
// (rows from b_row and 0).  Token t sees min(k_len, t + off) keys in all.
struct JoinEntry {
    int32_t q_row0, n_tok, k_len, off, a0, nA, a_step, a_row, b0, nB, b_row, c0, nC;
};

// Partial results: values and sums unnormalised against the row's reference maximum m (base 2),
//   o [slot][kv head][16 chunks of 8 dims][R rows][8] f32 (a warp with a row per lane writes
//   neighbouring 32 bytes), ml [slot][kv head][R] (m, l);  R = 128 (a) or 8 (b).
struct Partials {
    float *a_o = nullptr, *b_o = nullptr;
    float2 *a_ml = nullptr, *b_ml = nullptr;
};

// Bounded waits of attn_tiles.cuh: how long one may take, and where a CTA of which one gave up records it.
struct AttnWaits {
    uint32_t* record = nullptr;   // device word (null: the current device's own)
    uint32_t code = 0;            // bits set in it; 0: one is added
    uint32_t limit = 1u << 29;    // cycles: a quarter second, far beyond any wait that ends
    int starve = 0;               // failure tests: the loader of K (1) or V (2) leaves out the second tile of
                                  // each CTA's first unit, so that what waits for it runs out
};

template <int NV, int NE>
struct TileArgs {
    static constexpr int VIEWS = NV, ENTRIES = NE;
    static constexpr bool WINDOW = false, PAGED = false;
    alignas(64) unsigned long long map_q[16];
    alignas(64) unsigned long long map_k[NV][16], map_v[NV][16];
    AttnIo io;
    int n_entries;
    float c;              // |scale| log2(e)
    int negate;           // scale < 0
    int g_shift;          // log2(Hq / Hkv)
    uint32_t inv_hkv;     // ceil(2^31 / Hkv): units (below 2^31 / 1024) are divided by a product
    AttnWaits waits;
    Partials part;
    AttnSeq seq[MAX_SEQS];
    TileEntry e[NE];
};
// The parameters of a launch travel with it (2 us for 3 KB, 3.5 us for 30 KB), so short lists
// over one view or a few have types of their own.
using TileArgs1S = TileArgs<1, 64>;
using TileArgs1 = TileArgs<1, 1536>;
using TileArgsNS = TileArgs<17, 192>;
using TileArgsN = TileArgs<MAX_SEQS, 768>;
static_assert(sizeof(TileArgs1) <= 32764 && sizeof(TileArgsN) <= 32764, "kernel parameters");
// Windows and sinks over views (kv: the views' rows), or over pages (one map of the whole pool).
template <int NV, int NE, bool PAGES>
struct WindowTileArgs : TileArgs<NV, NE> {
    static constexpr bool WINDOW = true, PAGED = PAGES;
    AttnMask mask;
    KvRows kv[PAGES ? 1 : NV];
    KvPages pages;
};
using WindowArgs1S = WindowTileArgs<1, 64, false>;
using WindowArgs1 = WindowTileArgs<1, 1536, false>;
using WindowArgsN = WindowTileArgs<MAX_SEQS, 576, false>;
using PagedArgsS = WindowTileArgs<1, 64, true>;
using PagedArgsL = WindowTileArgs<1, 1536, true>;
static_assert(sizeof(WindowArgs1) <= 32764 && sizeof(WindowArgsN) <= 32764 && sizeof(PagedArgsL) <= 32764, "kernel parameters");
template <class Args>
void launch_tiles(const Args& a, cudaStream_t s);
cudaError_t attn_tiles_prepare();     // per device, before the first launch
cudaError_t attn_window_tiles_prepare();
cudaError_t attn_page_word(uint32_t** word);   // the current device's count of table entries without a page (never cleared)
cudaError_t attn_wait_word(uint32_t** word);   // the current device's own record (a count, never cleared)

constexpr int MAX_GROUPS = MAX_SEQS;
constexpr int ROWS_CTAS_SM = 3;                     // CTAs of attn_rows.cu per SM (159 to 168 registers x 128)
constexpr int ROWS_CTAS = ROWS_CTAS_SM * ATTN_SMS;  // ..  that run at once
constexpr int MAX_ITEMS = ROWS_CTAS + MAX_GROUPS;   // (a group is one item at least)
struct RowsArgs {
    static constexpr bool WINDOW = false, PAGED = false;
    AttnIo io;
    int n_items;
    float c;              // scale log2(e)
    Partials part;
    uint8_t group[MAX_ITEMS];   // of an item
    RowGroup g[MAX_GROUPS];
    KvRows kv[MAX_GROUPS];
};
// Windows and pages: the groups' keys lie on a line, of which an item (a CTA per kv head) takes an equal part, whatever groups that
// meets.  group: the first group of an item's part.  (A chunk of one group per item left some SMs three long ones and
// others two: window of 2048, 16 single tokens, 32 / 8 heads, 25 % above the mean.)
template <bool PAGES>
struct WindowRowsArgs : RowsArgs {
    static constexpr bool WINDOW = true, PAGED = PAGES;
    AttnMask mask;
    KvPages pages;
    int n_groups;
    int64_t share;              // an item's part of the line
    int64_t pos[MAX_GROUPS];    // where a group begins on it: ROWS_START, then its keys
};
// What the beginning of a group costs in keys (32: 32 tokens over pages 50.9 us, four tokens over 100 keys 9.0; 64: 49.8 and
// 5.4; 128: 51.0 and 5.3).
constexpr int ROWS_START = 64;
constexpr int ROWS_WHOLE = 128;   // keys of a group that is not cut, at most: the item with the first of them takes all
// Keys that a CTA's warps take at a time: cuts are whole ones from a group's first key on (60000 keys, one token 47.7 us, cut
// at any 16 keys 48.3).
constexpr int ROWS_STEP = 64;
FQ_HD inline int64_t rows_line(int keys) { return ROWS_START + (keys > 0 ? ((int64_t)keys + ROWS_STEP - 1) / ROWS_STEP * ROWS_STEP : ROWS_STEP); }
// Where a cut of the line falls in a group that begins at `first`, in keys.
FQ_HD inline int rows_cut(int64_t cut, int64_t first, int keys) {
    if (cut <= first) return 0;
    const int64_t at = (cut - first) / ROWS_STEP * ROWS_STEP;
    return at < keys ? (int)at : keys;
}
// The items that have a part of it: [i0, i1].
FQ_HD inline void rows_items(int64_t share, int64_t first, int keys, int& i0, int& i1) {
    i0 = (int)((first + (keys > ROWS_WHOLE ? ROWS_STEP - 1 : 0)) / share);
    i1 = keys > ROWS_WHOLE ? (int)((first + ((int64_t)keys + ROWS_STEP - 1) / ROWS_STEP * ROWS_STEP - 1) / share) : i0;
}
// The next group from g on of which the item has a part, and the numbers [c0, c1) of its keys; false: there is none.
template <class Args>
FQ_HD inline bool rows_part(const Args& a, int item, int& g, int& c0, int& c1) {
    const int64_t begin = item * a.share, end = begin + a.share;
    for (; g < a.n_groups && a.pos[g] < end; ++g) {
        const int keys = a.g[g].keys;
        const int64_t first = a.pos[g] + ROWS_START;
        c0 = rows_cut(begin, first, keys);
        c1 = rows_cut(end, first, keys);
        if (keys <= ROWS_WHOLE) {
            c0 = 0;
            c1 = keys;
            if (first >= begin && first < end) return true;
        } else if (c0 < c1) {
            return true;
        }
    }
    return false;
}
cudaError_t attn_rows_prepare();      // per device, before the first launch
cudaError_t attn_window_rows_prepare();
// beside: it may run beside launch_tiles of the same call, launched just before
void launch_attn_rows(const RowsArgs& a, bool beside, cudaStream_t s);
void launch_attn_window_rows(const WindowRowsArgs<false>& a, bool beside, cudaStream_t s);
void launch_attn_window_rows(const WindowRowsArgs<true>& a, bool beside, cudaStream_t s);

template <int NE>
struct JoinArgs {
    static constexpr int ENTRIES = NE;
    AttnIo io;
    int n_entries, max_tok, max_parts;   // tokens and partial results of an entry, at most
    Partials part;
    JoinEntry e[NE];
};
using JoinArgsS = JoinArgs<64>;
using JoinArgsL = JoinArgs<512>;
static_assert(sizeof(JoinArgsL) <= 32764, "kernel parameters");
// behind launch_tiles, launch_attn_rows or another join of the same call
template <class Args>
void launch_attn_join(const Args& a, cudaStream_t s);

// The entry points fq_attn_prompt and fq_attn_shared with the record of their waits, and fq_attn_prompt of one
// sequence with whole units (no workspace).
fq_status attn_prompt(const AttnWaits& waits, const void* q, uint64_t q_stride, const fq_kv_view* views, uint32_t n_views,
                      uint32_t n_seq, const uint32_t* q_len, const uint32_t* kv_row0, const uint32_t* k_len, uint32_t Hq,
                      uint32_t Hkv, float scale, void* out, uint64_t out_stride, fq_dtype out_dtype, void* workspace,
                      size_t workspace_bytes, void* stream);
fq_status attn_shared(const AttnWaits& waits, const void* q, uint64_t q_stride, uint32_t n_seq, const fq_kv_view* prefix,
                      uint32_t prefix_len, const fq_kv_view* tails, const uint32_t* tail_len, uint32_t Hq, uint32_t Hkv,
                      float scale, void* out, uint64_t out_stride, fq_dtype out_dtype, void* workspace,
                      size_t workspace_bytes, void* stream);
// The current device's number and the word that counts its give-ups of calls that belong to no model; and the word that counts
// table entries without a page there (one for all paged calls), for fq_attn_check.
fq_status attn_device(int* dev, uint32_t** waits);
void attn_set_page_word(int dev, uint32_t* word);
fq_status attn_prompt_whole(const AttnWaits& waits, const void* q, const fq_kv_view* view, uint32_t q_len, uint32_t k_len,
                            uint32_t Hq, uint32_t Hkv, void* out, void* stream);

}  // namespace fq
