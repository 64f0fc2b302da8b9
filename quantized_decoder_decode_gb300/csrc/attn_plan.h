// Arguments of the prompt and shared-prompt attention operators' kernels, and their work lists, made on the host
// (attn_api.cu) and passed by value to attn_tiles.cu, attn_rows.cu and attn_join.cu.
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

// QK-norm + rope of packed rows, q -> q_out, k and v -> cache rows (qk_rows.cu)
struct QkRowsArgs {
    const float* qkv;             // [rows][(Hq + 2 Hkv) * 128]
    int64_t qkv_stride;
    const float *q_norm, *k_norm; // [128]
    const float2* rope;           // [positions][64] (cos, sin)
    float eps;
    int Hq, Hkv, n_seq, rows;
    uint16_t* q_out;              // bf16 [rows][Hq * 128]
    int64_t q_stride;
    int32_t row0[MAX_SEQ], pos0[MAX_SEQ], kv_row0[MAX_SEQ];   // per sequence: first row, position, cache row
    KvRows kv[MAX_SEQ];
};
void launch_qk_rows(const QkRowsArgs& a, cudaStream_t s);

struct AttnIo {
    const uint16_t* q;            // bf16 [rows][Hq][128]
    int64_t q_stride;
    void* out;                    // bf16 or f32 [rows][Hq][128]
    int64_t out_stride;
    int out_f32;
    int Hq, Hkv;
    float scale;
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

// One unit of attn_tiles.cu per kv head: two query tiles (pair) over the same keys, or one tile
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

// Bounded waits of attn_tiles.cu: how long one may take, and where a CTA of which one gave up records it.
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
template <class Args>
void launch_tiles(const Args& a, cudaStream_t s);
cudaError_t attn_tiles_prepare();     // per device, before the first launch
cudaError_t attn_wait_word(uint32_t** word);   // the current device's own record (a count, never cleared)

constexpr int MAX_GROUPS = MAX_SEQS;
constexpr int ROWS_CTAS_SM = 3;                     // CTAs of attn_rows.cu per SM (158 registers x 128)
constexpr int ROWS_CTAS = ROWS_CTAS_SM * ATTN_SMS;  // ..  that run at once
constexpr int MAX_ITEMS = ROWS_CTAS + MAX_GROUPS;   // (a group is one item at least)
struct RowsArgs {
    AttnIo io;
    int n_items;
    float c;              // scale log2(e)
    Partials part;
    uint8_t group[MAX_ITEMS];   // of an item
    RowGroup g[MAX_GROUPS];
    KvRows kv[MAX_GROUPS];
};
cudaError_t attn_rows_prepare();      // per device, before the first launch
// beside: it may run beside launch_tiles of the same call, launched just before
void launch_attn_rows(const RowsArgs& a, bool beside, cudaStream_t s);

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
fq_status attn_prompt_whole(const AttnWaits& waits, const void* q, const fq_kv_view* view, uint32_t q_len, uint32_t k_len,
                            uint32_t Hq, uint32_t Hkv, void* out, void* stream);

}  // namespace fq
