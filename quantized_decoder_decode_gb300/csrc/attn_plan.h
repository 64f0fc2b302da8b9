// Work lists of the prompt and shared-prompt attention kernels, made on the host
// (attn_api.cu) and passed by value to attn_tiles.cu, attn_rows.cu and its join kernel.
//
// "Packed rows": a kv head's query rows are (token, head of its group) with the head running
// fastest, so G heads x tokens fill the 128 rows (or 8 columns) of a matrix product.
#pragma once

#include "kernels.h"

namespace fq {

constexpr int ATTN_SMS = 152;         // SMs that the work lists are made for
constexpr int TILE_ROWS = 128;        // packed rows of a query tile = keys of a key tile
constexpr int ROWS_MAX = 8;           // packed rows that attn_rows.cu takes
constexpr int32_t SEES_ALL = 1 << 30; // PromptSeq::off of rows that see every key

// Row i (token) of a sequence sees keys [0, min(k_len, i + off)), off = k_len - q_len + 1.
struct PromptSeq {
    int32_t q_row0, q_len, k_row0, k_len, off;
};

// One unit of attn_tiles.cu per kv head: two query tiles (pair) over the same keys, or one tile
// whose key tiles alternate between the two softmax warpgroups.
struct TileEntry {
    int32_t tok0;         // first token (of its sequence)
    uint32_t info;        // sequence | single tile << 6 | (slot + 1) << 8; slot: partial blocks (a
                          // pair uses slot, slot + 1), 0 = finished outputs
    int32_t j0, j1;       // key tiles [j0, j1) (clipped to what the rows see)
};
constexpr uint32_t TILE_SINGLE = 1u << 6;

// A row group of attn_rows.cu: up to ROWS_MAX packed rows over keys [0, k_len) in `splits`
// chunks, one CTA per chunk and kv head.
struct RowGroup {
    int32_t q_row0, n_tok, k_row0, k_len, off;
    int32_t item0;        // first work item (chunk) of the group
    int32_t chunk;        // keys per item, a multiple of 64
    int32_t slot0;        // first partial block, or -1: one item that writes finished outputs
};

// Rows whose output is joined from partial results: nA blocks of attn_tiles.cu (slots a0, a0 +
// a_step, ..; row of token t: a_row + t * G), nB and nC blocks of attn_rows.cu (slots b0 .. and
// c0 .., rows from b_row and 0).  Token t sees min(k_len, t + off) keys in all.
struct JoinEntry {
    int32_t q_row0, n_tok, k_len, off, a0, nA, a_step, a_row, b0, nB, b_row, c0, nC;
};

// Partial results: sums and values unnormalised against the row's reference maximum m (base 2).
//   tiles: o [slot][kv head][16 dim chunks][128 rows][8] f32 (a warp with a row per lane writes
//          neighbouring rows), ml [slot][kv head][128] (m, l)
//   rows:  o [slot][kv head][8 rows][128],           ml [slot][kv head][8]
struct Partials {
    float *a_o = nullptr, *b_o = nullptr;
    float2 *a_ml = nullptr, *b_ml = nullptr;
};

constexpr int MAX_JOIN = 512;
constexpr int MAX_GROUPS = MAX_SEQ + 1;
constexpr int ROWS_CTAS_SM = 3;                     // CTAs of attn_rows.cu per SM (156 registers x 128)
constexpr int ROWS_CTAS = ROWS_CTAS_SM * ATTN_SMS;  // ..  that run at once
constexpr int MAX_ITEMS = ROWS_CTAS + MAX_GROUPS;   // (a group is one item at least)

template <int NV, int NE>
struct TileArgs {
    static constexpr int VIEWS = NV, ENTRIES = NE;
    alignas(64) unsigned long long map_q[16];
    alignas(64) unsigned long long map_k[NV][16], map_v[NV][16];
    AttnIo io;
    int n_entries;
    float c;              // |scale| log2(e)
    int negate;           // scale < 0
    Partials part;
    PromptSeq seq[MAX_SEQ];
    TileEntry e[NE];
};
// Every sequence over one view, or a view per sequence.  The parameters of a launch travel with
// it, so the common short list has a type of its own.
using TileArgsS = TileArgs<1, 64>;
using TileArgs1 = TileArgs<1, 1536>;
using TileArgsN = TileArgs<MAX_SEQ, 768>;
static_assert(sizeof(TileArgs1) <= 32764 && sizeof(TileArgsN) <= 32764, "kernel parameters");
template <class Args>
void launch_tiles(const Args& a, cudaStream_t s);
cudaError_t attn_tiles_prepare();     // per device, before the first launch
cudaError_t attn_wait_record(uint32_t* host, cudaStream_t s);

struct RowsArgs {
    AttnIo io;
    int n_groups, n_items;
    float c;              // scale log2(e)
    Partials part;
    uint8_t group[MAX_ITEMS];   // of an item
    RowGroup g[MAX_GROUPS];
    KvRows kv[MAX_GROUPS];
};
// dependent: behind launch_tiles of the same call, whose CTAs it may run beside
void launch_attn_rows(const RowsArgs& a, bool dependent, cudaStream_t s);

template <int NE>
struct JoinArgs {
    static constexpr int ENTRIES = NE;
    AttnIo io;
    int n_entries, max_tok;
    Partials part;
    JoinEntry e[NE];
};
using JoinArgsS = JoinArgs<64>;
using JoinArgsL = JoinArgs<MAX_JOIN>;
static_assert(sizeof(JoinArgsL) <= 32764, "kernel parameters");
// behind launch_tiles or launch_attn_rows of the same call
template <class Args>
void launch_attn_join(const Args& a, cudaStream_t s);

}  // namespace fq
