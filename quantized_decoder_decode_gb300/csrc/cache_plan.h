// Arguments of the kernels that make caches shorter: the attention weights that keys receive (key_weights.cu), and
// the choice and the move of the rows that stay (evict.cu).  Made on the host in attn_cache_api.cu, passed by value.
#pragma once

#include "attn_plan.h"

namespace fq {

// Gathered weights of a view's rows: of row r and kv head h at [h * stride + r].
struct KeyWeights {
    const float* before = nullptr;   // null: zeros
    float* after = nullptr;
    int64_t before_stride = 0, after_stride = 0;
};

// A unit of key_weights.cu per kv head.  Query blocks are 96 packed rows of the sequence (whole tokens of every group).
constexpr int KW_BLOCK = 96;
struct KwEntry {
    int32_t info;         // sequence | kind
    int32_t j0, j1;       // key tiles
    int32_t b0, b1;       // query blocks
    int32_t slot;         // partial sums of the unit's 256 keys, or -1: finished
};
constexpr int KW_KEYS = 0;           // up to two key tiles stay, query blocks [b0, b1) pass by
constexpr int KW_ROWS = 1 << 7;      // the only query block stays, key tiles [j0, j1) pass by
constexpr int KW_NONE = 2 << 7;      // keys that no row sees
constexpr int KW_KEY_TILES = 2;      // .. that stay

// Keys whose sums come from several units: n partial sums from slot on.
struct KwJoin {
    int32_t seq, j0, j1, slot, n;   // of key tiles [j0, j1)
};

template <int NV, int NE>
struct KwArgs {
    static constexpr int VIEWS = NV, ENTRIES = NE;
    alignas(64) unsigned long long map_q[16];
    alignas(64) unsigned long long map_k[NV][16];
    const float* lse;     // [rows][Hq]
    int Hq, Hkv, g_shift, n_entries;
    float c;              // scale log2(e)
    AttnMask mask;
    AttnWaits waits;
    float* part;          // [slot][kv head][256]
    AttnSeq seq[MAX_SEQ];
    KeyWeights w[NV];
    KwEntry e[NE];
};
using KwArgs1S = KwArgs<1, 64>;
using KwArgs1M = KwArgs<1, 256>;
using KwArgs1 = KwArgs<1, 1152>;
using KwArgsN = KwArgs<MAX_SEQ, 768>;
static_assert(sizeof(KwArgs1) <= 32764 && sizeof(KwArgsN) <= 32764, "kernel parameters");
template <class Args>
void launch_key_weights(const Args& a, cudaStream_t s);

struct KwJoinArgs {
    static constexpr int ENTRIES = 896;
    const float* part;
    int Hkv, n_entries;
    AttnSeq seq[MAX_SEQ];
    KeyWeights w[MAX_SEQ];
    KwJoin e[ENTRIES];
};
static_assert(sizeof(KwJoinArgs) <= 32764, "kernel parameters");
void launch_key_weights_join(const KwJoinArgs& a, cudaStream_t s);   // behind launch_key_weights of the same call
cudaError_t key_weights_prepare();    // per device, before the first launch

struct EvictSeq {
    const float* w;       // gathered weight of the sequence's first row, kv head 0
    float* w_to;          // or null
    int64_t w_stride, w_to_stride;
    KvRows from, to;      // at the sequence's first row
    int32_t len, n;       // rows, rows that stay
    int64_t kept0;        // its numbers in `kept`: [kv head][n] from here
    int32_t block0;       // first thread block of the move
};
struct EvictArgs {
    int n_seq, Hkv, sinks, recent;
    int32_t* kept;
    EvictSeq s[MAX_SEQ];
};
constexpr int EVICT_ROWS = 32;        // rows that a thread block moves
void launch_evict(const EvictArgs& a, int max_len, int blocks, cudaStream_t s);

}  // namespace fq
