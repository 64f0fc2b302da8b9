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

// The work of key_weights.cu is a line of entries, once per kv head, that the thread blocks share out in equal parts wherever
// the cuts fall (units dealt out whole, longest first, left SMs idle: one prompt of 4096 tokens, 32 / 8 heads, 82 us,
// 65 now).  Query blocks are 96 packed rows of the sequence (whole tokens of every group).
constexpr int KW_BLOCK = 96;
struct KwEntry {
    int32_t info;         // sequence | kind | KW_MORE
    int32_t j0, j1;       // key tiles
    int32_t b0, len;      // first query block; length on the line
    int32_t pos;          // where it begins on the line: kw_start in front of len
};
constexpr int KW_KEYS = 0;           // up to two key tiles [j0, j1) stay, query blocks b0 .. b0 + len - 1 pass by
constexpr int KW_ROWS = 1 << 7;      // the only query block stays, key tiles j0 .. j0 + len - 1 pass by
constexpr int KW_NONE = 2 << 7;      // keys that no row sees, KW_REST tiles of [j0, j1) each
constexpr int KW_MORE = 1 << 9;      // adds to what an earlier launch of the call left
constexpr int KW_KEY_TILES = 2;      // .. that stay
constexpr int KW_REST = 32;
// Query blocks of an entry that is not cut, at most (64 tokens over 16000 keys, 32 / 8 heads: 22.5 us, 23.8 with cuts;
// 8 instead of 4: 2048 tokens, 16 / 8 heads, 19.3 instead of 17.6 us).
constexpr int KW_WHOLE = 4;
// What the beginning of a unit costs in query blocks passing by (5 to 7 from the cycles of units of 12 to 300 blocks,
// some of it the tiles that are masked in part; 8192 tokens 220 us, with 6 222.5, with 8 226.6).
FQ_HD inline int kw_start(int kind) { return kind == KW_KEYS ? 4 : kind == KW_ROWS ? 1 : 0; }

// The part of an entry and kv head that a thread block takes.
struct KwUnit {
    int seq, head, kind, j0, j1, b0, b1;
    int slot;             // partial sums of its 256 keys, or -1: nobody else has a part of them
    bool more;
    int stay, pass;       // tiles that stay; that pass by
};
struct KwLine {
    int64_t begin, end, base;   // the thread block's part; where its kv head's line begins
    int head, e, cta;
};
template <class Args>
FQ_HD inline KwLine kw_line(const Args& a, int cta) {
    KwLine l;
    const int64_t all = (int64_t)a.total * a.Hkv;
    l.cta = cta;
    l.begin = cta * a.share;
    l.end = l.begin + a.share < all ? l.begin + a.share : all;
    l.head = (int)(l.begin / a.total);
    l.base = (int64_t)l.head * a.total;
    const int64_t at = l.begin - l.base;
    int lo = 0, hi = a.n_entries;   // the last entry that begins there or before
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.e[mid].pos <= at) lo = mid;
        else hi = mid;
    }
    l.e = lo;
    return l;
}
// The next of its units; false: there is none.  Short entries (KW_WHOLE) go to the thread block with their first block.  A cut in front of an entry's first block leaves the whole entry to the thread block
// behind the cut.  Of an entry that is cut every thread block has one part, so two slots each are enough: for the part
// that begins an entry (its last unit), and for one that goes on with an entry (its first).
template <class Args>
FQ_HD inline bool kw_next(const Args& a, KwLine& l, KwUnit& u) {
    for (;;) {
        if (l.e == a.n_entries) {
            l.e = 0;
            ++l.head;
            l.base += a.total;
        }
        const KwEntry& e = a.e[l.e];
        if (l.base + e.pos >= l.end) return false;
        ++l.e;
        u.kind = e.info & (KW_ROWS | KW_NONE);
        const int64_t first = l.base + e.pos + kw_start(u.kind);
        int lo = l.begin > first ? (int)(l.begin - first < e.len ? l.begin - first : e.len) : 0;
        int hi = l.end - first < e.len ? (int)(l.end > first ? l.end - first : 0) : e.len;
        if (u.kind == KW_KEYS && e.len <= KW_WHOLE) {
            lo = lo > 0 || l.end <= first ? e.len : 0;
            hi = e.len;
        }
        if (lo >= hi) continue;
        u.seq = e.info & 127;
        u.head = l.head;
        u.more = e.info & KW_MORE;
        u.j0 = e.j0;
        u.j1 = e.j1;
        u.b0 = 0;
        u.b1 = 1;
        u.slot = -1;
        u.stay = u.pass = 0;
        if (u.kind == KW_KEYS) {
            u.b0 = e.b0 + lo;
            u.b1 = e.b0 + hi;
            if (lo > 0 || hi < e.len) u.slot = 2 * l.cta + (lo == 0);
            u.stay = u.j1 - u.j0;
            u.pass = hi - lo;
        } else if (u.kind == KW_ROWS) {
            u.j0 = e.j0 + lo;
            u.j1 = e.j0 + hi;
            u.stay = 1;
            u.pass = hi - lo;
        } else {
            u.j0 = e.j0 + KW_REST * lo;
            u.j1 = hi < e.len ? e.j0 + KW_REST * hi : e.j1;
        }
        return true;
    }
}
// The thread blocks [c0, c1] that have parts of entry i (KW_KEYS) and a kv head.
template <class Args>
FQ_HD inline void kw_parts(const Args& a, int i, int head, int& c0, int& c1) {
    const int64_t first = (int64_t)head * a.total + a.e[i].pos + kw_start(KW_KEYS);
    c0 = (int)(first / a.share);
    c1 = a.e[i].len <= KW_WHOLE ? c0 : (int)((first + a.e[i].len - 1) / a.share);
}

template <int NV, int NE>
struct KwArgs {
    static constexpr int VIEWS = NV, ENTRIES = NE;
    alignas(64) unsigned long long map_q[16];
    alignas(64) unsigned long long map_k[NV][16];
    const float* lse;     // [rows][Hq]
    int Hq, Hkv, g_shift, n_entries;
    float c;              // scale log2(e)
    int total;            // length of a kv head's line
    int64_t share;        // .. of a thread block's part
    AttnMask mask;
    AttnWaits waits;
    float* part;          // [slot][256]
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
void launch_key_weights(const Args& a, int grid, cudaStream_t s);
template <class Args>
void launch_key_weights_join(const Args& a, cudaStream_t s);   // sums of keys that several thread blocks have parts of, just behind it
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
