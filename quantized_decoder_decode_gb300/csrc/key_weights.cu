// The attention weight that every key receives, on the 5th-generation tensor cores (tcgen05, sm_103a):
//   after[j] = before[j] + sum over query rows i (and the heads of the group) that see key j of 2^(c q_i.k_j - lse_i log2(e)),
// c = scale log2(e), lse_i the log-sum that the attention of the same rows left.
//
// The scores are taken the other way round than in attention, S = K Q^T with the keys as the rows of the product: a
// thread then has one key's scores in its own lane of tensor memory and adds their exponentials up by itself.  No
// maximum is needed, no weight leaves the registers, and no two threads write the same sum (atomics would add
// in any order).  Sums of a tile of 96 weights go to the thread's total by compensated addition.  Behind that, sums are added
// plainly, always in the same order: those of the two warpgroups that share a key's query blocks, and those of the
// thread blocks that have parts of it (up to 152, a rounding of 2^-24 of the sum each at most; a prompt of 8192 tokens is off by
// 6e-8 in the root mean square, as much as one rounding).
//
// A unit holds what is few and lets the rest pass by through a ring of 32 KB tiles (TMA):
//   KW_KEYS  two key tiles stay (one for each of two pairs of warpgroups), query blocks of 96 packed rows pass by;
//   KW_ROWS  the rows of a query block stay (single tokens, a few observed ones), key tiles pass by, to the four
//            warpgroups in turn: K is read once, which is what bounds it.
// What stays has two sets of buffers, so that the next unit's comes while this one is worked on; keys that stay move on to
// tensor memory, as the product's first operand (with both operands in shared memory its reads, those of the statistics and
// the copies coming in ask for more than its 128 bytes a cycle).  All units of a call are laid in a line that the CTAs share
// out in equal parts; keys of which several CTAs have a part get their sums from a second kernel, which adds the parts up in order.
//
// Tensor memory: an S buffer of 96 columns for each of four warpgroups, two key tiles.  Shared memory: 2 x 2 tiles that stay, 3
// that pass by.  Roles (608 threads, one CTA per SM, looping over its units): warps 0-15 exponentials and sums, a key per thread; warp 16
// loads; warp 17 issues the products; warp 18 brings the rows' log-sums.  Every wait is bounded; one that gives up records it,
// and all roles leave.
//
// What bounds it.  16 single tokens over 512 to 4097 keys, 32 / 8 heads (79 MB): 11.1 us, memory (floor 11.5 at the rate of a
// plain copy).  One prompt, 32 / 8 heads: 2048 tokens 25 us, 4096 65, 8192 220 (products alone 144).  The exponentials of a
// tile take the special-function units as long as its product takes the tensor cores (384 cycles for 96 columns), and a
// block of query rows, two tiles, takes 1380 cycles: of a warpgroup's round of 2760 cycles (four tiles, one for each) some 580 pass
// until its one S buffer is filled again, and tensor memory has no room for a second.  A tile that is masked in part
// takes half as long again; a warp whose keys all see none of its rows leaves it out, and keys that see all of
// them beside keys that see none (a window's sinks) take the short way: 8192 tokens with a window of 1000, 137 -> 80 us.
//
// Slower, of 8192 tokens: two warpgroups with two S buffers each (384 us), four that share tiles by their columns (297),
// operands in shared memory (260), S in halves of 48 columns (287: such a product takes the tensor cores as long as one of 96).
// No faster: reads of 24 columns, of 32 (they spill), S given back before its last columns are worked on, a second issuing thread.

#include <cstddef>

#include "attn.cuh"
#include "cache_plan.h"
#include "tc.cuh"

namespace fq {

namespace {

constexpr int KW_THREADS = 608;
constexpr int KW_RING = 3;
constexpr int KW_TILE_BYTES = TILE_ROWS * HEAD_DIM * 2;   // 32 KB
constexpr int KW_PANEL = KW_TILE_BYTES / 2;               // 64 dims of 128 keys
constexpr int KW_Q_PANEL = KW_BLOCK * 128;                // 64 dims of a query block
constexpr uint32_t KW_S = 0, KW_K = 4 * KW_BLOCK;         // tensor-memory columns: four S buffers, two key tiles (64 each)
static_assert(KW_K + 128 <= 512, "tensor memory");

// Warpgroup x + 2 y (x, y = 0, 1).  Where keys stay, x is its key tile and the query blocks go to y = 0 and 1 in turn; where query blocks
// stay, the key tiles go to warpgroups 0, 1, 2, 3 in turn.
struct KwShared {
    uint64_t st_full[2], st_empty[2];              // per set of tiles that stay
    uint64_t ring_full[KW_RING], ring_empty[KW_RING];
    uint64_t s_full[4], s_free[4];                 // per warpgroup: its S buffer
    uint64_t neg_full[2][2], neg_empty[2][2];      // per y, two buffers in turn
    uint64_t half_full[2];                         // per x: the sums of y = 1 are in its S buffer
    uint64_t k_go[2], k_ready[2];                  // per x: its key tile may move to tensor memory; is there
    uint32_t tmem;
    uint32_t limit;                                // cycles that a wait may take; 0: one gave up, all roles leave
    alignas(16) float neg[2][2][KW_BLOCK];         // (read 16 bytes at a time) -lse log2(e) of a query block's rows
};
constexpr int KW_SMEM = (4 + KW_RING) * KW_TILE_BYTES + 3072;
static_assert(sizeof(KwShared) <= 3072 && KW_SMEM <= 232448, "shared memory");
static_assert(offsetof(KwShared, neg) % 16 == 0, "16-byte reads");

// one column of tensor memory, a value per lane
FQ_DEV void tmem_st1(uint32_t taddr, float x) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(__float_as_uint(x)) : "memory");
}
FQ_DEV float tmem_ld1(uint32_t taddr) {
    uint32_t x;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;" : "=r"(x) : "r"(taddr) : "memory");
    return __uint_as_float(x);
}

FQ_DEV uint32_t wait_limit(const KwShared* sh) { return *(const volatile uint32_t*)&sh->limit; }
FQ_DEV bool kw_wait(uint64_t* bar, uint32_t parity, KwShared* sh) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint32_t t0 = (uint32_t)clock();
    while (!mbar_try_wait(bar, parity)) {
        const uint32_t limit = wait_limit(sh);
        if ((uint32_t)clock() - t0 > limit) {
            if (limit) *(volatile uint32_t*)&sh->limit = 0;
            return false;
        }
    }
    return true;
}
FQ_DEV bool kw_wait_warp(uint64_t* bar, uint32_t parity, KwShared* sh) {
    return __all_sync(0xFFFFFFFFu, kw_wait(bar, parity, sh));
}
FQ_DEV void kw_drain() {   // copies in flight land within microseconds of a wait that gave up
    const long long t0 = clock64();
    while (clock64() - t0 < 1 << 20) {
    }
}

// By one thread: key tile j or query block b of a unit's sequence.
template <class Args>
FQ_DEV void kw_load_k(const Args& a, const KwUnit& u, int j, uint8_t* dst, uint64_t* bar) {
    const AttnSeq& s = a.seq[u.seq];
    const void* map = a.map_k[Args::VIEWS == 1 ? 0 : s.view];
    tma_load_3d(dst, map, 0, s.k_row0 + j * TILE_ROWS, u.head, bar);
    tma_load_3d(dst + KW_PANEL, map, 64, s.k_row0 + j * TILE_ROWS, u.head, bar);
}
template <class Args>
FQ_DEV void kw_load_q(const Args& a, const KwUnit& u, int b, uint8_t* dst, uint64_t* bar) {
    const int row = a.seq[u.seq].q_row0 + (b * KW_BLOCK >> a.g_shift);
    tma_load_4d(dst, a.map_q, 0, 0, u.head, row, bar);
    tma_load_4d(dst + KW_Q_PANEL, a.map_q, 64, 0, u.head, row, bar);
}

// Columns of a product: a query block's rows, or (a block that stays) what there are of them, in steps of 32.
template <class Args>
FQ_DEV int kw_columns(const Args& a, const KwUnit& u) {
    return u.kind == KW_KEYS ? KW_BLOCK : ((a.seq[u.seq].q_len << a.g_shift) + 31) & ~31;
}

// ---------------- warp 16
template <class Args>
FQ_DEV void kw_load(const Args& a, KwShared* sh, uint8_t* stay, uint8_t* ring) {
    uint32_t n = 0, un = 0;   // tiles that pass by; units with tiles
    bool ok = true;
    KwUnit u;
    for (KwLine l = kw_line(a, blockIdx.x); ok && kw_next(a, l, u);) {
        if (!u.pass) continue;
        const int set = un & 1;
        if (!(ok = kw_wait_warp(&sh->st_empty[set], ((un >> 1) & 1) ^ 1, sh))) break;
        ++un;
        if (elect_one()) {
            mbar_arrive_expect_tx(&sh->st_full[set], u.stay * (u.kind == KW_ROWS ? 2 * KW_Q_PANEL : KW_TILE_BYTES));
            for (int x = 0; x < u.stay; ++x) {
                uint8_t* dst = stay + (2 * set + x) * KW_TILE_BYTES;
                if (u.kind == KW_ROWS) kw_load_q(a, u, u.b0 + x, dst, &sh->st_full[set]);
                else kw_load_k(a, u, u.j0 + x, dst, &sh->st_full[set]);
            }
        }
        __syncwarp();
        for (int i = 0; i < u.pass; ++i, ++n) {
            const int s = n % KW_RING;
            if (!(ok = kw_wait_warp(&sh->ring_empty[s], ((n / KW_RING) & 1) ^ 1, sh))) break;
            if (elect_one()) {
                mbar_arrive_expect_tx(&sh->ring_full[s], u.kind == KW_ROWS ? KW_TILE_BYTES : 2 * KW_Q_PANEL);
                if (u.kind == KW_ROWS) kw_load_k(a, u, u.j0 + i, ring + s * KW_TILE_BYTES, &sh->ring_full[s]);
                else kw_load_q(a, u, u.b0 + i, ring + s * KW_TILE_BYTES, &sh->ring_full[s]);
            }
            __syncwarp();
        }
    }
    // the products' arrivals at these barriers come by themselves: the CTA leaves behind the last of them
#pragma unroll 1
    for (uint32_t i = n > KW_RING ? n - KW_RING : 0; i < n && ok; ++i) ok = kw_wait_warp(&sh->ring_empty[i % KW_RING], (i / KW_RING) & 1, sh);
#pragma unroll 1
    for (uint32_t i = un > 2 ? un - 2 : 0; i < un && ok; ++i) ok = kw_wait_warp(&sh->st_empty[i & 1], (i >> 1) & 1, sh);
    if (!ok) kw_drain();
}

// ---------------- warp 17, one thread of it.  A product takes the tensor cores 384 cycles, and this loop has no more for it: its waits are
// tests of one thread, its addresses are counted on, and what depends on the kind of unit is decided outside it.
template <bool ROWS>
FQ_DEV bool kw_unit_products(KwShared* sh, const KwUnit& u, uint64_t d_stay, uint64_t d_ring, uint32_t tm, uint32_t idesc, uint32_t& slot,
                             uint32_t& slot_ph, uint32_t& free_ph) {
    uint64_t dr = d_ring + (uint32_t)(slot * (KW_TILE_BYTES >> 4));
#pragma unroll 1
    for (int i = 0; i < u.pass; ++i) {
        if (!kw_wait(&sh->ring_full[slot], slot_ph, sh)) return false;
#pragma unroll
        for (int x = 0; x < (ROWS ? 1 : 2); ++x) {
            if (x >= u.stay) break;
            const int wg = ROWS ? i & 3 : x + 2 * (i & 1);
            if (!kw_wait(&sh->s_free[wg], (free_ph >> wg & 1) ^ 1, sh)) return false;
            free_ph ^= 1u << wg;
            tc_fence_after();
            const uint32_t d = tm + KW_S + KW_BLOCK * wg;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint32_t q_off = (k >> 2) * (KW_Q_PANEL >> 4) + (k & 3) * 2, k_off = (k >> 2) * (KW_PANEL >> 4) + (k & 3) * 2;
                if (ROWS) mma_f16(d, dr + k_off, d_stay + q_off, idesc, k > 0);
                else mma_f16_ta(d, tm + KW_K + 64 * x + 8 * k, dr + q_off, idesc, k > 0);
            }
            mma_commit(&sh->s_full[wg]);
        }
        mma_commit(&sh->ring_empty[slot]);
        dr += KW_TILE_BYTES >> 4;
        if (++slot == KW_RING) {
            slot = 0;
            slot_ph ^= 1;
            dr = d_ring;
        }
    }
    return true;
}

template <class Args>
FQ_DEV void kw_products(const Args& a, KwShared* sh, uint8_t* stay, uint8_t* ring, uint32_t tm) {
    const uint64_t d_stay = sdesc_sw128(smem_u32(stay)), d_ring = sdesc_sw128(smem_u32(ring));
    uint32_t un = 0, free_ph = 0, ready_ph = 0, slot = 0, slot_ph = 0;   // units; phase bits of s_free and of k_ready; the ring's next tile
    KwUnit u;
    for (KwLine l = kw_line(a, blockIdx.x); kw_next(a, l, u);) {
        if (!u.pass) continue;
        const int set = un & 1;
        if (!kw_wait(&sh->st_full[set], (un >> 1) & 1, sh)) break;
        ++un;
        const uint32_t idesc = idesc_bf16_f32(TILE_ROWS, kw_columns(a, u), false, false);
        if (u.kind == KW_ROWS) {
            if (!kw_unit_products<true>(sh, u, d_stay + (uint32_t)(2 * set * (KW_TILE_BYTES >> 4)), d_ring, tm, idesc, slot, slot_ph, free_ph)) break;
            mma_commit(&sh->st_empty[set]);
            continue;
        }
        // the key tiles become operands in tensor memory
        for (int x = 0; x < u.stay; ++x) mbar_arrive(&sh->k_go[x]);
        bool ok = true;
        for (int x = 0; x < u.stay && ok; ++x) {
            ok = kw_wait(&sh->k_ready[x], ready_ph >> x & 1, sh);
            ready_ph ^= 1u << x;
        }
        if (!ok) break;
        tc_fence_after();
        mbar_arrive(&sh->st_empty[set]);
        if (!kw_unit_products<false>(sh, u, 0, d_ring, tm, idesc, slot, slot_ph, free_ph)) break;
    }
}

// ---------------- warp 18: -lse log2(e) of the rows of query blocks, for y = 0 and 1 in turn where keys stay, for both where
// query blocks do.  A block's values are on their way while the one before is put down.
template <class Args>
FQ_DEV void kw_statistics(const Args& a, KwShared* sh, int lane) {
    constexpr float LOG2E = 1.4426950408889634f;
    const int shift = a.g_shift, G = 1 << shift;
    uint32_t blk[2] = {0, 0};
    bool ok = true;
    KwUnit u;
    for (KwLine l = kw_line(a, blockIdx.x); ok && kw_next(a, l, u);) {
        if (u.kind == KW_NONE) continue;
        const AttnSeq& sq = a.seq[u.seq];
        const int n = u.b1 - u.b0;
        auto fetch = [&](int b, float (&v)[4]) {   // rows 4 lane .. (beyond the sequence: a weight of 0)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int p = b * KW_BLOCK + 4 * lane + k, tok = p >> shift;
                v[k] = 4 * lane < KW_BLOCK && tok < sq.q_len ? __ldg(a.lse + (int64_t)(sq.q_row0 + tok) * a.Hq + (u.head << shift) + (p & (G - 1))) : INFINITY;
            }
        };
        float v[4];
        fetch(u.b0, v);
        for (int i = 0; i < n && ok; ++i) {
            float now[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) now[k] = -LOG2E * v[k];
            if (i + 1 < n) fetch(u.b0 + i + 1, v);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                if (u.kind != KW_ROWS && y != (i & 1)) continue;
                const int s = blk[y] & 1;
                if (!(ok = kw_wait_warp(&sh->neg_empty[y][s], ((blk[y] >> 1) & 1) ^ 1, sh))) break;
                ++blk[y];
                if (4 * lane < KW_BLOCK) *reinterpret_cast<float4*>(&sh->neg[y][s][4 * lane]) = make_float4(now[0], now[1], now[2], now[3]);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->neg_full[y][s]);
            }
        }
    }
}

// ---------------- warps 0-15
// A number with the rounding errors of its additions beside it (compensated summation).
struct Total {
    float sum = 0.f, err = 0.f;
    FQ_DEV void add(float x) {
        const float y = __fsub_rn(x, err), t = __fadd_rn(sum, y);
        err = fabsf(t) < INFINITY ? __fsub_rn(__fsub_rn(t, sum), y) : 0.f;   // an infinite sum stays one
        sum = t;
    }
};

// tcgen05.wait::ld, for 16 registers: what uses them comes behind it
FQ_DEV void tmem_wait_ld16(uint32_t* r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :
                 : "memory");
}

// The sum of 2^(c s + neg) over `columns` columns (a multiple of 32) of a score tile's row; of those, [lo, hi) count (PART: not all
// do).  16 columns are on their way from tensor memory while the 16 before are worked on.  s_free (if any) is told when
// the scores are read.
template <bool PART>
FQ_DEV float kw_row(uint32_t tS, uint64_t* s_free, const float* neg, uint64_t c2, int columns, int lo, int hi, int lane) {
    uint64_t acc[4] = {0, 0, 0, 0};
    uint32_t x[2][16];
    tmem_ld16(tS, x[0]);
#pragma unroll 1
    for (int h = 0; h < columns; h += 32) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            const int at = h + 16 * b;
            ulonglong2 m[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) m[k] = *reinterpret_cast<const ulonglong2*>(neg + at + 4 * k);
            [[maybe_unused]] uint32_t seen = 0;   // a bit per column
            if (PART) {
                const int from = max(0, min(16, lo - at)), to = max(0, min(16, hi - at));
                seen = (1u << to) - 1 >> from << from;
            }
            tmem_wait_ld16(x[b]);
            if (b == 0 || h + 32 < columns) {
                tmem_ld16(tS + at + 16, x[b ^ 1]);
            } else if (s_free) {   // the next scores may come
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free);
            }
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
                float p[4];
                unpair(fma2(pair(__uint_as_float(x[b][k]), __uint_as_float(x[b][k + 1])), c2, m[k >> 2].x), p[0], p[1]);
                unpair(fma2(pair(__uint_as_float(x[b][k + 2]), __uint_as_float(x[b][k + 3])), c2, m[k >> 2].y), p[2], p[3]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[e] = ex2(p[e]);
                    if (PART) p[e] = seen & 1u << (k + e) ? p[e] : 0.f;
                }
                acc[(k >> 1) & 3] = add2(acc[(k >> 1) & 3], pair(p[0], p[1]));
                acc[((k >> 1) & 3) + 1] = add2(acc[((k >> 1) & 3) + 1], pair(p[2], p[3]));
            }
        }
    }
    float a0, a1;
    unpair(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])), a0, a1);
    return a0 + a1;
}

// The packed rows of a sequence that see a key: [lo, hi), relative to query block b's first and kept near it.
struct KwRange {
    int lo, hi;
};
FQ_DEV KwRange kw_range(const AttnMask& m, const AttnSeq& sq, int key, int b, int shift) {
    constexpr int64_t FAR = 1 << 30;
    const int64_t p0 = (int64_t)b * KW_BLOCK;
    int64_t end = sq.q_len;
    if (key >= m.sinks) end = min(end, (int64_t)key + m.window - sq.off + 1);
    if (key >= sq.k_len) end = 0;
    const int64_t lo = (max((int64_t)0, (int64_t)key - sq.off + 1) << shift) - p0, hi = (max((int64_t)0, end) << shift) - p0;
    return KwRange{(int)max(-FAR, min(FAR, lo)), (int)max(-FAR, min(FAR, hi))};
}

// what a key had before (maybe where `after` is written)
FQ_DEV float kw_had(const KeyWeights& w, bool more, int head, int64_t row) {
    return more ? w.after[head * w.after_stride + row] : w.before ? w.before[head * w.before_stride + row] : 0.f;
}

template <class Args>
FQ_DEV void kw_sum(const Args& a, KwShared* sh, const uint8_t* stay, uint32_t tm, int wg, int row, int lane) {
    const int x = wg & 1, y = wg >> 1, shift = a.g_shift;
    const uint32_t lanes = (uint32_t)(row >> 5) << 21, tS = tm + KW_S + KW_BLOCK * wg + lanes;
    const uint64_t c2 = pair(a.c, a.c);
    uint32_t tile = 0, blk = 0, halves = 0;   // score tiles; query blocks of this y; units whose halves were added
    uint32_t un = 0, moved = 0;               // units with tiles; key tiles moved
    bool ok = true;
    KwUnit u;
    for (KwLine l = kw_line(a, blockIdx.x); ok && kw_next(a, l, u);) {
        const AttnSeq& sq = a.seq[u.seq];
        const KeyWeights& kw = a.w[Args::VIEWS == 1 ? 0 : sq.view];
        auto finish = [&](int key, float sum) {
            if (key >= sq.k_len) return;
            const int64_t r = sq.k_row0 + key;
            kw.after[u.head * kw.after_stride + r] = kw_had(kw, u.more, u.head, r) + sum;
        };
        if (u.kind == KW_NONE) {
            for (int64_t key = (int64_t)u.j0 * TILE_ROWS + TILE_ROWS * wg + row; key < min((int64_t)sq.k_len, (int64_t)u.j1 * TILE_ROWS); key += 4 * TILE_ROWS)
                finish((int)key, 0.f);
            continue;
        }
        // the statistics of the next query block of this y
        auto bring = [&]() {
            ok = kw_wait_warp(&sh->neg_full[y][blk & 1], (blk >> 1) & 1, sh);
            ++blk;
        };
        auto leave = [&](int s) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->neg_empty[y][s]);
        };
        auto score_tile = [&](int s, int columns, int lo, int hi, uint64_t* s_free) -> float {
            if (!(ok = kw_wait_warp(&sh->s_full[wg], tile & 1, sh))) return 0.f;
            ++tile;
            tc_fence_after();
            const float* neg = sh->neg[y][s];
            // (keys that see none of these rows beside keys that see all of them: a window's sinks)
            const bool all = lo <= 0 && hi >= columns, none = lo >= min(hi, columns) || hi <= 0;
            if (__all_sync(0xFFFFFFFFu, none)) {
                if (s_free) {
                    tc_fence_before();
                    if (lane == 0) mbar_arrive(s_free);
                }
                return 0.f;
            }
            if (__any_sync(0xFFFFFFFFu, !all && !none)) return kw_row<true>(tS, s_free, neg, c2, columns, lo, hi, lane);
            const float sum = kw_row<false>(tS, s_free, neg, c2, columns, lo, hi, lane);
            return none ? 0.f : sum;
        };
        if (u.kind == KW_ROWS) {
            ++un;
            const int s = blk & 1, columns = kw_columns(a, u);
            bring();
            for (int i = wg; i < u.pass && ok; i += 4) {
                const int key = (u.j0 + i) * TILE_ROWS + row;
                const KwRange r = kw_range(a.mask, sq, key, 0, shift);
                const float sum = score_tile(s, columns, r.lo, r.hi, &sh->s_free[wg]);
                if (ok) finish(key, sum);
            }
            if (!ok) break;
            leave(s);
            continue;
        }
        const int key = (u.j0 + x) * TILE_ROWS + row;
        const bool idle = x >= u.stay;
        const int set = un & 1, set_ph = un >> 1 & 1;
        ++un;
        if (y == 0 && !idle) {
            // The key tile to tensor memory, a row per thread.  (What held this place has been multiplied: this warpgroup had
            // all sums of the unit before.)
            if (!(ok = kw_wait_warp(&sh->k_go[x], moved++ & 1, sh) && kw_wait_warp(&sh->st_full[set], set_ph, sh))) break;
            const uint8_t* k_sm = stay + (2 * set + x) * KW_TILE_BYTES;
#pragma unroll 1
            for (int h = 0; h < 4; ++h) {   // 32 dims
                uint32_t v[16];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint4 t = *reinterpret_cast<const uint4*>(k_sm + (h >> 1) * KW_PANEL + sw128_offset(row, 4 * (h & 1) + j));
                    v[4 * j] = t.x;
                    v[4 * j + 1] = t.y;
                    v[4 * j + 2] = t.z;
                    v[4 * j + 3] = t.w;
                }
                tmem_st16(tm + KW_K + 64 * x + 16 * h + lanes, v);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->k_ready[x]);
        }
        KwRange r = kw_range(a.mask, sq, key, u.b0 + y, shift);
        Total total;
        for (int b = u.b0 + y; b < u.b1 && ok; b += 2, r.lo -= 2 * KW_BLOCK, r.hi -= 2 * KW_BLOCK) {
            const int s = blk & 1;
            bring();
            if (!ok) break;
            // (the last S buffer of y = 1 takes its sums first)
            if (!idle) total.add(score_tile(s, KW_BLOCK, r.lo, r.hi, y && b + 2 >= u.b1 ? nullptr : &sh->s_free[wg]));
            leave(s);
        }
        if (!ok) break;
        if (idle) continue;
        if (u.b0 + 1 < u.b1) {   // both have sums
            if (y) {
                tmem_st1(tS, total.sum);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->half_full[x]);
                continue;
            }
            if (!(ok = kw_wait_warp(&sh->half_full[x], halves++ & 1, sh))) break;
            tc_fence_after();
            float other = tmem_ld1(tm + KW_S + KW_BLOCK * (x + 2) + lanes);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->s_free[x + 2]);
            total.add(other);
        } else if (y) {
            continue;
        }
        if (u.slot < 0) finish(key, total.sum);
        else a.part[(int64_t)u.slot * (KW_KEY_TILES * TILE_ROWS) + x * TILE_ROWS + row] = total.sum;
    }
}

template <class Args>
__global__ void __launch_bounds__(KW_THREADS, 1) key_weights_kernel(const __grid_constant__ Args a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* stay = smem;
    uint8_t* ring = smem + 4 * KW_TILE_BYTES;
    KwShared* sh = reinterpret_cast<KwShared*>(ring + KW_RING * KW_TILE_BYTES);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_trigger();
    if (warp == 16) {
        if (lane == 0) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(&sh->st_full[i], 1);
                mbar_init(&sh->st_empty[i], 1);
                mbar_init(&sh->half_full[i], 4);
                mbar_init(&sh->k_go[i], 1);
                mbar_init(&sh->k_ready[i], 4);
                for (int b = 0; b < 2; ++b) {
                    mbar_init(&sh->neg_full[i][b], 1);
                    mbar_init(&sh->neg_empty[i][b], 8);
                    mbar_init(&sh->s_full[2 * i + b], 1);
                    mbar_init(&sh->s_free[2 * i + b], 4);
                }
            }
            for (int s = 0; s < KW_RING; ++s) {
                mbar_init(&sh->ring_full[s], 1);
                mbar_init(&sh->ring_empty[s], 1);
            }
            // the 128-byte swizzle wants 1024-byte aligned tiles
            sh->limit = (smem_u32(smem) & 1023) ? 0 : a.waits.limit;
            mbar_fence_init();
        }
        __syncwarp();
    } else if (warp == 17) {
        tmem_alloc(&sh->tmem, 512);
        tmem_relinquish();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sh->tmem;
    if (wait_limit(sh) != 0) {   // (not with a misaligned base)
        if (warp < 16) kw_sum(a, sh, stay, tm, warp >> 2, tid & 127, lane);
        else if (warp == 16) kw_load(a, sh, stay, ring);
        else if (warp == 18) kw_statistics(a, sh, lane);
        else if (elect_one()) kw_products(a, sh, stay, ring, tm);
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 17) tmem_dealloc(tm, 512);
    if (tid == 0 && wait_limit(sh) == 0) atomicAdd(a.waits.record, 1u);
}

// Sums of keys that several thread blocks have parts of, part after part.
template <class Args>
__global__ void __launch_bounds__(KW_KEY_TILES* TILE_ROWS) key_weights_join_kernel(const __grid_constant__ Args a) {
    const int i = blockIdx.x / a.Hkv, head = blockIdx.x - i * a.Hkv;
    const KwEntry& e = a.e[i];
    int c0 = 0, c1 = 0;
    if (!(e.info & (KW_ROWS | KW_NONE))) kw_parts(a, i, head, c0, c1);
    pdl_wait();   // the partial sums are written
    if (c0 == c1) return;
    const AttnSeq& sq = a.seq[e.info & 127];
    const KeyWeights& kw = a.w[Args::VIEWS == 1 ? 0 : sq.view];
    const int64_t key = (int64_t)e.j0 * TILE_ROWS + threadIdx.x;
    if (key >= sq.k_len || key >= (int64_t)e.j1 * TILE_ROWS) return;
    const int64_t row = sq.k_row0 + key;
    const float had = kw_had(kw, e.info & KW_MORE, head, row);
    float sum = 0.f;
#pragma unroll 4
    for (int c = c0; c <= c1; ++c) sum += a.part[(int64_t)(2 * c + (c == c0)) * (KW_KEY_TILES * TILE_ROWS) + threadIdx.x];
    kw.after[head * kw.after_stride + row] = had + sum;
}

}  // namespace

template <class Args>
static cudaError_t prepare() {
    return cudaFuncSetAttribute(key_weights_kernel<Args>, cudaFuncAttributeMaxDynamicSharedMemorySize, KW_SMEM);
}
cudaError_t key_weights_prepare() {
    cudaError_t e = prepare<KwArgs1S>();
    if (e == cudaSuccess) e = prepare<KwArgs1M>();
    if (e == cudaSuccess) e = prepare<KwArgs1>();
    return e != cudaSuccess ? e : prepare<KwArgsN>();
}

template <class Args>
void launch_key_weights(const Args& a, int grid, cudaStream_t s) {
    key_weights_kernel<Args><<<grid, KW_THREADS, KW_SMEM, s>>>(a);
}
template void launch_key_weights<KwArgs1S>(const KwArgs1S&, int, cudaStream_t);
template void launch_key_weights<KwArgs1M>(const KwArgs1M&, int, cudaStream_t);
template void launch_key_weights<KwArgs1>(const KwArgs1&, int, cudaStream_t);
template void launch_key_weights<KwArgsN>(const KwArgsN&, int, cudaStream_t);

template <class Args>
void launch_key_weights_join(const Args& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)((int64_t)a.n_entries * a.Hkv));
    cfg.blockDim = dim3(KW_KEY_TILES * TILE_ROWS);
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, key_weights_join_kernel<Args>, a);
}
template void launch_key_weights_join<KwArgs1S>(const KwArgs1S&, cudaStream_t);
template void launch_key_weights_join<KwArgs1M>(const KwArgs1M&, cudaStream_t);
template void launch_key_weights_join<KwArgs1>(const KwArgs1&, cudaStream_t);
template void launch_key_weights_join<KwArgsN>(const KwArgsN&, cudaStream_t);

}  // namespace fq
