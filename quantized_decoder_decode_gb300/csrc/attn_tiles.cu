// Attention of query tiles on the 5th-generation tensor cores (tcgen05, sm_103a): prompts, chunks
// of prompts behind cached rows, the shared prefix of a decode batch (few rows: attn_rows.cu).
//
// One pass over the keys per query tile of 128 packed rows (token, head of the kv head's group):
//   S = Q K^T (f32, tensor memory),  p = 2^(c S - c m - lift),  O += bf16(p) V,  l += p,
// c = scale log2(e), m a reference maximum per row.  m follows the running maximum only when that
// has grown by more than 2^8 = 256 (conditional rescaling, a published method: then O and l of the
// warp's rows are rescaled); until then p <= 2^(8 - lift), which bf16 and the f32 sums carry at the
// same relative precision.  lift = 9 + log2(keys): the weights of a row add up to less than 1, so that O, which is
// divided by l only at the end, stays below the largest |V| and does not overflow where the output is finite.
// What it costs is at the other end: weights below 2^(lift - 126) of the row's largest are zero.
//
// A work unit is a pair of query tiles over the same keys, or (few rows, short prompts) one tile
// whose key tiles alternate between the two softmax warpgroups and whose halves are joined at the
// end.  Either way the tensor cores work for one warpgroup while the other turns scores into
// weights; S is in registers before the weights are made, so one S buffer serves both in turn:
//   S_A | S_B, PV_A | S_A', PV_B | S_B', PV_A' | ...
// Tensor memory: S, P_A and P_B (the weights as bf16 pairs, the A operand of P V straight from
// there), O_A, O_B: 128 + 64 + 64 + 128 + 128 = all 512 columns.
// Shared memory: Q (2 x 32 KB), three 32 KB stages for K tiles and two for V tiles of 128 keys.
//
// Roles (512 threads, one CTA per SM, looping over its units):
//   warps 0-3, 4-7  softmax of tile A / B, one row per thread
//   warp 8          issues the products with K
//   warp 9          loads Q and K by TMA
//   warp 10         loads V by TMA; in tiles with keys that some row does not see a weight of 0 times
//                   NaN would still be NaN, so values that are not finite are taken out of the
//                   tile and noted per column with their first key; the rows that see that key get
//                   them back in their output.  (Tiles of finite values, the rule, are only scanned.)
//   warp 11         issues the products with V
//   warps 12-15     outputs, while the next unit's scores are made
// The two kinds of products have a warp each because issuing one blocks until the tensor cores take
// it: what a warp waits for between its products then costs the other kind nothing.  In a pair, P V of a
// score tile is issued behind the scores of the tile after the next: those are what a softmax warpgroup
// and the one S buffer wait for next, and beside P V they would take twice as long (8192 tokens 369
// -> 349 us, 333 tokens behind 7000 45.2 -> 43.1 us; in single units 2048 tokens would lose 0.5 us).
// Every wait is bounded; one that gives up records it, and all roles leave.
//
// What bounds it.  One prompt of 8192 tokens, 32 / 8 heads, 349 us (the products alone 283): a pair of
// 128 x 128 tiles is 2048 cycles of tensor work and takes 2800, as the S buffer goes round: 610 cycles
// for the product, 270 until the warpgroup sees it, 180 to load it, 300 until the next product begins,
// twice.  The softmax of a tile (1060 cycles of arithmetic, 600 of waits and stores) fits in that.  2048
// tokens, 16 / 8 heads, 23.5 us: 2.5 us until the first scores, 12 us of the 16 tiles of the longest unit (0.76 us
// each), 2 us for the last values, 1.7 us of outputs: 18.2; the other 5 (the start and end of the grid, and what
// two short units on one SM take more than a long one) are not told apart.
// Taken out again: the softmax warps as output warps (2048 tokens 24.7 -> 26.0 us), one
// loading warp for K and V in the order of their use (packed prompts 50 -> 54), three lanes of one warp
// that load Q, K and V each on their own (2 us more for 2048 tokens: a lane's turn comes too late),
// outputs transposed between lanes for longer stores (packed prompts 50 -> 71 us) or with the next dims read
// from tensor memory ahead of the stores (55), K tiles released by the softmax warps (8192 tokens 366 -> 373 us).

#include "attn.cuh"
#include "attn_plan.h"
#include "tc.cuh"

namespace fq {

namespace {

constexpr int AT_THREADS = 512;
// registers: 512 x 128 at launch = 256 x 184 (softmax: a row's 128 scores) + 128 x 56 + 128 x 88
constexpr int AT_REGS = 128, AT_REGS_SOFTMAX = 184, AT_REGS_ISSUE = 56, AT_REGS_OUT = 88;
static_assert(256 * AT_REGS_SOFTMAX + 128 * AT_REGS_ISSUE + 128 * AT_REGS_OUT <= AT_THREADS * AT_REGS, "registers");
constexpr int AT_KS = 3, AT_VS = 2;                       // stages for K and for V tiles
constexpr int AT_TILE_BYTES = TILE_ROWS * HEAD_DIM * 2;   // 32 KB
constexpr int AT_PANEL = AT_TILE_BYTES / 2;               // 64 dims of 128 rows
constexpr uint32_t AT_S = 0, AT_P = 128, AT_O = 256;      // tensor-memory columns: S, P_A, P_B (64 each), O_A, O_B

struct AtShared {
    uint64_t q_full[2], q_empty[2];   // per Q buffer: of tile A, of tile B; single units take them in turn
    // One warp consumes K tiles and another V tiles, and a phase bit tells a waiter only whether the
    // phase it waits for or the one before is the current one: each has stages of its own, so that it
    // has always seen the phase before.
    uint64_t k_full[AT_KS], k_empty[AT_KS], v_full[AT_VS], v_empty[AT_VS], v_raw[AT_VS];
    uint64_t s_full[2], s_free, p_full[2], o_done[2];    // per score tile
    uint64_t o_last[2], o_free[2], stat_full[2];         // per unit
    uint32_t tmem;
    uint32_t limit;                       // cycles that a wait may take; 0: one gave up, all roles leave
    uint32_t poison_unit;                 // unit number + 1 that the notes are of
    uint32_t scores_issued;               // score tiles whose products are issued
    uint16_t done[4];                     // units that each output warp has finished (a CTA has at most 1536 x 1024 / 152)
    float2 stat[2][TILE_ROWS];            // (m, l) of each row at the end of a unit
    uint16_t poison[3][HEAD_DIM];         // first key (from the unit's first partly seen tile) of +inf, -inf, NaN
};
constexpr int AT_SMEM = (2 + AT_KS + AT_VS) * AT_TILE_BYTES + 3072;
static_assert(sizeof(AtShared) <= 3072, "shared memory");
static_assert(AT_SMEM <= 232448, "shared memory");

__device__ uint32_t g_attn_waits;   // CTAs that gave up, of calls that name no other record

// One unit as every role sees it.
struct Unit {
    int seq, head, slot;          // slot: first partial block + 1, or 0
    bool single, small;
    int tok_a, tok_b, rows_a, rows_b;   // first token and packed rows of tile A / B
    int j0;                       // first key tile
    int n_a, n_b, nt;             // key tiles of warpgroup A / B, of the unit
    int jm;                       // first key tile with a key that some row does not see
    int step;                     // key tiles that a warpgroup's next one is further
    FQ_DEV int n(int x) const { return x ? n_b : n_a; }
};

// The unit of a CTA in its round r: forth and back over the list (longest first), so that the
// CTAs' sums come out nearly even (8192 tokens, 32 / 8 heads: 2% over the mean instead of 14%).
FQ_DEV int unit_at(int r) { return r * (int)gridDim.x + (int)(r & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x); }

template <class Args>
FQ_DEV Unit unit_of(const Args& a, int w) {
    Unit u;
    const int entry = (int)((uint64_t)(uint32_t)w * a.inv_hkv >> 31);   // w / Hkv
    const TileEntry& e = a.e[entry];
    const int tpt = TILE_ROWS >> a.g_shift;
    u.head = w - entry * a.io.Hkv;
    u.seq = e.info & 127;
    u.single = (e.info & TILE_SINGLE) != 0;
    u.small = (e.info & TILE_SMALL) != 0;
    u.slot = (int)(e.info >> TILE_SLOT_SHIFT);
    const AttnSeq& s = a.seq[u.seq];
    u.tok_a = e.tok0;
    u.tok_b = e.tok0 + (u.single ? 0 : tpt);
    u.j0 = e.j0;
    u.step = u.single ? 2 : 1;
    auto tiles = [&](int tok, int n_tok) {   // key tiles of the range that the tile's last row sees into
        const int last = min(s.k_len, tok + n_tok - 1 + s.off);
        return n_tok > 0 && last > 0 ? max(0, min(e.j1, (last + TILE_ROWS - 1) / TILE_ROWS) - e.j0) : 0;
    };
    const int ta = max(0, min(tpt, s.q_len - u.tok_a)), tb = max(0, min(tpt, s.q_len - u.tok_b));
    u.rows_a = ta << a.g_shift;
    u.rows_b = tb << a.g_shift;
    u.n_a = tiles(u.tok_a, ta);
    u.n_b = tiles(u.tok_b, tb);
    u.nt = max(u.n_a, u.n_b);
    if (u.single) {
        u.n_a = (u.nt + 1) / 2;
        u.n_b = u.nt / 2;
    }
    u.jm = max(0, min(s.k_len, u.tok_a + s.off)) / TILE_ROWS;
    return u;
}

// By one thread: a query tile, a K or V tile.
template <class Args>
FQ_DEV void load_q(const Args& a, int row, int head, uint8_t* dst, uint64_t* bar) {
    mbar_arrive_expect_tx(bar, AT_TILE_BYTES);
    tma_load_4d(dst, a.map_q, 0, 0, head, row, bar);
    tma_load_4d(dst + AT_PANEL, a.map_q, 64, 0, head, row, bar);
}
FQ_DEV void load_kv(const void* map, uint8_t* dst, int row, int head, uint64_t* bar) {
    mbar_arrive_expect_tx(bar, AT_TILE_BYTES);
    tma_load_3d(dst, map, 0, row, head, bar);
    tma_load_3d(dst + AT_PANEL, map, 64, row, head, bar);
}

FQ_DEV void give_up(AtShared* sh) {   // (recorded when all roles have left)
    *(volatile uint32_t*)&sh->limit = 0;
}
FQ_DEV uint32_t wait_limit(const AtShared* sh) { return *(const volatile uint32_t*)&sh->limit; }
// LONG: a wait for the end of a unit of other roles, which takes as long as the unit has keys.  What is
// bounded then is the time without a new score tile.
template <bool LONG = false>
FQ_DEV bool at_wait(uint64_t* bar, uint32_t parity, AtShared* sh) {
    if (mbar_try_wait(bar, parity)) return true;
    uint32_t t0 = (uint32_t)clock(), issued = 0xFFFFFFFFu;
    while (!mbar_try_wait(bar, parity)) {
        const uint32_t limit = wait_limit(sh);
        if ((uint32_t)clock() - t0 > limit) {
            if (LONG && limit && *(volatile uint32_t*)&sh->scores_issued != issued) {
                issued = *(volatile uint32_t*)&sh->scores_issued;
                t0 = (uint32_t)clock();
                continue;
            }
            if (limit) give_up(sh);
            return false;
        }
    }
    return true;
}
// The same by a whole warp, with one answer for all lanes.
template <bool LONG = false>
FQ_DEV bool at_wait_warp(uint64_t* bar, uint32_t parity, AtShared* sh) {
    return __all_sync(0xFFFFFFFFu, at_wait<LONG>(bar, parity, sh));
}
// The outputs of n units are written.
FQ_DEV bool units_done(uint32_t n, int lane, AtShared* sh) {
    const uint32_t t0 = (uint32_t)clock();
    while (!__all_sync(0xFFFFFFFFu, *(volatile uint16_t*)&sh->done[lane & 3] >= n)) {
        const uint32_t limit = wait_limit(sh);
        if (__any_sync(0xFFFFFFFFu, (uint32_t)clock() - t0 > limit)) {
            if (lane == 0 && limit) give_up(sh);
            return false;
        }
    }
    return true;
}
// The products of n score tiles are issued.
FQ_DEV bool scores_ahead(uint32_t n, AtShared* sh) {
    const uint32_t t0 = (uint32_t)clock();
    bool ok = true;
    while (ok && *(volatile uint32_t*)&sh->scores_issued < n) {
        const uint32_t limit = wait_limit(sh);
        ok = (uint32_t)clock() - t0 <= limit;
        if (!ok && limit) give_up(sh);
    }
    return __all_sync(0xFFFFFFFFu, ok);
}
constexpr long long DRAIN_CYCLES = 1 << 20;   // half a millisecond

FQ_DEV uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
// 32 bytes to a 32-byte (wide) or 16-byte aligned address
FQ_DEV void st_piece(uint8_t* p, const uint32_t* w, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                     "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}
template <int N>
FQ_DEV void set_regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
FQ_DEV void set_regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// No copy may still be landing when the CTA exits.  A role gave up after a quarter second of waiting;
// copies that were issued land within microseconds of that.
FQ_DEV void drain() {
    const long long t0 = clock64();
    while (clock64() - t0 < DRAIN_CYCLES) {
    }
}

// ---------------- warp 9: K and query tiles, each as soon as its buffer is free.  A unit's first K tiles
// go ahead of its query tiles, whose buffer may be the one that the unit before still reads.
// (The query tiles and the first K tile of the first unit are on their way already: their release may
// come before this warp gets here, so it is not waited for again.)
template <class Args>
FQ_DEV void load_keys(const Args& a, AtShared* sh, uint8_t* q_sm, uint8_t* ring, int units, bool preloaded) {
    uint32_t n = preloaded, it = 0;     // K tiles, units
    uint32_t sel = 0, qp = 0, qu = 0;   // buffer of the next single unit; phase bits of q_empty; buffers used
    bool ok = true;
    for (int w; (w = unit_at(it)) < units && ok; ++it) {
        const Unit u = unit_of(a, w);
        const AttnSeq& sq = a.seq[u.seq];
        if (u.nt == 0) continue;
        const bool pre = preloaded && it == 0;
        const int vw = Args::VIEWS == 1 ? 0 : sq.view;
        const int row0 = sq.k_row0 + u.j0 * TILE_ROWS;
        for (int t = pre ? 1 : 0; t <= u.nt && ok; ++t) {
            if (t == min(2, u.nt)) {
#pragma unroll 1
                for (int x = 0; x < (u.single ? 1 : 2) && ok; ++x) {
                    if (u.n(x) == 0) continue;
                    const uint32_t b = u.single ? sel : x;
                    if (!pre) {
                        if (!(ok = at_wait_warp(&sh->q_empty[b], ((qp >> b) & 1) ^ 1, sh))) break;
                        if (elect_one()) load_q(a, sq.q_row0 + (x ? u.tok_b : u.tok_a), u.head, q_sm + b * AT_TILE_BYTES, &sh->q_full[b]);
                        __syncwarp();
                    }
                    qp ^= 1u << b;
                    qu |= 1u << b;
                }
                if (u.single) sel ^= 1;
            }
            if (t == u.nt || !ok) break;
            const int s = n % AT_KS;
            if (!(ok = at_wait_warp(&sh->k_empty[s], ((n / AT_KS) & 1) ^ 1, sh))) break;
            ++n;
            if (elect_one() && !(a.waits.starve == 1 && it == 0 && t == 1))
                load_kv(a.map_k[vw], ring + s * AT_TILE_BYTES, row0 + t * TILE_ROWS, u.head, &sh->k_full[s]);
            __syncwarp();
        }
    }
    // The products' arrivals at these barriers come by themselves: the CTA's shared memory must not
    // be given to another CTA before the last of them.
#pragma unroll 1
    for (uint32_t i = n > AT_KS ? n - AT_KS : 0; i < n && ok; ++i) ok = at_wait_warp(&sh->k_empty[i % AT_KS], (i / AT_KS) & 1, sh);
#pragma unroll 1
    for (uint32_t b = 0; b < 2 && ok; ++b)
        if (qu >> b & 1) ok = at_wait_warp(&sh->q_empty[b], (qp >> b & 1) ^ 1, sh);
    if (!ok) drain();
}

// ---------------- warp 10: V tiles, and the check of those that some row sees in part
struct PartTile {
    uint32_t it;                   // its unit
    int s, tile, k_len, first, jm;   // stage, key tile; keys; keys that every row sees; the unit's first such tile
};

// Waits for a V tile and takes values that are not finite out of it.
FQ_DEV bool check_values(AtShared* sh, uint8_t* ring, const PartTile& p, uint32_t& raw_ph, int lane) {
    if (!at_wait_warp(&sh->v_raw[p.s], (raw_ph >> p.s) & 1, sh)) return false;
    raw_ph ^= 1u << p.s;
    uint8_t* tile = ring + (AT_KS + p.s) * AT_TILE_BYTES;
    // x * 0 is NaN where x is not finite (rows before `from` are seen by every row)
    const int from = max(0, p.first - p.tile * TILE_ROWS);
    uint32_t z[4] = {0, 0, 0, 0};
#pragma unroll 2
    for (int i = from * 8 + lane; i < TILE_ROWS * 8; i += 32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint4 v = reinterpret_cast<const uint4*>(tile + h * AT_PANEL)[i];
            z[0] = fma_bf16x2(v.x, 0u, z[0]);
            z[1] = fma_bf16x2(v.y, 0u, z[1]);
            z[2] = fma_bf16x2(v.z, 0u, z[2]);
            z[3] = fma_bf16x2(v.w, 0u, z[3]);
        }
    }
    bool odd = false;
#pragma unroll
    for (int h = 0; h < 4; ++h) odd |= (z[h] & 0x7FFF7FFFu) != 0;
    if (__any_sync(0xFFFFFFFFu, odd)) {
        if (*(volatile uint32_t*)&sh->poison_unit != p.it + 1) {
            if (!units_done(p.it, lane, sh)) return false;   // the notes before are read
            for (int i = lane; i < 3 * HEAD_DIM; i += 32) sh->poison[0][i] = 0xFFFFu;
            __syncwarp();
        }
        // lane l owns columns 4l .. 4l+3: 8 bytes of every row
        uint8_t* col = tile + (lane >> 4) * AT_PANEL;
#pragma unroll 1
        for (int r = from; r < TILE_ROWS; ++r) {
            uint16_t* v = reinterpret_cast<uint16_t*>(col + sw128_offset(r, (lane & 15) >> 1) + (lane & 1) * 8);
            const int key = p.tile * TILE_ROWS + r;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                const uint32_t b = v[c];
                if ((b & 0x7F80u) != 0x7F80u) continue;
                v[c] = 0;
                if (key >= p.k_len) continue;   // seen by no row
                uint16_t& f = sh->poison[(b & 0x7Fu) ? 2 : (b & 0x8000u) ? 1 : 0][4 * lane + c];
                const uint16_t k16 = (uint16_t)(key - p.jm * TILE_ROWS);
                if (k16 < f) f = k16;
            }
        }
        __syncwarp();
        if (lane == 0) *(volatile uint32_t*)&sh->poison_unit = p.it + 1;
        __threadfence_block();
        fence_async_smem();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->v_full[p.s]);
    return true;
}

template <class Args>
FQ_DEV void load_values(const Args& a, AtShared* sh, uint8_t* ring, int units, int lane) {
    uint32_t n = 0, raw_ph = 0;   // V tiles; phase bits of v_raw
    PartTile part[2];             // loaded and not checked yet: at most one per stage
    static_assert(AT_VS == 2, "two tiles to check at most");
    int pending = 0, it = -1, t = 0, vw = 0, row0 = 0, seen = 0, k_len = 0;
    bool more = true, ok = true;
    Unit u;
    u.nt = 0;
#pragma unroll 1
    while (ok) {
        while (more && t == u.nt) {   // the next unit
            const int w = unit_at(++it);
            more = w < units;
            if (!more) break;
            u = unit_of(a, w);
            const AttnSeq& sq = a.seq[u.seq];
            vw = Args::VIEWS == 1 ? 0 : sq.view;
            row0 = sq.k_row0 + u.j0 * TILE_ROWS;
            k_len = sq.k_len;
            seen = max(0, min(k_len, u.tok_a + sq.off));
            t = 0;
        }
        const int s = n % AT_VS;
        const uint32_t parity = ((n / AT_VS) & 1) ^ 1;
        // checks wait behind a load that can be issued, not behind one that cannot
        if (pending && !(more && __all_sync(0xFFFFFFFFu, mbar_test_wait(&sh->v_empty[s], parity)))) {
            ok = check_values(sh, ring, part[0], raw_ph, lane);
            part[0] = part[1];
            --pending;
            continue;
        }
        if (!more || !(ok = at_wait_warp(&sh->v_empty[s], parity, sh))) break;
        const bool whole = u.j0 + t < u.jm;
        if (elect_one() && !(a.waits.starve == 2 && it == 0 && t == 1))
            load_kv(a.map_v[vw], ring + (AT_KS + s) * AT_TILE_BYTES, row0 + t * TILE_ROWS, u.head,
                    whole ? &sh->v_full[s] : &sh->v_raw[s]);
        __syncwarp();
        if (!whole) {
            const PartTile p{(uint32_t)it, s, u.j0 + t, k_len, seen, u.jm};
            if (pending) part[1] = p;
            else part[0] = p;
            ++pending;
        }
        ++t;
        ++n;
    }
#pragma unroll 1
    for (uint32_t i = n > AT_VS ? n - AT_VS : 0; i < n && ok; ++i) ok = at_wait_warp(&sh->v_empty[i % AT_VS], (i / AT_VS) & 1, sh);
    if (!ok) drain();
}

// ---------------- warp 8: S = Q K^T
template <class Args>
FQ_DEV void scores(const Args& a, AtShared* sh, uint8_t* q_sm, uint8_t* ring, int units, uint32_t tm) {
    const uint32_t idesc = idesc_bf16_f32(TILE_ROWS, TILE_ROWS, false, a.negate != 0);
    const uint64_t dq0 = sdesc_sw128(smem_u32(q_sm)), dk0 = sdesc_sw128(smem_u32(ring));
    uint32_t kn = 0, qp = 0, sel = 0, sn = 0, it = 0;   // K tiles; phase bits of q_full; buffer of the next single unit; score tiles; units
    bool ok = true;
    for (int w; (w = unit_at(it)) < units && ok; ++it) {
        const Unit u = unit_of(a, w);
        if (u.nt == 0) continue;
        for (int t = 0; t < u.nt && ok; ++t) {
            const int s = kn % AT_KS;
            if (!(ok = at_wait_warp(&sh->k_full[s], (kn / AT_KS) & 1, sh))) break;
            ++kn;
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
                if (u.single ? x != (t & 1) : t >= u.n(x)) continue;
                const uint32_t b = u.single ? sel : x;   // the query tile's buffer
                if (t == 0) {
                    if (!(ok = at_wait_warp(&sh->q_full[b], (qp >> b) & 1, sh))) break;
                    qp ^= 1u << b;
                }
                // the scores before are in registers
                if (!(ok = at_wait_warp(&sh->s_free, (sn++ & 1) ^ 1, sh))) break;
                tc_fence_after();
                const uint64_t dq = dq0 + b * (uint32_t)(AT_TILE_BYTES >> 4);
                const uint64_t dk = dk0 + (uint32_t)(s * (AT_TILE_BYTES >> 4));
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t off = (k >> 2) * (AT_PANEL >> 4) + (k & 3) * 2;
                        mma_f16(tm + AT_S, dq + off, dk + off, idesc, k > 0);
                    }
                    mma_commit(&sh->s_full[x]);
                    *(volatile uint32_t*)&sh->scores_issued = sn;
                    if (t + 1 == (u.single ? u.nt : u.n(x))) mma_commit(&sh->q_empty[b]);
                }
                __syncwarp();
            }
            if (!ok) break;
            if (elect_one()) mma_commit(&sh->k_empty[s]);
            __syncwarp();
        }
        if (u.single) sel ^= 1;
    }
}

// ---------------- warp 11: O += P V
template <class Args>
FQ_DEV void values(const Args& a, AtShared* sh, uint8_t* ring, int units, uint32_t tm) {
    const uint32_t idesc = idesc_bf16_f32(TILE_ROWS, HEAD_DIM, true, false);
    const uint64_t dv0 = sdesc_sw128_mn(smem_u32(ring + AT_KS * AT_TILE_BYTES), AT_PANEL);
    uint32_t vn = 0, pc = 0, oc = 0, it = 0;   // V tiles; phase bits of p_full and o_free; units
    uint32_t n = 0, n_unit = 0;                // score tiles so far; up to the unit's end
    bool ok = true;
    for (int w; (w = unit_at(it)) < units && ok; ++it) {
        const Unit u = unit_of(a, w);
        n_unit += u.single ? u.nt : u.n_a + u.n_b;
        for (int t = 0; t < u.nt && ok; ++t) {
            const int s = vn % AT_VS;
            if (!(ok = at_wait_warp(&sh->v_full[s], (vn / AT_VS) & 1, sh))) break;
            ++vn;
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
                if (u.single ? x != (t & 1) : t >= u.n(x)) continue;
                const bool first = t < u.step, last = u.single ? t + 2 >= u.nt : t + 1 == u.n(x);
                if (first) {   // the unit before's outputs are read
                    if (!(ok = at_wait_warp(&sh->o_free[x], ((oc >> x) & 1) ^ 1, sh))) break;
                    oc ^= 1u << x;
                }
                ++n;
                if (!u.single && !(ok = scores_ahead(min(n + 2, n_unit), sh))) break;
                if (!(ok = at_wait_warp(&sh->p_full[x], (pc >> x) & 1, sh))) break;
                pc ^= 1u << x;

                tc_fence_after();
                const uint64_t dv = dv0 + (uint32_t)(s * (AT_TILE_BYTES >> 4));
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        mma_f16_ta(tm + AT_O + 128 * x, tm + AT_P + 64 * x + 8 * k, dv + (uint32_t)(k * (2048 >> 4)), idesc,
                                   k > 0 || !first);
                    mma_commit(&sh->o_done[x]);
                    if (last) mma_commit(&sh->o_last[x]);
                }
                __syncwarp();
            }
            if (!ok) break;
            if (elect_one()) mma_commit(&sh->v_empty[s]);
            __syncwarp();
        }
    }
}

// ---------------- warps 0-3 (x = 0), 4-7 (x = 1): softmax, thread = row
template <class Args>
FQ_DEV void softmax(const Args& a, AtShared* sh, int units, uint32_t tm, int x, int row, int lane) {
    const int g_shift = a.g_shift;
    const uint32_t lane_base = (uint32_t)(row >> 5) << 21;      // 32 lanes per warp, lane in bits 16..
    const uint32_t tS = tm + AT_S + lane_base, tP = tm + AT_P + 64 * x + lane_base, tO = tm + AT_O + 128 * x + lane_base;
    const float c = a.c;
    uint32_t sc = 0, it = 0;   // score tiles, units
    bool ok = true;
    for (int w; (w = unit_at(it)) < units && ok; ++it) {
        const Unit u = unit_of(a, w);
        const AttnSeq& sq = a.seq[u.seq];
        const int n = u.n(x);
        if (n == 0) continue;
        // keys that the row sees, from the unit's first (of this warpgroup) on
        int left = (row < (x ? u.rows_b : u.rows_a) ? max(0, min(sq.k_len, (x ? u.tok_b : u.tok_a) + (row >> g_shift) + sq.off)) : 0) -
                   (u.j0 + (u.single ? x : 0)) * TILE_ROWS;
        float m = -INFINITY, l = 0.f;
        for (int i = 0; i < n; ++i, left -= u.step * TILE_ROWS) {
            if (!(ok = at_wait_warp<true>(&sh->s_full[x], sc & 1, sh))) break;   // (its tile in the units before may have been empty)
            tc_fence_after();
            float s[TILE_ROWS];
#pragma unroll
            for (int h = 0; h < 4; ++h) tmem_ld32(tS + 32 * h, reinterpret_cast<uint32_t*>(s) + 32 * h);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->s_free);   // the next scores may come
            if (__any_sync(0xFFFFFFFFu, left < TILE_ROWS)) {
#pragma unroll
                for (int k = 0; k < TILE_ROWS; ++k) s[k] = k < left ? s[k] : -INFINITY;
            }
            float mx[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) mx[k] = fmaxf(s[k], s[4 + k]);
#pragma unroll
            for (int k = 8; k < TILE_ROWS; k += 2) mx[(k >> 1) & 3] = max3(mx[(k >> 1) & 3], s[k], s[k + 1]);
            const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
            // (a row without a key so far has m = -inf and moves at its first one)
            const bool move = (top - m) * c > 8.f;
            const float f = move ? ex2((m - top) * c) : 1.f;
            if (move) m = top;
            const float mc = m == -INFINITY ? 0.f : fmaf(m, c, a.io.lift);
            const uint64_t c2 = pair(c, c), mc2 = pair(-mc, -mc);
            uint64_t ls[2] = {0, 0};   // two pairs of partial sums
            uint32_t p[TILE_ROWS / 2];
#pragma unroll
            for (int k = 0; k < TILE_ROWS / 2; ++k) {
                float p0, p1;
                unpair(fma2(pair(s[2 * k], s[2 * k + 1]), c2, mc2), p0, p1);
                p0 = ex2(p0);
                p1 = ex2(p1);
                ls[k & 1] = add2(ls[k & 1], pair(p0, p1));
                p[k] = bf16x2(p0, p1);
            }
            // P V of the tile before has read P and written O: it ran beside the exponentials
            if (sc > 0) {
                if (!(ok = at_wait_warp(&sh->o_done[x], (sc - 1) & 1, sh))) break;
                tc_fence_after();
            }
            if (i > 0 && __any_sync(0xFFFFFFFFu, move)) {
#pragma unroll 1
                for (int h = 0; h < 8; ++h) {
                    uint32_t o[16];
                    tmem_ld16(tO + 16 * h, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
                    tmem_st16(tO + 16 * h, o);
                }
            }
#pragma unroll
            for (int h = 0; h < 4; ++h) tmem_st16(tP + 16 * h, p + 16 * h);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->p_full[x]);
            float l0, l1;
            unpair(add2(ls[0], ls[1]), l0, l1);
            l = fmaf(l, f, l0 + l1);
            ++sc;
        }
        if (!ok || !(ok = units_done(it, lane, sh))) break;   // the statistics before are read
        sh->stat[x][row] = make_float2(m, l);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->stat_full[x]);
    }
}

// ---------------- warps 12-15: outputs, thread = row
template <class Args>
FQ_DEV void outputs(const Args& a, AtShared* sh, int units, uint32_t tm, int row, int lane) {
    const int g_shift = a.g_shift;
    const uint32_t lane_base = (uint32_t)(row >> 5) << 21;
    const bool out_f32 = a.io.out_f32 != 0;
    const bool wide_out = ((reinterpret_cast<uintptr_t>(a.io.out) | (uintptr_t)(a.io.out_stride * (out_f32 ? 4 : 2))) & 31) == 0;
    uint32_t it = 0, uc = 0;   // units; phase bits of stat_full and o_last
    bool ok = true;
    for (int w; (w = unit_at(it)) < units && ok; ++it) {
        const Unit u = unit_of(a, w);
        const AttnSeq& sq = a.seq[u.seq];
        for (int x = 0; x < (u.single ? 1 : 2) && ok; ++x) {
            const int tok = (x ? u.tok_b : u.tok_a) + (row >> g_shift);
            const bool valid = row < (x ? u.rows_b : u.rows_a);
            const int limit = valid ? max(0, min(sq.k_len, tok + sq.off)) : 0;   // keys the row sees
            // the accumulator(s) of the rows: of the tile, or both of a single unit
            float m = -INFINITY, l = 0.f, f0 = 1.f, f1 = 0.f;
            const bool have = u.n(x) > 0, two = u.single && u.n_b > 0;
            for (int y = x; y <= (two ? 1 : x); ++y) {
                if (!have) break;
                if (!(ok = at_wait_warp<true>(&sh->stat_full[y], (uc >> y) & 1, sh) && at_wait_warp(&sh->o_last[y], (uc >> y) & 1, sh))) break;
                uc ^= 1u << y;
                const float2 st = sh->stat[y][row];
                if (y == x) {
                    m = st.x;
                    l = st.y;
                } else {
                    const float M = fmaxf(m, st.x);
                    f0 = m == M ? 1.f : ex2((m - M) * a.c);
                    f1 = st.x == M ? 1.f : ex2((st.x - M) * a.c);
                    l = l * f0 + st.y * f1;
                    m = M;
                }
            }
            if (!ok) break;
            tc_fence_after();
            if (!u.slot && limit > 0) {
                const float inv = 1.f / l;
                f0 *= inv;
                f1 *= inv;
            }
            const int64_t blk = (int64_t)(u.slot - 1 + x) * a.io.Hkv + u.head;   // partial block
            const int R = u.small ? SMALL_ROWS : TILE_ROWS;
            const bool f32 = u.slot || out_f32;
            uint8_t* part = (uint8_t*)((u.small ? a.part.b_o : a.part.a_o) + blk * HEAD_DIM * R + row * 8);
            uint8_t* out = (uint8_t*)a.io.out + ((int64_t)(sq.q_row0 + tok) * a.io.out_stride +
                                                 (int64_t)((u.head << g_shift) + (row & ((1 << g_shift) - 1))) * HEAD_DIM) *
                                                    (f32 ? 4 : 2);
            uint8_t* dst = u.slot ? part : out;
            const int64_t step = u.slot ? R * 32 : 32;   // between 32-byte pieces of the row
            const bool wide = u.slot || wide_out;
            const uint32_t t0 = tm + AT_O + lane_base + 128 * x;
            // (16 dims at a time in a short loop: its instructions are fetched anew for every unit)
#pragma unroll 1
            for (int h = __any_sync(0xFFFFFFFFu, valid) ? 0 : 8; h < 8; ++h) {
                uint32_t y[16];
                __syncwarp();
                if (have) {
                    tmem_ld16(t0 + 16 * h, y);
                    if (two) {
                        uint32_t y1[16];
                        tmem_ld16(t0 + 128 + 16 * h, y1);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            y[k] = __float_as_uint(fmaf(__uint_as_float(y1[k]), f1, __uint_as_float(y[k]) * f0));
                    } else {
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 16; ++k) y[k] = __float_as_uint(__uint_as_float(y[k]) * f0);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 16; ++k) y[k] = 0;
                }
                if (valid) {
                    if (f32) {
                        st_piece(dst, y, wide);
                        st_piece(dst + step, y + 8, wide);
                        dst += 2 * step;
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k) y[k] = bf16x2(__uint_as_float(y[2 * k]), __uint_as_float(y[2 * k + 1]));
                        st_piece(dst, y, wide);
                        dst += step;
                    }
                }
            }
            if (have) {   // the accumulators are read
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&sh->o_free[x]);
                    if (two) mbar_arrive(&sh->o_free[1]);
                }
            }
            if (valid && *(volatile uint32_t*)&sh->poison_unit == it + 1) {   // values that are not finite
                const int seen = limit - u.jm * TILE_ROWS;                     // noted keys below this are the row's
                dst = u.slot ? part : out;
#pragma unroll 1
                for (int d = 0; d < HEAD_DIM; ++d) {
                    const float add = (sh->poison[0][d] < seen ? INFINITY : 0.f) + (sh->poison[1][d] < seen ? -INFINITY : 0.f) +
                                      (sh->poison[2][d] < seen ? NAN : 0.f);
                    if (add == 0.f) continue;
                    uint8_t* at = dst + (f32 ? (d >> 3) * step + (d & 7) * 4 : d * 2);
                    if (f32) *(volatile float*)at += add;
                    else *(volatile uint16_t*)at = __bfloat16_as_ushort(__float2bfloat16_rn(bf2f(*(volatile uint16_t*)at) + add));
                }
            }
            if (u.slot && valid) (u.small ? a.part.b_ml : a.part.a_ml)[blk * R + row] = make_float2(m * a.c, l);
        }
        if (!ok) break;
        __syncwarp();
        __threadfence_block();
        if (lane == 0) *(volatile uint16_t*)&sh->done[row >> 5] = (uint16_t)(it + 1);
    }
}

template <class Args>
__global__ void __launch_bounds__(AT_THREADS, 1) attn_tiles_kernel(const __grid_constant__ Args a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* q_sm = smem;
    uint8_t* ring = smem + 2 * AT_TILE_BYTES;
    AtShared* sh = reinterpret_cast<AtShared*>(ring + (AT_KS + AT_VS) * AT_TILE_BYTES);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int units = a.n_entries * a.io.Hkv;

    bool preloaded = false;   // (warp 9)
    pdl_trigger();   // the kernel behind this one in the call may start beside it
    if (warp == 9) {
        if (lane == 0) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(&sh->q_full[i], 1);
                mbar_init(&sh->q_empty[i], 1);
            }
            for (int s = 0; s < AT_KS; ++s) {
                mbar_init(&sh->k_full[s], 1);
                mbar_init(&sh->k_empty[s], 1);
            }
            for (int s = 0; s < AT_VS; ++s) {
                mbar_init(&sh->v_full[s], 1);
                mbar_init(&sh->v_empty[s], 1);
                mbar_init(&sh->v_raw[s], 1);
            }
            mbar_init(&sh->s_free, 4);
            for (int x = 0; x < 2; ++x) {
                mbar_init(&sh->s_full[x], 1);
                mbar_init(&sh->p_full[x], 4);
                mbar_init(&sh->o_done[x], 1);
                mbar_init(&sh->o_last[x], 1);
                mbar_init(&sh->o_free[x], 4);
                mbar_init(&sh->stat_full[x], 4);
            }
            for (int i = 0; i < 4; ++i) sh->done[i] = 0;
            sh->poison_unit = 0;
            sh->scores_issued = 0;
            // the 128-byte swizzle wants 1024-byte aligned tiles
            sh->limit = (smem_u32(smem) & 1023) ? 0 : a.waits.limit;
            mbar_fence_init();
        }
        __syncwarp();
        // Q and the first K tile of the first unit, before the CTA meets
        const Unit u = unit_of(a, blockIdx.x);
        const AttnSeq& sq = a.seq[u.seq];
        const int vw = Args::VIEWS == 1 ? 0 : sq.view;
        const bool pre = u.nt > 0 && sh->limit != 0;
        if (pre && elect_one()) {
            if (u.n_a > 0) load_q(a, sq.q_row0 + u.tok_a, u.head, q_sm, &sh->q_full[0]);
            if (!u.single && u.n_b > 0) load_q(a, sq.q_row0 + u.tok_b, u.head, q_sm + AT_TILE_BYTES, &sh->q_full[1]);
            load_kv(a.map_k[vw], ring, sq.k_row0 + u.j0 * TILE_ROWS, u.head, &sh->k_full[0]);
        }
        preloaded = pre;
        __syncwarp();
    } else if (warp == 8) {
        tmem_alloc(&sh->tmem, 512);
        tmem_relinquish();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sh->tmem;
    const bool run = wait_limit(sh) != 0;   // (not with a misaligned base)
    if (warp < 8) {
        set_regs_up<AT_REGS_SOFTMAX>();
        if (run) softmax(a, sh, units, tm, warp >> 2, tid & 127, lane);
    } else if (warp < 12) {
        set_regs_down<AT_REGS_ISSUE>();
        if (run) {
            if (warp == 8) scores(a, sh, q_sm, ring, units, tm);
            else if (warp == 9) load_keys(a, sh, q_sm, ring, units, preloaded);
            else if (warp == 10) load_values(a, sh, ring, units, lane);
            else values(a, sh, ring, units, tm);
        }
    } else {
        set_regs_down<AT_REGS_OUT>();
        if (run) outputs(a, sh, units, tm, tid & 127, lane);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tm, 512);
    if (tid == 0 && wait_limit(sh) == 0) {
        if (a.waits.code) atomicOr(a.waits.record, a.waits.code);
        else atomicAdd(a.waits.record, 1u);
    }
}

template <class Args>
cudaError_t prepare_t() {
    cudaFuncAttributes fa;
    cudaError_t e = cudaFuncGetAttributes(&fa, attn_tiles_kernel<Args>);
    if (e != cudaSuccess) return e;
    if (fa.numRegs != AT_REGS) return cudaErrorInvalidKernelImage;   // the split would wait for registers that are not there
    return cudaFuncSetAttribute(attn_tiles_kernel<Args>, cudaFuncAttributeMaxDynamicSharedMemorySize, AT_SMEM);
}

}  // namespace

cudaError_t attn_tiles_prepare() {
    cudaError_t e = prepare_t<TileArgs1S>();
    if (e == cudaSuccess) e = prepare_t<TileArgs1>();
    if (e == cudaSuccess) e = prepare_t<TileArgsNS>();
    return e != cudaSuccess ? e : prepare_t<TileArgsN>();
}

template <class Args>
void launch_tiles(const Args& a, cudaStream_t s) {
    const int64_t units = (int64_t)a.n_entries * a.io.Hkv;
    const int grid = (int)(units < ATTN_SMS ? units : ATTN_SMS);
    attn_tiles_kernel<Args><<<grid, AT_THREADS, AT_SMEM, s>>>(a);
}
template void launch_tiles<TileArgs1S>(const TileArgs1S&, cudaStream_t);
template void launch_tiles<TileArgs1>(const TileArgs1&, cudaStream_t);
template void launch_tiles<TileArgsNS>(const TileArgsNS&, cudaStream_t);
template void launch_tiles<TileArgsN>(const TileArgsN&, cudaStream_t);

cudaError_t attn_wait_word(uint32_t** word) { return cudaGetSymbolAddress((void**)word, g_attn_waits); }

}  // namespace fq
