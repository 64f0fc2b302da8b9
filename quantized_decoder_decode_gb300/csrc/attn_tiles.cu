// Attention of query tiles on the 5th-generation tensor cores (tcgen05, sm_103a): prompts, chunks
// of prompts behind cached rows, and the shared prefix of a decode batch.
//
// One pass over the keys per query tile of 128 packed rows (token, head of the kv head's group):
//   S = Q K^T (f32, tensor memory),  p = 2^(c S - c m),  O += bf16(p) V,  l += p,
// c = scale log2(e), m a reference maximum per row.  m follows the running maximum only when that
// has grown by more than 2^8 = 256 (then O and l of the warp's rows are rescaled); until then
// p <= 256, which bf16 and the f32 sums carry at the same relative precision.
//
// A work unit is a pair of query tiles over the same keys, or (few rows) one tile whose key tiles
// alternate between the two softmax warpgroups, which are joined at the end.  Either way the
// tensor cores work for one warpgroup while the other turns scores into weights:
//   S_A | S_B | PV_A S_A' | PV_B S_B' | ...
// Tensor memory: S_A, S_B (128 columns each; the weights P overwrite the first 64 as bf16 pairs
// and are the A operand of P V straight from there), O_A, O_B (128 columns each): all 512.
// Shared memory: Q (2 x 32 KB), three 32 KB stages for K tiles and two for V tiles of 128 keys.
//
// Roles (384 threads, one CTA per SM, looping over its units):
//   warps 0-3, 4-7  softmax of tile A / B, one row per thread, and the outputs
//   warp 8          one thread issues the products
//   warp 9          one thread loads Q, K, V by TMA
//   warp 10         V tiles whose keys some row does not see: a weight of 0 times NaN would
//                   still be NaN, so values that are not finite are taken out of the tile and
//                   noted per column with their first key; the rows that see that key get them back
//                   in their output.  (Tiles of finite values, the rule, are only scanned.)
//   warp 11         idle
// Every wait is bounded; one that gives up records it, and all roles leave.

#include "attn_plan.h"
#include "common.cuh"
#include "tc.cuh"

namespace fq {

namespace {

constexpr int AT_THREADS = 384;
constexpr int AT_KS = 3, AT_VS = 2, AT_STAGES = AT_KS + AT_VS;   // stages for K and for V tiles
constexpr int AT_TILE_BYTES = TILE_ROWS * HEAD_DIM * 2;   // 32 KB
constexpr int AT_PANEL = AT_TILE_BYTES / 2;               // 64 dims of 128 rows
constexpr uint32_t AT_S = 0, AT_P = 128, AT_O = 256;      // tensor-memory columns: S, P_A, P_B (64 each), O_A, O_B

struct AtShared {
    uint64_t q_full, q_empty, join;
    // One warp consumes K tiles and another V tiles, and a phase bit tells a waiter only whether the
    // phase it waits for or the one before is the current one: each has stages of its own, so that it
    // has always seen the phase before.
    uint64_t k_full[AT_KS], k_empty[AT_KS], v_full[AT_VS], v_empty[AT_VS], v_raw[AT_VS];
    uint64_t s_full[2], p_full[2], o_done[2], s_free;
    uint32_t tmem, abort, preloaded;
    uint32_t done[8];                     // units that each softmax warp has finished
    uint32_t poison_unit[2];              // unit number + 1 whose notes the buffer holds
    float exchange[2][TILE_ROWS];
    uint16_t poison[2][3][HEAD_DIM];      // first key (from the unit's first partly seen tile) of +inf, -inf, NaN
};
constexpr int AT_SMEM = (2 + AT_STAGES) * AT_TILE_BYTES + 3072;
static_assert(sizeof(AtShared) <= 3072, "shared memory");
static_assert(AT_SMEM <= 232448, "shared memory");

__device__ uint32_t g_attn_waits;   // waits that gave up, since the last check

// One unit as every role sees it.
struct Unit {
    int seq, head, slot;          // slot: first partial block + 1, or 0
    bool single, small;
    int tok[2], n_tok[2];         // tokens of tile A / B
    int j0;                       // first key tile
    int n[2];                     // key tiles of warpgroup A / B
    int nt;                       // key tiles of the unit
    int jm;                       // first key tile with a key that some row does not see
    int step;
};

// The unit of a CTA in its round r: forth and back over the list (longest first), so that the
// CTAs' sums come out nearly even (8192 tokens, 32 / 8 heads: 2% over the mean instead of 14%).
FQ_DEV int unit_at(int r) { return r * (int)gridDim.x + (int)(r & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x); }

template <class Args>
FQ_DEV Unit unit_of(const Args& a, int w) {
    Unit u;
    const TileEntry& e = a.e[w / a.io.Hkv];
    const int G = a.io.Hq / a.io.Hkv, tpt = TILE_ROWS / G;
    u.head = w % a.io.Hkv;
    u.seq = e.info & 127;
    u.single = (e.info & TILE_SINGLE) != 0;
    u.small = (e.info & TILE_SMALL) != 0;
    u.slot = (int)(e.info >> TILE_SLOT_SHIFT);
    const AttnSeq& s = a.seq[u.seq];
    u.tok[0] = e.tok0;
    u.tok[1] = e.tok0 + (u.single ? 0 : tpt);
    u.j0 = e.j0;
    u.step = u.single ? 2 : 1;
    int tiles[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        u.n_tok[x] = max(0, min(tpt, s.q_len - u.tok[x]));
        const int last = min(s.k_len, u.tok[x] + u.n_tok[x] - 1 + s.off);   // keys the tile's last row sees
        tiles[x] = u.n_tok[x] > 0 && last > 0 ? max(0, min(e.j1, (last + TILE_ROWS - 1) / TILE_ROWS) - e.j0) : 0;
    }
    if (u.single) {
        u.nt = tiles[0];
        u.n[0] = (u.nt + 1) / 2;
        u.n[1] = u.nt / 2;
    } else {
        u.n[0] = tiles[0];
        u.n[1] = tiles[1];
        u.nt = max(tiles[0], tiles[1]);
    }
    u.jm = max(0, min(s.k_len, u.tok[0] + s.off)) / TILE_ROWS;
    return u;
}

// By one thread: the unit's query tiles; one K or V tile.
template <class Args>
FQ_DEV void load_q(const Args& a, const Unit& u, const AttnSeq& sq, uint8_t* q_sm, AtShared* sh) {
    const int q0 = u.n[0] > 0 ? 0 : 1, q1 = u.single || u.n[1] == 0 ? 1 : 2;
    mbar_arrive_expect_tx(&sh->q_full, (uint32_t)((q1 - q0) * AT_TILE_BYTES));
    for (int x = q0; x < q1; ++x) {
        const int row = sq.q_row0 + u.tok[x];
        tma_load_4d(q_sm + x * AT_TILE_BYTES, a.map_q, 0, 0, u.head, row, &sh->q_full);
        tma_load_4d(q_sm + x * AT_TILE_BYTES + AT_PANEL, a.map_q, 64, 0, u.head, row, &sh->q_full);
    }
}
FQ_DEV void load_kv(const void* map, uint8_t* dst, int row, int head, uint64_t* bar) {
    mbar_arrive_expect_tx(bar, AT_TILE_BYTES);
    tma_load_3d(dst, map, 0, row, head, bar);
    tma_load_3d(dst + AT_PANEL, map, 64, row, head, bar);
}

FQ_DEV bool at_wait(uint64_t* bar, uint32_t parity, AtShared* sh) {
    if (mbar_try_wait(bar, parity)) return true;
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity)) {
        if (*(volatile uint32_t*)&sh->abort) return false;
        if (clock64() - t0 > WAIT_BUDGET_CYCLES) {
            *(volatile uint32_t*)&sh->abort = 1;
            atomicAdd(&g_attn_waits, 1u);
            return false;
        }
    }
    return true;
}

// The same by a whole warp, with one answer for all lanes.
FQ_DEV bool at_wait_warp(uint64_t* bar, uint32_t parity, AtShared* sh) {
    return __all_sync(0xFFFFFFFFu, at_wait(bar, parity, sh));
}
// All softmax warps have finished n units (a count each: a warpgroup whose tile is empty may be
// units ahead of the other one, which no phase bit could tell).
FQ_DEV bool units_done(uint32_t n, int lane, AtShared* sh) {
    const long long t0 = clock64();
    while (!__all_sync(0xFFFFFFFFu, *(volatile uint32_t*)&sh->done[lane & 7] >= n)) {
        const bool late = clock64() - t0 > WAIT_BUDGET_CYCLES;
        if (__any_sync(0xFFFFFFFFu, late || *(volatile uint32_t*)&sh->abort)) {
            if (lane == 0 && late) {
                *(volatile uint32_t*)&sh->abort = 1;
                atomicAdd(&g_attn_waits, 1u);
            }
            return false;
        }
    }
    return true;
}
constexpr long long DRAIN_CYCLES = 1 << 20;   // half a millisecond
FQ_DEV uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
// 32 bytes to a 32-byte aligned address
FQ_DEV void st_global32(void* p, const uint32_t* v) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
// N pieces of 32 bytes, `step` bytes apart, at 32-byte (wide) or 16-byte aligned addresses
template <int N>
FQ_DEV void st_pieces(uint8_t* p, int64_t step, const uint32_t* v, bool wide) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (wide) {
            st_global32(p + k * step, v + 8 * k);
        } else {
            uint4* d = reinterpret_cast<uint4*>(p + k * step);
            d[0] = make_uint4(v[8 * k], v[8 * k + 1], v[8 * k + 2], v[8 * k + 3]);
            d[1] = make_uint4(v[8 * k + 4], v[8 * k + 5], v[8 * k + 6], v[8 * k + 7]);
        }
    }
}
template <int N>
FQ_DEV void set_regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
FQ_DEV void set_regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

template <class Args>
__global__ void __launch_bounds__(AT_THREADS, 1) attn_tiles_kernel(const __grid_constant__ Args a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* q_sm = smem;
    uint8_t* ring = smem + 2 * AT_TILE_BYTES;
    AtShared* sh = reinterpret_cast<AtShared*>(ring + AT_STAGES * AT_TILE_BYTES);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int units = a.n_entries * a.io.Hkv;
    const int G = a.io.Hq / a.io.Hkv;
    pdl_trigger();   // the kernels behind this one in the call may start beside it
    if (warp == 9) {
        // (the loads of the first unit start before the CTA meets)
        if (lane == 0) {
            mbar_init(&sh->q_full, 1);
            mbar_init(&sh->q_empty, 1);
            for (int i = 0; i < 8; ++i) sh->done[i] = 0;
            mbar_init(&sh->join, 8);
            mbar_init(&sh->s_free, 4);
            for (int s = 0; s < AT_KS; ++s) {
                mbar_init(&sh->k_full[s], 1);
                mbar_init(&sh->k_empty[s], 1);
            }
            for (int s = 0; s < AT_VS; ++s) {
                mbar_init(&sh->v_full[s], 1);
                mbar_init(&sh->v_empty[s], 1);
                mbar_init(&sh->v_raw[s], 1);
            }
            for (int x = 0; x < 2; ++x) {
                mbar_init(&sh->s_full[x], 1);
                mbar_init(&sh->p_full[x], 4);
                mbar_init(&sh->o_done[x], 1);
                sh->poison_unit[x] = 0;
            }
            // the 128-byte swizzle wants 1024-byte aligned tiles
            sh->abort = (smem_u32(smem) & 1023) ? 1 : 0;
            if (sh->abort) atomicAdd(&g_attn_waits, 1u);
            mbar_fence_init();
        }
        __syncwarp();
        const Unit u = unit_of(a, blockIdx.x);
        const AttnSeq& sq = a.seq[u.seq];
        const int vw = Args::VIEWS == 1 ? 0 : sq.view;
        const bool pre = u.nt > 0 && sh->abort == 0;
        if (pre && elect_one()) {
            load_q(a, u, sq, q_sm, sh);
            load_kv(a.map_k[vw], ring, sq.k_row0 + u.j0 * TILE_ROWS, u.head, &sh->k_full[0]);
        }
        if (lane == 0) sh->preloaded = pre;
        __syncwarp();
    } else if (warp == 8) {
        tmem_alloc(&sh->tmem, 512);
        tmem_relinquish();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sh->tmem;

    // registers: 384 x 168 at launch = 256 x 216 (softmax: a row's 128 scores) + 128 x 72
    const bool broken = *(volatile uint32_t*)&sh->abort != 0;   // (only with a misaligned base)
    if (warp >= 8) {
    set_regs_down<72>();
    if (broken) {
    } else if (warp == 9) {
        // ---------------- loads
        // Q and the first K tile of the first unit are on their way: neither is waited for again
        // here (their release may come before this warp gets to it)
        uint32_t kn = sh->preloaded, vn = 0, qn = sh->preloaded, it = 0;   // K and V tiles, Q tiles, units
        bool ok = true;
        for (int w; (w = unit_at(it)) < units && ok; ++it) {
            const Unit u = unit_of(a, w);
            const AttnSeq& sq = a.seq[u.seq];
            if (it >= 2 && !(ok = units_done(it - 1, lane, sh))) break;   // all but the unit before
            if (u.nt == 0) continue;
            const bool pre = it == 0;
            if (!pre) {
                if (!(ok = at_wait_warp(&sh->q_empty, (qn & 1) ^ 1, sh))) break;
                ++qn;
                if (elect_one()) load_q(a, u, sq, q_sm, sh);
                __syncwarp();
            }
            const int vw = Args::VIEWS == 1 ? 0 : sq.view;
            auto load_k = [&](int t) {
                const int s = kn % AT_KS;
                if (!(ok = at_wait_warp(&sh->k_empty[s], ((kn / AT_KS) & 1) ^ 1, sh))) return;
                ++kn;
                if (elect_one())
                    load_kv(a.map_k[vw], ring + s * AT_TILE_BYTES, sq.k_row0 + (u.j0 + t) * TILE_ROWS, u.head, &sh->k_full[s]);
                __syncwarp();
            };
            auto load_v = [&](int t) {
                const int s = vn % AT_VS;
                if (!(ok = at_wait_warp(&sh->v_empty[s], ((vn / AT_VS) & 1) ^ 1, sh))) return;
                ++vn;
                if (elect_one())
                    load_kv(a.map_v[vw], ring + (AT_KS + s) * AT_TILE_BYTES, sq.k_row0 + (u.j0 + t) * TILE_ROWS, u.head,
                            u.j0 + t >= u.jm ? &sh->v_raw[s] : &sh->v_full[s]);
                __syncwarp();
            };
            // in the order of their use: a pair makes the scores of one tile ahead of the values, a
            // single unit of two
            for (int t = pre ? 1 : 0; t < u.step && t < u.nt && ok; ++t) load_k(t);
            for (int t = 0; t < u.nt && ok; ++t) {
                if (t + u.step < u.nt) load_k(t + u.step);
                if (ok) load_v(t);
            }
        }
        // The products' arrivals at these barriers come by themselves: the CTA's shared memory must
        // not be given to another CTA before the last of them.
        for (uint32_t n = kn > AT_KS ? kn - AT_KS : 0; n < kn && ok; ++n)
            ok = at_wait_warp(&sh->k_empty[n % AT_KS], (n / AT_KS) & 1, sh);
        for (uint32_t n = vn > AT_VS ? vn - AT_VS : 0; n < vn && ok; ++n)
            ok = at_wait_warp(&sh->v_empty[n % AT_VS], (n / AT_VS) & 1, sh);
        if (qn && ok) ok = at_wait_warp(&sh->q_empty, (qn - 1) & 1, sh);
        if (!ok) {
            // No copy may still be landing when the CTA exits.  A role gave up after a quarter
            // second of waiting; copies that were issued land within microseconds of that.
            const long long t0 = clock64();
            while (clock64() - t0 < DRAIN_CYCLES) {
            }
        }
    } else if (warp == 8) {
        // ---------------- scores
        const uint32_t idesc = idesc_bf16_f32(TILE_ROWS, TILE_ROWS, false, a.negate != 0);
        const uint64_t dq0 = sdesc_sw128(smem_u32(q_sm)), dk0 = sdesc_sw128(smem_u32(ring));
        uint32_t kn = 0, qn = 0, sn = 0, it = 0;   // K tiles, Q tiles, score tiles, units
        bool ok = true;
        for (int w; (w = unit_at(it)) < units && ok; ++it) {
            const Unit u = unit_of(a, w);
            if (u.nt == 0) continue;
            if (!(ok = at_wait_warp(&sh->q_full, qn++ & 1, sh))) break;
            for (int t = 0; t < u.nt && ok; ++t) {
                const int s = kn % AT_KS;
                if (!(ok = at_wait_warp(&sh->k_full[s], (kn / AT_KS) & 1, sh))) break;
                ++kn;
                for (int x = 0; x < 2; ++x) {
                    if (u.single ? x != (t & 1) : t >= u.n[x]) continue;
                    // the scores before are in registers
                    if (!(ok = at_wait_warp(&sh->s_free, (sn++ & 1) ^ 1, sh))) break;
                    tc_fence_after();
                    const uint64_t dq = dq0 + (uint32_t)((u.single ? 0 : x) * (AT_TILE_BYTES >> 4));
                    const uint64_t dk = dk0 + (uint32_t)(s * (AT_TILE_BYTES >> 4));
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const uint32_t off = (k >> 2) * (AT_PANEL >> 4) + (k & 3) * 2;
                            mma_f16(tm + AT_S, dq + off, dk + off, idesc, k > 0);
                        }
                        mma_commit(&sh->s_full[x]);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (elect_one()) {
                    mma_commit(&sh->k_empty[s]);
                    if (t + 1 == u.nt) mma_commit(&sh->q_empty);
                }
                __syncwarp();
            }
        }
    } else if (warp == 11) {
        // ---------------- values
        const uint32_t idesc = idesc_bf16_f32(TILE_ROWS, HEAD_DIM, true, false);
        const uint64_t dv0 = sdesc_sw128_mn(smem_u32(ring + AT_KS * AT_TILE_BYTES), AT_PANEL);
        uint32_t vn = 0, pc = 0, it = 0;   // V tiles; pc: parities of p_full
        bool ok = true;
        for (int w; (w = unit_at(it)) < units && ok; ++it) {
            const Unit u = unit_of(a, w);
            for (int t = 0; t < u.nt && ok; ++t) {
                const int s = vn % AT_VS;
                if (!(ok = at_wait_warp(&sh->v_full[s], (vn / AT_VS) & 1, sh))) break;
                ++vn;
                for (int x = 0; x < 2; ++x) {
                    if (u.single ? x != (t & 1) : t >= u.n[x]) continue;
                    if (!(ok = at_wait_warp(&sh->p_full[x], (pc >> x) & 1, sh))) break;
                    pc ^= 1u << x;
                    tc_fence_after();
                    const uint64_t dv = dv0 + (uint32_t)(s * (AT_TILE_BYTES >> 4));
                    const uint32_t first = t < u.step ? 0u : 1u;
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            mma_f16_ta(tm + AT_O + 128 * x, tm + AT_P + 64 * x + 8 * k, dv + (uint32_t)(k * (2048 >> 4)), idesc,
                                       k > 0 ? 1u : first);
                        mma_commit(&sh->o_done[x]);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (elect_one()) mma_commit(&sh->v_empty[s]);
                __syncwarp();
            }
        }
    } else if (warp == 10) {
        // ---------------- partly seen V tiles
        uint32_t vn = 0, it = 0, raw_ph = 0;
        bool ok = true;
        for (int w; (w = unit_at(it)) < units && ok; ++it) {
            const Unit u = unit_of(a, w);
            const int k_len = a.seq[u.seq].k_len;
            for (int t = max(0, u.jm - u.j0); t < u.nt; ++t) {
                const int s = (vn + t) % AT_VS;
                if (!(ok = at_wait_warp(&sh->v_raw[s], (raw_ph >> s) & 1, sh))) break;
                raw_ph ^= 1u << s;
                uint8_t* tile = ring + (AT_KS + s) * AT_TILE_BYTES;
                // x * 0 is NaN where x is not finite (rows before `from` are seen by every row)
                const int from = max(0, min(k_len, u.tok[0] + a.seq[u.seq].off) - (u.j0 + t) * TILE_ROWS);
                uint32_t z[4] = {0, 0, 0, 0};
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
                for (int h = 0; h < 4; ++h) odd |= (z[h] & 0x7FFFu) != 0 || (z[h] & 0x7FFF0000u) != 0;
                if (__any_sync(0xFFFFFFFFu, odd)) {
                    const int buf = it & 1;
                    uint16_t(*note)[HEAD_DIM] = sh->poison[buf];
                    if (sh->poison_unit[buf] != it + 1) {
                        for (int i = lane; i < 3 * HEAD_DIM; i += 32) note[0][i] = 0xFFFFu;
                        __syncwarp();
                    }
                    // lane l owns columns 4l .. 4l+3: 8 bytes of every row
                    uint8_t* col = tile + (lane >> 4) * AT_PANEL;
                    for (int r = from; r < TILE_ROWS; ++r) {
                        uint16_t* p = reinterpret_cast<uint16_t*>(col + sw128_offset(r, (lane & 15) >> 1) + (lane & 1) * 8);
                        const int key = (u.j0 + t) * TILE_ROWS + r;
                        for (int c = 0; c < 4; ++c) {
                            const uint32_t b = p[c];
                            if ((b & 0x7F80u) != 0x7F80u) continue;
                            p[c] = 0;
                            if (key >= k_len) continue;   // seen by no row
                            uint16_t& f = note[(b & 0x7Fu) ? 2 : (b & 0x8000u) ? 1 : 0][4 * lane + c];
                            const uint16_t k16 = (uint16_t)(key - u.jm * TILE_ROWS);
                            if (k16 < f) f = k16;
                        }
                    }
                    __syncwarp();
                    if (lane == 0) *(volatile uint32_t*)&sh->poison_unit[buf] = it + 1;
                    __threadfence_block();
                    fence_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->v_full[s]);
            }
            vn += u.nt;
        }
    }
    } else {
    set_regs_up<216>();
    if (!broken) {
        // ---------------- softmax and outputs: thread = row
        const int x = warp >> 2, row = tid & 127;
        const uint32_t lane_base = (uint32_t)(warp & 3) << 21;      // 32 lanes per warp, lane in bits 16..
        const uint32_t tS = tm + AT_S + lane_base, tP = tm + AT_P + 64 * x + lane_base, tO = tm + AT_O + 128 * x + lane_base;
        const float c = a.c;
        const bool wide = ((reinterpret_cast<uintptr_t>(a.io.out) | (uintptr_t)(a.io.out_stride * (a.io.out_f32 ? 4 : 2))) & 31) == 0;
        uint32_t sc = 0, it = 0, jc = 0, oc = 0;   // score tiles, units, joins, products with V
        bool ok = true;
        // both warpgroups meet (a bounded wait, unlike a named barrier)
        auto join = [&]() -> bool {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->join);
            const bool met = at_wait_warp(&sh->join, jc++ & 1, sh);
            tc_fence_after();
            return met;
        };
        for (int w; (w = unit_at(it)) < units && ok; ++it) {
            const Unit u = unit_of(a, w);
            const AttnSeq& sq = a.seq[u.seq];
            const int tok = u.tok[x] + row / G;
            const bool valid = row / G < u.n_tok[x];
            const int limit = valid ? max(0, min(sq.k_len, tok + sq.off)) : 0;   // keys the row sees
            float m = -INFINITY, l = 0.f;
            for (int i = 0; i < u.n[x]; ++i) {
                if (!(ok = at_wait_warp(&sh->s_full[x], sc & 1, sh))) break;
                tc_fence_after();
                float s[TILE_ROWS];
#pragma unroll
                for (int h = 0; h < 4; ++h) tmem_ld32(tS + 32 * h, reinterpret_cast<uint32_t*>(s) + 32 * h);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->s_free);   // the other tile's scores may come
                const int left = limit - (u.j0 + (u.single ? 2 * i + x : i)) * TILE_ROWS;   // keys of this tile that the row sees
                if (__any_sync(0xFFFFFFFFu, left < TILE_ROWS)) {
#pragma unroll
                    for (int k = 0; k < TILE_ROWS; ++k) s[k] = k < left ? s[k] : -INFINITY;
                }
                // One pass over the scores: weights against the reference m, while the maximum is
                // taken for the check of m; the rare tile whose maximum is too far above goes
                // through twice.  A unit's first tile takes its maximum first.
                if (i == 0) {
                    float mx[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) mx[k] = fmaxf(s[k], s[4 + k]);
#pragma unroll
                    for (int k = 8; k < TILE_ROWS; k += 2) mx[(k >> 1) & 3] = max3(mx[(k >> 1) & 3], s[k], s[k + 1]);
                    m = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
                }
                if (i > 0) {   // P V of the tile before has read P and written O
                    if (!(ok = at_wait_warp(&sh->o_done[x], oc++ & 1, sh))) break;
                    tc_fence_after();
                }
                uint64_t ls[2];
                for (;;) {
                    const float mc = m == -INFINITY ? 0.f : m * c;
                    const uint64_t c2 = pair(c, c), mc2 = pair(-mc, -mc);
                    float mx[2] = {-INFINITY, -INFINITY};
                    ls[0] = ls[1] = 0;   // two pairs of partial sums
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        uint32_t p[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const float s0 = s[32 * h + 2 * k], s1 = s[32 * h + 2 * k + 1];
                            float p0, p1;
                            unpair(fma2(pair(s0, s1), c2, mc2), p0, p1);
                            p0 = ex2(p0);
                            p1 = ex2(p1);
                            mx[k & 1] = max3(mx[k & 1], s0, s1);
                            ls[k & 1] = add2(ls[k & 1], pair(p0, p1));
                            p[k] = bf16x2(p0, p1);
                        }
                        tmem_st16(tP + 16 * h, p);
                    }
                    // (a row without a key so far has m = -inf and moves at its first one)
                    const float top = fmaxf(mx[0], mx[1]);
                    const bool move = (top - m) * c > 8.f;
                    if (!__any_sync(0xFFFFFFFFu, move)) break;
                    const float f = move ? ex2((m - top) * c) : 1.f;
                    if (move) m = top;
                    l *= f;
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
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->p_full[x]);
                float l0, l1;
                unpair(add2(ls[0], ls[1]), l0, l1);
                l += l0 + l1;
                ++sc;
            }
            if (!ok) break;
            if (u.n[x] > 0) {
                if (!(ok = at_wait_warp(&sh->o_done[x], oc++ & 1, sh))) break;
                tc_fence_after();
            }
            // weights of the tile's accumulator(s): single units join A and B here, A's threads
            // writing dims 0-63 and B's 64-127 of the same rows
            float f0 = 1.f, f1 = 0.f, lsum = l, mref = m;
            if (u.single) {
                sh->exchange[x][row] = m;
                if (!(ok = join())) break;
                const float mo = sh->exchange[x ^ 1][row];
                if (!(ok = join())) break;
                mref = fmaxf(m, mo);
                const float own = m == mref ? 1.f : ex2((m - mref) * c), other = mo == mref ? 1.f : ex2((mo - mref) * c);
                sh->exchange[x][row] = l * own;
                if (!(ok = join())) break;
                lsum = l * own + sh->exchange[x ^ 1][row];
                f0 = x == 0 ? own : other;    // weight of O_A
                f1 = x == 0 ? other : own;    // weight of O_B
                if (u.nt == 1) f1 = 0.f;
            }
            const bool noted = *(volatile uint32_t*)&sh->poison_unit[it & 1] == it + 1;
            const int seen = limit - u.jm * TILE_ROWS;   // noted keys below this are the row's
            const float inv = u.slot || limit == 0 ? 1.f : 1.f / lsum;
            f0 *= inv;
            f1 *= inv;
            // where the row goes, 32 dims at a time: 32-byte pieces `step` bytes apart
            const int64_t blk = (int64_t)(u.slot - 1 + (u.single ? 0 : x)) * a.io.Hkv + u.head;   // partial block
            const int R = u.small ? SMALL_ROWS : TILE_ROWS;
            const int d0 = u.single ? 64 * x : 0;
            const bool f32 = u.slot || a.io.out_f32;
            uint8_t* dst = u.slot ? (uint8_t*)((u.small ? a.part.b_o : a.part.a_o) + (blk * HEAD_DIM + d0) * R + row * 8)
                                  : (uint8_t*)a.io.out + ((int64_t)(sq.q_row0 + tok) * a.io.out_stride +
                                                          (int64_t)(u.head * G + row % G) * HEAD_DIM + d0) * (f32 ? 4 : 2);
            const int64_t step = u.slot ? R * 32 : 32;
            const bool wide32 = u.slot || wide;
            const bool have = u.single ? u.nt > 0 : u.n[x] > 0, two = u.single && u.nt > 1;
            const uint32_t t0 = tm + AT_O + lane_base + (u.single ? 0 : 128 * x) + d0;
            // (a short loop: its instructions are fetched anew for every unit)
#pragma unroll 1
            for (int h = 0; h < (u.single ? 2 : 4); ++h) {
                uint32_t o[32];
                __syncwarp();
                if (have) {
                    tmem_ld32(t0 + 32 * h, o);
                    tmem_wait_ld();
                    if (two) {
                        uint32_t o1[32];
                        tmem_ld32(t0 + 128 + 32 * h, o1);
                        tmem_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            o[k] = __float_as_uint(fmaf(__uint_as_float(o1[k]), f1, __uint_as_float(o[k]) * f0));
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f0);
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = 0;
                }
                if (valid) {
                    if (f32) {
                        st_pieces<4>(dst, step, o, wide32);
                        dst += 4 * step;
                    } else {
#pragma unroll
                        for (int k = 0; k < 16; ++k) o[k] = bf16x2(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1]));
                        st_pieces<2>(dst, step, o, wide32);
                        dst += 2 * step;
                    }
                }
            }
            if (noted && valid) {   // values that are not finite, for the rows that see them
                const int dn = u.single ? 64 : HEAD_DIM;
                dst -= dn / 8 * step / (f32 ? 1 : 2);
                for (int d = 0; d < dn; ++d) {
                    const uint16_t(*note)[HEAD_DIM] = sh->poison[it & 1];
                    const float add = (note[0][d0 + d] < seen ? INFINITY : 0.f) + (note[1][d0 + d] < seen ? -INFINITY : 0.f) +
                                      (note[2][d0 + d] < seen ? NAN : 0.f);
                    if (add == 0.f) continue;
                    uint8_t* at = dst + (f32 ? (d >> 3) * step + (d & 7) * 4 : (d >> 4) * step + (d & 15) * 2);
                    if (f32) *(float*)at += add;
                    else *(__nv_bfloat16*)at = __float2bfloat16_rn(__bfloat162float(*(__nv_bfloat16*)at) + add);
                }
            }
            if (u.slot && valid && (!u.single || x == 0))
                (u.small ? a.part.b_ml : a.part.a_ml)[blk * R + row] = make_float2(mref * c, lsum);
            // the next unit's products may overwrite O once both warpgroups have read it
            tc_fence_before();
            if (u.single && !(ok = join())) break;
            __threadfence_block();
            __syncwarp();
            if (lane == 0) *(volatile uint32_t*)&sh->done[warp] = it + 1;
        }
    }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 8) tmem_dealloc(tm, 512);
}

constexpr int AT_REGS = 168;   // what the register split above draws on

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
template void launch_tiles<TileArgsNS>(const TileArgsNS&, cudaStream_t);
template void launch_tiles<TileArgs1>(const TileArgs1&, cudaStream_t);
template void launch_tiles<TileArgsN>(const TileArgsN&, cudaStream_t);

// Waits that gave up on the current device, read (and cleared) after the work queued on s.
cudaError_t attn_wait_record(uint32_t* host, cudaStream_t s) {
    cudaError_t e = cudaMemcpyFromSymbolAsync(host, g_attn_waits, sizeof(uint32_t), 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e != cudaSuccess || *host == 0) return e;
    const uint32_t zero = 0;
    e = cudaMemcpyToSymbolAsync(g_attn_waits, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, s);
    return e == cudaSuccess ? cudaStreamSynchronize(s) : e;
}

}  // namespace fq
