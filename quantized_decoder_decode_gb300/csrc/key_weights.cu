// The attention weight that every key receives, on the 5th-generation tensor cores (tcgen05, sm_103a):
//   after[j] = before[j] + sum over query rows i (and the heads of the group) that see key j of 2^(c q_i.k_j - lse_i log2(e)),
// c = scale log2(e), lse_i the log-sum that the attention of the same rows left.
//
// The scores are taken the other way round than in attention, S = K Q^T with the keys as the rows of the product: a
// thread then has one key's scores in its own lane of tensor memory and adds their exponentials up by itself.  No
// maximum is needed, no weight leaves the registers, and no two threads write the same sum (atomics would add
// in any order).  Sums of a tile of 128 weights go to the key's total by compensated addition: 2^15 rows add up as exactly
// as one tile does.
//
// A unit holds what is few and lets the rest pass by through a ring of 32 KB tiles (TMA):
//   KW_KEYS  two key tiles stay (one for each of the two warpgroups), query blocks of 128 packed rows pass by;
//   KW_ROWS  up to two query blocks stay (single tokens, a few observed rows), key tiles pass by, to the two
//            warpgroups in turn: K is read once, which is what bounds it.
// What stays has two sets of buffers, so that the next unit's comes while this one is worked on.  Long ranges of query
// blocks are cut into units of their own, whose partial sums (4 bytes a key) a second kernel adds up in order.
//
// Tensor memory: two S buffers of 128 columns for each warpgroup.  Shared memory: 2 x 2 tiles that stay, 3 that pass by.
// Roles (320 threads, one CTA per SM, looping over its units): warps 0-3 and 4-7 exponentials and sums, a key per thread; warp
// 8 loads; warp 9 issues the products.  Every wait is bounded; one that gives up records it, and all roles leave.

#include <cstddef>

#include "attn.cuh"
#include "cache_plan.h"
#include "tc.cuh"

namespace fq {

namespace {

constexpr int KW_THREADS = 320;
constexpr int KW_RING = 3;
constexpr int KW_TILE_BYTES = TILE_ROWS * HEAD_DIM * 2;   // 32 KB
constexpr int KW_PANEL = KW_TILE_BYTES / 2;               // 64 dims of 128 rows

struct KwShared {
    uint64_t st_full[2], st_empty[2];              // per set of tiles that stay
    uint64_t ring_full[KW_RING], ring_empty[KW_RING];
    uint64_t s_full[2][2], s_free[2][2];           // per warpgroup and S buffer
    uint64_t neg_full[2][2];                       // per warpgroup and buffer of statistics
    uint32_t tmem;
    uint32_t limit;                                // cycles that a wait may take; 0: one gave up, all roles leave
    alignas(16) float neg[2][2][TILE_ROWS];        // (read 16 bytes at a time) -lse log2(e) of a query block's rows: per warpgroup, two in turn
};
constexpr int KW_SMEM = (4 + KW_RING) * KW_TILE_BYTES + 3072;
static_assert(sizeof(KwShared) <= 3072 && KW_SMEM <= 232448, "shared memory");
static_assert(offsetof(KwShared, neg) % 16 == 0, "16-byte reads");

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

// One unit as every role sees it.
struct KwUnit {
    int seq, head, kind, j0, j1, b0, b1, slot;
    int stay, pass;       // tiles that stay; that pass by
};
FQ_DEV int kw_unit_at(int r) { return r * (int)gridDim.x + (int)(r & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x); }
template <class Args>
FQ_DEV KwUnit kw_unit(const Args& a, int w) {
    KwUnit u;
    const int entry = w / a.Hkv;
    const KwEntry& e = a.e[entry];
    u.head = w - entry * a.Hkv;
    u.seq = e.info & 127;
    u.kind = e.info & (KW_ROWS | KW_NONE);
    u.j0 = e.j0;
    u.j1 = e.j1;
    u.b0 = e.b0;
    u.b1 = e.b1;
    u.slot = e.slot;
    u.stay = u.kind == KW_NONE ? 0 : u.kind == KW_ROWS ? u.b1 - u.b0 : u.j1 - u.j0;
    u.pass = u.kind == KW_NONE ? 0 : u.kind == KW_ROWS ? u.j1 - u.j0 : u.b1 - u.b0;
    return u;
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
    const int row = a.seq[u.seq].q_row0 + (b * TILE_ROWS >> a.g_shift);
    tma_load_4d(dst, a.map_q, 0, 0, u.head, row, bar);
    tma_load_4d(dst + KW_PANEL, a.map_q, 64, 0, u.head, row, bar);
}

// Columns of a product with query block b: packed rows, in steps of 32 where the block stays.
template <class Args>
FQ_DEV int kw_columns(const Args& a, const KwUnit& u, int b) {
    if (u.kind == KW_KEYS) return TILE_ROWS;
    return min(TILE_ROWS, ((a.seq[u.seq].q_len << a.g_shift) - b * TILE_ROWS + 31) & ~31);
}

// ---------------- warp 8
template <class Args>
FQ_DEV void kw_load(const Args& a, KwShared* sh, uint8_t* stay, uint8_t* ring, int units) {
    uint32_t n = 0, un = 0;   // tiles that pass by; units with tiles
    bool ok = true;
    for (int it = 0, w; (w = kw_unit_at(it)) < units && ok; ++it) {
        const KwUnit u = kw_unit(a, w);
        if (!u.pass) continue;
        const int set = un & 1;
        if (!(ok = kw_wait_warp(&sh->st_empty[set], ((un >> 1) & 1) ^ 1, sh))) break;
        ++un;
        if (elect_one()) {
            mbar_arrive_expect_tx(&sh->st_full[set], u.stay * KW_TILE_BYTES);
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
                mbar_arrive_expect_tx(&sh->ring_full[s], KW_TILE_BYTES);
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

// ---------------- warp 9
template <class Args>
FQ_DEV void kw_products(const Args& a, KwShared* sh, uint8_t* stay, uint8_t* ring, int units, uint32_t tm) {
    const uint64_t d_stay = sdesc_sw128(smem_u32(stay)), d_ring = sdesc_sw128(smem_u32(ring));
    uint32_t n = 0, un = 0, tiles[2] = {0, 0};   // tiles that passed; units; score tiles of a warpgroup
    bool ok = true;
    for (int it = 0, w; (w = kw_unit_at(it)) < units && ok; ++it) {
        const KwUnit u = kw_unit(a, w);
        if (!u.pass) continue;
        const int set = un & 1;
        if (!(ok = kw_wait_warp(&sh->st_full[set], (un >> 1) & 1, sh))) break;
        ++un;
        for (int i = 0; i < u.pass && ok; ++i, ++n) {
            const int s = n % KW_RING;
            if (!(ok = kw_wait_warp(&sh->ring_full[s], (n / KW_RING) & 1, sh))) break;
#pragma unroll 1
            for (int x = 0; x < u.stay; ++x) {
                const int g = u.kind == KW_ROWS ? i & 1 : x;   // the warpgroup
                const uint32_t t = g ? tiles[1]++ : tiles[0]++;
                if (!(ok = kw_wait_warp(&sh->s_free[g][t & 1], ((t >> 1) & 1) ^ 1, sh))) break;
                tc_fence_after();
                const uint64_t dx = d_stay + (uint32_t)((2 * set + x) * (KW_TILE_BYTES >> 4)), dr = d_ring + (uint32_t)(s * (KW_TILE_BYTES >> 4));
                const uint64_t dk = u.kind == KW_ROWS ? dr : dx, dq = u.kind == KW_ROWS ? dx : dr;
                const uint32_t idesc = idesc_bf16_f32(TILE_ROWS, kw_columns(a, u, u.b0 + x), false, a.negate != 0);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t off = (k >> 2) * (KW_PANEL >> 4) + (k & 3) * 2;
                        mma_f16(tm + 256 * g + 128 * (t & 1), dk + off, dq + off, idesc, k > 0);
                    }
                    mma_commit(&sh->s_full[g][t & 1]);
                }
                __syncwarp();
            }
            if (!ok) break;
            if (elect_one()) {
                mma_commit(&sh->ring_empty[s]);
                if (i + 1 == u.pass) mma_commit(&sh->st_empty[set]);
            }
            __syncwarp();
        }
    }
}

// ---------------- warps 0-3 (g = 0), 4-7 (g = 1)
// A number with the rounding errors of its additions beside it (compensated summation).
struct Total {
    float sum = 0.f, err = 0.f;
    FQ_DEV void add(float x) {
        const float y = __fsub_rn(x, err), t = __fadd_rn(sum, y);
        err = __fsub_rn(__fsub_rn(t, sum), y);
        sum = t;
    }
};

// (in order with the loads around them: the compiler would fetch a whole tile's at once, and spill)
FQ_DEV void lds_pairs(const float* p, uint64_t& a, uint64_t& b) {
    asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(smem_u32(p)));
}
// tcgen05.wait::ld for 32 registers: what uses them comes behind it
FQ_DEV void tmem_wait_ld32(uint32_t* r) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                   "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                   "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                   "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29])
                 :
                 : "memory");
    asm volatile("" : "+r"(r[30]), "+r"(r[31]));
}

// The sum of 2^(c s + neg) over the columns [lo, hi) of a score tile's row (PART: they are not all).
template <bool PART>
FQ_DEV float kw_row(uint32_t tS, uint64_t* s_free, const float* neg, uint64_t c2, int columns, int lo, int hi, int lane) {
    uint64_t acc[4] = {0, 0, 0, 0};
    uint32_t s[2][32];
    tmem_ld32(tS, s[0]);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        if (32 * h < columns) {
            tmem_wait_ld32(s[h & 1]);
            if (32 * (h + 1) < columns) {
                if (h < 3) tmem_ld32(tS + 32 * (h + 1), s[(h + 1) & 1]);
            } else {   // the next scores may come
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(s_free);
            }
            const uint32_t* x = s[h & 1];
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
                uint64_t m0, m1;
                float p[4];
                lds_pairs(neg + 32 * h + k, m0, m1);
                unpair(fma2(pair(__uint_as_float(x[k]), __uint_as_float(x[k + 1])), c2, m0), p[0], p[1]);
                unpair(fma2(pair(__uint_as_float(x[k + 2]), __uint_as_float(x[k + 3])), c2, m1), p[2], p[3]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[e] = ex2(p[e]);
                    if (PART) p[e] = 32 * h + k + e >= lo && 32 * h + k + e < hi ? p[e] : 0.f;
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

template <class Args>
FQ_DEV void kw_sum(const Args& a, KwShared* sh, int units, uint32_t tm, int g, int row, int lane) {
    constexpr float LOG2E = 1.4426950408889634f;
    const int shift = a.g_shift, G = 1 << shift;
    const uint32_t tS = tm + 256 * g + ((uint32_t)(row >> 5) << 21);
    const uint64_t c2 = pair(a.c, a.c);
    uint32_t tile = 0, blk = 0;   // score tiles; buffers of statistics filled
    bool ok = true;
    for (int it = 0, w; (w = kw_unit_at(it)) < units && ok; ++it) {
        const KwUnit u = kw_unit(a, w);
        const AttnSeq& sq = a.seq[u.seq];
        const KeyWeights& kw = a.w[Args::VIEWS == 1 ? 0 : sq.view];
        auto finish = [&](int key, float sum) {
            if (key >= sq.k_len) return;
            const int64_t r = sq.k_row0 + key;
            if (kw.before) sum += __ldg(kw.before + u.head * kw.before_stride + r);
            kw.after[u.head * kw.after_stride + r] = sum;
        };
        if (u.kind == KW_NONE) {
            for (int64_t key = (int64_t)u.j0 * TILE_ROWS + TILE_ROWS * g + row; key < min((int64_t)sq.k_len, (int64_t)u.j1 * TILE_ROWS); key += 2 * TILE_ROWS)
                finish((int)key, 0.f);
            continue;
        }
        const bool rows_stay = u.kind == KW_ROWS;
        if (!rows_stay && g >= u.stay) continue;
        // -lse log2(e) of this thread's column of query block b (beyond the sequence: a weight of 0)
        auto statistic = [&](int b) {
            const int p = b * TILE_ROWS + row, tok = p >> shift;
            return tok < sq.q_len ? -LOG2E * __ldg(a.lse + (int64_t)(sq.q_row0 + tok) * a.Hq + (u.head << shift) + (p & (G - 1))) : -INFINITY;
        };
        // The next buffer of statistics.  What it held two buffers ago is no longer read: every warp has come to the one
        // between, and comes there only when it is through with it.
        auto bring = [&](float x, bool write) {
            const int b = blk & 1;
            if (write) sh->neg[g][b][row] = x;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->neg_full[g][b]);
            ok = kw_wait_warp(&sh->neg_full[g][b], (blk >> 1) & 1, sh);
            ++blk;
        };
        float next = statistic(u.b0);
        const uint32_t blk0 = blk & 1;
        if (rows_stay) {
            const float x1 = u.stay > 1 ? statistic(u.b0 + 1) : 0.f;
            bring(next, true);
            if (ok) bring(x1, true);
        }
        Total total;
        for (int i = rows_stay ? g : 0; i < u.pass && ok; i += rows_stay ? 2 : 1) {
            const int key = (u.j0 + (rows_stay ? i : g)) * TILE_ROWS + row;
            float both = 0.f;
            for (int x = 0; x < (rows_stay ? u.stay : 1); ++x) {
                const int b = u.b0 + (rows_stay ? x : i);
                const float* neg = sh->neg[g][rows_stay ? blk0 ^ x : blk & 1];
                if (!rows_stay) {
                    bring(next, true);
                    if (!ok) break;
                    if (i + 1 < u.pass) next = statistic(b + 1);
                }
                const int columns = kw_columns(a, u, b), buf = tile & 1;
                // packed rows of the block that see the key: those of tokens [first, end)
                const int t0 = b * TILE_ROWS >> shift;
                const int64_t first = (int64_t)key - sq.off + 1 - t0;
                int64_t end = sq.q_len - t0;
                if (key >= a.mask.sinks) end = min(end, (int64_t)key + a.mask.window - sq.off + 1 - t0);
                const int lo = (int)max((int64_t)0, min((int64_t)TILE_ROWS, first)) << shift;
                const int hi = key < sq.k_len ? (int)max((int64_t)0, min((int64_t)TILE_ROWS, end)) << shift : 0;
                if (!(ok = kw_wait_warp(&sh->s_full[g][buf], (tile >> 1) & 1, sh))) break;
                ++tile;
                tc_fence_after();
                both += __any_sync(0xFFFFFFFFu, lo > 0 || hi < columns)
                            ? kw_row<true>(tS + 128 * buf, &sh->s_free[g][buf], neg, c2, columns, lo, hi, lane)
                            : kw_row<false>(tS + 128 * buf, &sh->s_free[g][buf], neg, c2, columns, lo, hi, lane);
            }
            if (!ok) break;
            if (rows_stay) finish(key, both);
            else total.add(both);
        }
        if (!ok) break;
        if (rows_stay) bring(0.f, false);   // (both buffers were in use: the next one waits for all warps)
        else if (u.slot < 0) finish((u.j0 + g) * TILE_ROWS + row, total.sum);
        else a.part[((int64_t)u.slot * a.Hkv + u.head) * (KW_KEY_TILES * TILE_ROWS) + g * TILE_ROWS + row] = total.sum;
    }
}

template <class Args>
__global__ void __launch_bounds__(KW_THREADS, 1) key_weights_kernel(const __grid_constant__ Args a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t* stay = smem;
    uint8_t* ring = smem + 4 * KW_TILE_BYTES;
    KwShared* sh = reinterpret_cast<KwShared*>(ring + KW_RING * KW_TILE_BYTES);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int units = a.n_entries * a.Hkv;
    pdl_trigger();
    if (warp == 8) {
        if (lane == 0) {
            for (int i = 0; i < 2; ++i) {
                mbar_init(&sh->st_full[i], 1);
                mbar_init(&sh->st_empty[i], 1);
                for (int b = 0; b < 2; ++b) {
                    mbar_init(&sh->s_full[i][b], 1);
                    mbar_init(&sh->s_free[i][b], 4);
                    mbar_init(&sh->neg_full[i][b], 4);
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
    } else if (warp == 9) {
        tmem_alloc(&sh->tmem, 512);
        tmem_relinquish();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sh->tmem;
    if (wait_limit(sh) != 0) {   // (not with a misaligned base)
        if (warp < 8) kw_sum(a, sh, units, tm, warp >> 2, tid & 127, lane);
        else if (warp == 8) kw_load(a, sh, stay, ring, units);
        else kw_products(a, sh, stay, ring, units, tm);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tm, 512);
    if (tid == 0 && wait_limit(sh) == 0) atomicAdd(a.waits.record, 1u);
}

// Sums of keys whose query blocks were cut into several units.
__global__ void __launch_bounds__(KW_KEY_TILES* TILE_ROWS) key_weights_join_kernel(const __grid_constant__ KwJoinArgs a) {
    const KwJoin e = a.e[blockIdx.x / a.Hkv];
    const int head = blockIdx.x % a.Hkv;
    const AttnSeq& sq = a.seq[e.seq];
    const KeyWeights& kw = a.w[e.seq];
    const int64_t key = (int64_t)e.j0 * TILE_ROWS + threadIdx.x;
    pdl_wait();   // the partial sums are written
    if (key >= sq.k_len || key >= (int64_t)e.j1 * TILE_ROWS) return;
    float sum = kw.before ? __ldg(kw.before + head * kw.before_stride + sq.k_row0 + key) : 0.f;
    float part = 0.f;
    for (int i = 0; i < e.n; ++i) part += a.part[((int64_t)(e.slot + i) * a.Hkv + head) * (KW_KEY_TILES * TILE_ROWS) + threadIdx.x];
    kw.after[head * kw.after_stride + sq.k_row0 + key] = sum + part;
}

}  // namespace

cudaError_t key_weights_prepare() {
    cudaError_t e = cudaFuncSetAttribute(key_weights_kernel<KwArgs1S>, cudaFuncAttributeMaxDynamicSharedMemorySize, KW_SMEM);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(key_weights_kernel<KwArgs1>, cudaFuncAttributeMaxDynamicSharedMemorySize, KW_SMEM);
    return e != cudaSuccess ? e : cudaFuncSetAttribute(key_weights_kernel<KwArgsN>, cudaFuncAttributeMaxDynamicSharedMemorySize, KW_SMEM);
}

template <class Args>
void launch_key_weights(const Args& a, cudaStream_t s) {
    const int64_t units = (int64_t)a.n_entries * a.Hkv;
    const int grid = (int)(units < ATTN_SMS ? units : ATTN_SMS);
    key_weights_kernel<Args><<<grid, KW_THREADS, KW_SMEM, s>>>(a);
}
template void launch_key_weights<KwArgs1S>(const KwArgs1S&, cudaStream_t);
template void launch_key_weights<KwArgs1>(const KwArgs1&, cudaStream_t);
template void launch_key_weights<KwArgsN>(const KwArgsN&, cudaStream_t);

void launch_key_weights_join(const KwJoinArgs& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)((int64_t)a.n_entries * a.Hkv));
    cfg.blockDim = dim3(KW_KEY_TILES * TILE_ROWS);
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, key_weights_join_kernel, a);
}

}  // namespace fq
