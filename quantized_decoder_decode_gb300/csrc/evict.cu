// A cache made shorter: per (sequence, kv head) the rows with the largest gathered weights stay, with the first and the
// most recent ones, and move to other rows in their order.
//
// The choice.  Rows [sinks, len - recent) compete for what the first and the last rows leave.  The weights become
// unsigned numbers of the same order (a NaN above all others, -0 as 0), and three passes of 11, 11 and 10 bits from the top
// count how many share each value of the digit: the digit of the last one that stays is where the counts from above
// reach the number wanted.  Then T is known in full, and how many of those equal to T stay: the first ones.  One more
// pass gives every row that stays its place.  A cluster of up to 8 thread blocks shares the work of one
// (sequence, head) beyond 8192 rows; each counts its part of the rows in its own shared memory and reads the others'.
//
// The move reads and writes 512 bytes per row, 16 per lane: half a warp a row of K, the other half the row of V.
//
// What bounds it.  One cache of 8192 rows and 8 heads down to 2048: 12.8 us; as launches by themselves the choice 11 (a chain:
// the rows' weights come once, then counts, a scan and a barrier for each digit) and the move 6.  Sixteen down to 1024 rows each (134 MB
// read and written): 28 us; by themselves the choice 11 and the move 19, at 7.0 TB/s.  Two blocks of 512 threads in a cluster instead of
// one of 1024: 13.7 and 32.8 us; four copies of the first digit's counters and digits of 9, 11 and 12 bits: 13.5 and 28.7.

#include <cooperative_groups.h>

#include "attn.cuh"
#include "cache_plan.h"

namespace fq {

namespace cg = cooperative_groups;

namespace {

constexpr int EV_THREADS = 1024, EV_PER = 8, EV_CHUNK = EV_THREADS * EV_PER;   // rows that a block holds at a time
constexpr int EV_BINS = 2048, EV_PASSES = 3, EV_CLUSTER = 8;
constexpr int EV_MOVE_WARPS = 4, EV_MOVE_ROWS = EVICT_ROWS / EV_MOVE_WARPS;   // rows of a warp

FQ_DEV uint32_t order_key(float w) {
    if (w != w) return 0xFFFFFFFFu;
    return float_order_key(w == 0.f ? 0.f : w);
}

// exclusive prefix sum over the block's threads, and the total
FQ_DEV uint32_t block_scan(uint32_t v, uint32_t* sums, uint32_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    static_assert(EV_THREADS / 32 == 32, "a lane per warp");
    __syncthreads();
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    uint32_t w = sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, w, o);
        if (lane >= o) w += y;
    }
    total = __shfl_sync(0xFFFFFFFFu, w, 31);
    const uint32_t before = __shfl_sync(0xFFFFFFFFu, w, (warp + 31) & 31);
    return (warp ? before : 0) + x - v;
}

__global__ void __launch_bounds__(EV_THREADS) evict_select_kernel(const __grid_constant__ EvictArgs a) {
    __shared__ __align__(16) uint32_t hist[EV_PASSES][EV_BINS];
    __shared__ uint32_t sums[EV_THREADS / 32];
    __shared__ uint32_t found[2];   // digit, how many of it stay
    __shared__ uint32_t counts[2];  // this block's rows that stay for sure, and those equal to the last one
    pdl_trigger();
    cg::cluster_group cluster = cg::this_cluster();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank(), tid = threadIdx.x;
    const int unit = blockIdx.x / C, head = unit % a.Hkv;
    const EvictSeq& s = a.s[unit / a.Hkv];
    const float* w = s.w + head * s.w_stride;
    int32_t* kept = a.kept + s.kept0 + (int64_t)head * s.n;
    const int len = s.len;
    // this block's rows: a whole number of 8 per thread
    const int per = ((len + C - 1) / C + EV_PER - 1) / EV_PER * EV_PER;
    const int r0 = (int)min((int64_t)len, (int64_t)rank * per), r1 = (int)min((int64_t)len, (int64_t)r0 + per);
    if (s.n == 0) return;   // (the whole cluster takes these ways; without rows that stay there are no addresses either)
    if (s.n == len) {
        for (int r = r0 + tid; r < r1; r += EV_THREADS) kept[r] = r;
        return;
    }
    const int lo = a.sinks, hi = len - a.recent;   // (sinks + recent <= n < len)
    uint32_t want = (uint32_t)(s.n - a.sinks - a.recent);

    for (int i = tid; i < EV_PASSES * EV_BINS; i += EV_THREADS) (&hist[0][0])[i] = 0;
    __syncthreads();
    uint32_t key[EV_PER];
    int held = -1;   // first row of the chunk in `key`
    auto load = [&](int base) {
        if (base == held) return;
        held = base;
#pragma unroll
        for (int i = 0; i < EV_PER; ++i) {
            const int64_t r = (int64_t)base + tid * EV_PER + i;
            key[i] = r >= lo && r < hi && r < r1 ? order_key(__ldg(w + r)) : 0u;
        }
    };
    auto meet = [&]() {
        if (C > 1) cluster.sync();
        else __syncthreads();
    };
    uint32_t top = 0;   // the digits found so far
    int shift = 32;
#pragma unroll 1
    for (int p = 0; p < EV_PASSES; ++p) {
        const int bits = p < 2 ? 11 : 10, above = shift;
        shift -= bits;
#pragma unroll 1
        for (int64_t base = r0; base < r1; base += EV_CHUNK) {
            load((int)base);
#pragma unroll
            for (int i = 0; i < EV_PER; ++i) {
                const int64_t r = base + tid * EV_PER + i;
                if (r >= lo && r < hi && r < r1 && (p == 0 || key[i] >> above == top))
                    atomicAdd(&hist[p][key[i] >> shift & ((1u << bits) - 1)], 1u);
            }
        }
        meet();
        // bins from the top: thread t has the two below EV_BINS - 2 t
        static_assert(EV_BINS == 2 * EV_THREADS, "two bins per thread");
        const int b0 = EV_BINS - 2 - 2 * tid;
        uint2 n = make_uint2(0, 0);
        if (C == 1) n = *reinterpret_cast<const uint2*>(&hist[p][b0]);
        else
#pragma unroll 1
            for (int c = 0; c < C; ++c) {
                const uint2 h = *reinterpret_cast<const uint2*>(cluster.map_shared_rank(&hist[p][0], c) + b0);
                n.x += h.x;
                n.y += h.y;
            }
        uint32_t total;
        const uint32_t over = block_scan(n.x + n.y, sums, total);   // in the bins above these
        if (over < want && want <= over + n.x + n.y) {
            const bool upper = want <= over + n.y;
            found[0] = (uint32_t)(b0 + upper);
            found[1] = want - over - (upper ? 0 : n.y);
        }
        __syncthreads();
        if (want) {
            top = top << bits | found[0];
            want = found[1];
        }
    }
    // top: the number of the last row that stays; `want` of those equal to it stay (0: none of the competing rows)
    const bool any = want != 0;
    auto classes = [&](int64_t base, uint32_t& sure, uint32_t& equal) {   // a bit per row
        load((int)base);
        sure = equal = 0;
#pragma unroll
        for (int i = 0; i < EV_PER; ++i) {
            const int64_t r = base + tid * EV_PER + i;
            if (r >= r1) continue;
            if (r < lo || r >= hi || (any && key[i] > top)) sure |= 1u << i;
            else if (any && key[i] == top) equal |= 1u << i;
        }
    };
    uint32_t sure = 0, equal = 0, before = 0, total = 0;   // of a chunk
    auto count = [&](int64_t base) {
        classes(base, sure, equal);
        before = block_scan((uint32_t)__popc(sure) << 16 | (uint32_t)__popc(equal), sums, total);
    };
    const bool once = r1 - r0 <= EV_CHUNK;   // one chunk is counted once
    if (C > 1) {
        uint32_t n_sure = 0, n_equal = 0;
#pragma unroll 1
        for (int64_t base = r0; base < r1; base += EV_CHUNK) {
            count(base);
            n_sure += total >> 16;
            n_equal += total & 0xFFFFu;
        }
        if (tid == 0) {
            counts[0] = n_sure;
            counts[1] = n_equal;
        }
        cluster.sync();
    }
    uint32_t equal_before = 0, place = 0;
#pragma unroll 1
    for (int c = 0; c < rank; ++c) {
        const uint32_t* n = cluster.map_shared_rank(&counts[0], c);
        place += n[0];
        equal_before += n[1];
    }
    place += min(equal_before, want);
#pragma unroll 1
    for (int64_t base = r0; base < r1; base += EV_CHUNK) {
        if (C == 1 || !once) count(base);
        uint32_t eq = equal_before + (before & 0xFFFFu);
        uint32_t at = place + (before >> 16) + (min(eq, want) - min(equal_before, want));
#pragma unroll
        for (int i = 0; i < EV_PER; ++i) {
            bool stays = sure >> i & 1;
            if (equal >> i & 1) stays = eq++ < want;
            if (stays) kept[at++] = (int32_t)(base + tid * EV_PER + i);
        }
        place += (total >> 16) + (min(equal_before + (total & 0xFFFFu), want) - min(equal_before, want));
        equal_before += total & 0xFFFFu;
    }
    if (C > 1) cluster.sync();   // the others have read this block's counts
}

__global__ void __launch_bounds__(EV_MOVE_WARPS * 32) evict_move_kernel(const __grid_constant__ EvictArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int lo = 0, hi = a.n_seq;   // the last sequence whose first block is not beyond this one
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.s[mid].block0 <= (int)blockIdx.x) lo = mid;
        else hi = mid;
    }
    const EvictSeq& s = a.s[lo];
    const int per = (s.n + EVICT_ROWS - 1) / EVICT_ROWS;   // blocks of a head
    const int b = (int)blockIdx.x - s.block0, head = b / per;
    const int i0 = (b - head * per) * EVICT_ROWS + warp * EV_MOVE_ROWS;
    const int n = min(EV_MOVE_ROWS, s.n - i0);
    const int d = (lane & 15) * 8;
    const uint16_t* from = (lane < 16 ? s.from.k : s.from.v) + (int64_t)head * s.from.head_stride + d;
    uint16_t* to = (lane < 16 ? s.to.k : s.to.v) + (int64_t)head * s.to.head_stride + d;
    pdl_wait();   // the rows are chosen
    if (n <= 0) return;
    int row = 0;
    if (lane < n) {
        row = __ldcg(a.kept + s.kept0 + (int64_t)head * s.n + i0 + lane);
        if (s.w_to) s.w_to[head * s.w_to_stride + i0 + lane] = __ldg(s.w + head * s.w_stride + row);
    }
    uint4 x[EV_MOVE_ROWS];
#pragma unroll
    for (int i = 0; i < EV_MOVE_ROWS; ++i) {
        const int r = __shfl_sync(0xFFFFFFFFu, row, i);
        if (i < n) x[i] = ld_stream16(from + (int64_t)r * s.from.row_stride);
    }
#pragma unroll
    for (int i = 0; i < EV_MOVE_ROWS; ++i)
        if (i < n) *reinterpret_cast<uint4*>(to + (int64_t)(i0 + i) * s.to.row_stride) = x[i];
}

}  // namespace

void launch_evict(const EvictArgs& a, int max_len, int blocks, cudaStream_t s) {
    int C = 1;
    while (C < EV_CLUSTER && (int64_t)C * EV_CHUNK < max_len) C *= 2;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)(a.n_seq * a.Hkv * C));
    cfg.blockDim = dim3(EV_THREADS);
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)C;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // Without a selection nothing may move: `kept` would hold anything.  (The caller reads the error, cudaGetLastError.)
    if (cudaLaunchKernelEx(&cfg, evict_select_kernel, a) != cudaSuccess) return;
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(EV_MOVE_WARPS * 32);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchKernelEx(&cfg, evict_move_kernel, a);
}

}  // namespace fq
