// QK-norm, rotary embedding and the cache append of packed rows: what a prompt's (or a batch's)
// raw projections need before attention reads them.
//
// For every q and k head x of a row (128 values, f32):
//   y = x / sqrt(mean(x^2) + eps) * gain,
//   (y_i, y_{i+64}) -> (y_i c - y_{i+64} s, y_i s + y_{i+64} c),  (c, s) = table[position][i],
// q to q_out, k and (unchanged) v to the row of the sequence's cache layer, rounded once to bf16.
//
// Memory bound: 4 bytes in and 2 out per value, 512 bytes of table per position.  A warp takes
// four heads of one row: eight 256-byte reads are in flight per warp before the first reduction, one
// read of the row's cos and sin serves four heads, and their sums of squares are reduced together
// (6 exchanges and 4 broadcasts; one head after the other took 20, and with the partner's exchange
// 36).  8191 rows of 32 + 2 x 8 heads: 50.4 us, 6.0 TB/s; 54 with separate reductions, 52.7 with CTAs
// of 256 threads, 66 as a loop over rows with the next row's reads ahead.

#include "attn.cuh"
#include "attn_plan.h"

namespace fq {

namespace {

constexpr int QR_HEADS = 4;      // heads per warp
constexpr int QR_THREADS = 64;

__global__ void __launch_bounds__(QR_THREADS) qk_rows_kernel(const __grid_constant__ QkRowsArgs a, int groups) {
    const int lane = threadIdx.x & 31;
    const uint32_t w = blockIdx.x * (QR_THREADS / 32) + (threadIdx.x >> 5);
    const int row = (int)(w / (uint32_t)groups), h0 = (int)(w % (uint32_t)groups) * QR_HEADS;
    if (row >= a.rows) return;
    const int H = a.Hq + 2 * a.Hkv;
    // a lane has dims 2 lane, 2 lane + 1 and their partners 64 further
    const float* src = a.qkv + (int64_t)row * a.qkv_stride + h0 * HEAD_DIM + 2 * lane;
    float2 x0[QR_HEADS], x1[QR_HEADS];
#pragma unroll
    for (int j = 0; j < QR_HEADS; ++j) {
        x0[j] = x1[j] = make_float2(0.f, 0.f);
        if (h0 + j < H) {
            x0[j] = __ldcs(reinterpret_cast<const float2*>(src + j * HEAD_DIM));
            x1[j] = __ldcs(reinterpret_cast<const float2*>(src + j * HEAD_DIM + 64));
        }
    }
    // the sequence of the row: the last whose first row is not beyond it (empty ones share
    // their first row with the next)
    int lo = 0, hi = a.n_seq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.row0[mid] <= row) lo = mid;
        else hi = mid;
    }
    const int i = row - a.row0[lo];
    const float4 cs = __ldg(reinterpret_cast<const float4*>(a.rope + (int64_t)(a.pos0[lo] + i) * (HEAD_DIM / 2) + 2 * lane));
    const KvRows& kv = a.kv[lo];
    const int64_t at = (int64_t)(a.kv_row0[lo] + i) * kv.row_stride;
    // The four sums of squares at once: each exchange halves what a lane still adds up; lanes
    // 8 j .. 8 j + 7 end up with head j's.
    float inv;
    {
        static_assert(QR_HEADS == 4, "four sums over 32 lanes");
        float ss[QR_HEADS];
#pragma unroll
        for (int j = 0; j < QR_HEADS; ++j)
            ss[j] = x0[j].x * x0[j].x + x0[j].y * x0[j].y + x1[j].x * x1[j].x + x1[j].y * x1[j].y;
        const bool upper = lane & 16, odd = lane & 8;
        const float u0 = (upper ? ss[2] : ss[0]) + __shfl_xor_sync(0xFFFFFFFFu, upper ? ss[0] : ss[2], 16);
        const float u1 = (upper ? ss[3] : ss[1]) + __shfl_xor_sync(0xFFFFFFFFu, upper ? ss[1] : ss[3], 16);
        float t = (odd ? u1 : u0) + __shfl_xor_sync(0xFFFFFFFFu, odd ? u0 : u1, 8);
        t += __shfl_xor_sync(0xFFFFFFFFu, t, 4);
        t += __shfl_xor_sync(0xFFFFFFFFu, t, 2);
        t += __shfl_xor_sync(0xFFFFFFFFu, t, 1);
        inv = rsqrtf(t * (1.f / HEAD_DIM) + a.eps);
    }
#pragma unroll
    for (int j = 0; j < QR_HEADS; ++j) {
        const int h = h0 + j;
        if (h >= H) break;
        float2 y0 = x0[j], y1 = x1[j];
        uint16_t* dst;
        if (h < a.Hq + a.Hkv) {
            const bool is_q = h < a.Hq;
            const float* gain = (is_q ? a.q_norm : a.k_norm) + 2 * lane;
            const float2 g0 = __ldg(reinterpret_cast<const float2*>(gain)), g1 = __ldg(reinterpret_cast<const float2*>(gain + 64));
            const float r = __shfl_sync(0xFFFFFFFFu, inv, 8 * j);
            const float2 z0 = make_float2(y0.x * (r * g0.x), y0.y * (r * g0.y)), z1 = make_float2(y1.x * (r * g1.x), y1.y * (r * g1.y));
            y0 = make_float2(z0.x * cs.x - z1.x * cs.y, z0.y * cs.z - z1.y * cs.w);
            y1 = make_float2(z0.x * cs.y + z1.x * cs.x, z0.y * cs.w + z1.y * cs.z);
            dst = is_q ? a.q_out + (int64_t)row * a.q_stride + h * HEAD_DIM
                       : kv.k + at + (int64_t)(h - a.Hq) * kv.head_stride;
        } else {
            dst = kv.v + at + (int64_t)(h - a.Hq - a.Hkv) * kv.head_stride;
        }
        reinterpret_cast<uint32_t*>(dst)[lane] = bf16x2(y0.x, y0.y);
        reinterpret_cast<uint32_t*>(dst + 64)[lane] = bf16x2(y1.x, y1.y);
    }
}

}  // namespace

void launch_qk_rows(const QkRowsArgs& a, cudaStream_t s) {
    const int groups = (a.Hq + 2 * a.Hkv + QR_HEADS - 1) / QR_HEADS;
    const int64_t warps = (int64_t)a.rows * groups;
    const int64_t ctas = (warps * 32 + QR_THREADS - 1) / QR_THREADS;
    qk_rows_kernel<<<(unsigned)ctas, QR_THREADS, 0, s>>>(a, groups);
}

}  // namespace fq
