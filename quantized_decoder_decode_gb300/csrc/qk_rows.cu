// QK-norm, rotary embedding and the cache append of packed rows: what a prompt's (or a batch's)
// raw projections need before attention reads them.
//
// For every q and k head x of a row (128 values, f32):
//   y = x / sqrt(mean(x^2) + eps) * gain,
//   (y_i, y_{i+64}) -> (y_i c - y_{i+64} s, y_i s + y_{i+64} c),  (c, s) = table[position][i],
// q to q_out, k and (unchanged) v to the row of the sequence's cache layer, rounded once to bf16.
//
// Memory bound: 4 bytes in and 2 out per value, 512 bytes of table per position.  A warp takes
// four heads of one row, so that four 512-byte reads are in flight per warp before the first
// reduction, and one read of the row's cos and sin serves its four heads.

#include "attn.cuh"
#include "attn_plan.h"

namespace fq {

namespace {

constexpr int QR_HEADS = 4;      // heads per warp
constexpr int QR_THREADS = 128;   // (8191 rows of 48 heads: 54 us, 5.6 TB/s; 59 with CTAs of 256, 62 of 512, 66 as a loop over rows)

__global__ void __launch_bounds__(QR_THREADS) qk_rows_kernel(const __grid_constant__ QkRowsArgs a, int groups) {
    const int lane = threadIdx.x & 31;
    const int64_t w = ((int64_t)blockIdx.x * QR_THREADS + threadIdx.x) >> 5;
    const int row = (int)(w / groups), h0 = (int)(w % groups) * QR_HEADS;
    if (row >= a.rows) return;
    const int H = a.Hq + 2 * a.Hkv;
    // the sequence of the row: the last whose first row is not beyond it (empty ones share
    // their first row with the next)
    int lo = 0, hi = a.n_seq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.row0[mid] <= row) lo = mid;
        else hi = mid;
    }
    const int i = row - a.row0[lo];
    const float* src = a.qkv + (int64_t)row * a.qkv_stride + 4 * lane;
    float4 x[QR_HEADS];
#pragma unroll
    for (int j = 0; j < QR_HEADS; ++j)
        if (h0 + j < H) x[j] = __ldcs(reinterpret_cast<const float4*>(src + (int64_t)(h0 + j) * HEAD_DIM));
    const float4* cs = reinterpret_cast<const float4*>(a.rope + (int64_t)(a.pos0[lo] + i) * (HEAD_DIM / 2) + ((4 * lane) & 63));
    const float4 cs01 = __ldg(cs), cs23 = __ldg(cs + 1);
    const float c[4] = {cs01.x, cs01.z, cs23.x, cs23.z}, s[4] = {cs01.y, cs01.w, cs23.y, cs23.w};
    const KvRows& kv = a.kv[lo];
    const int64_t at = (int64_t)(a.kv_row0[lo] + i) * kv.row_stride + 4 * lane;
#pragma unroll
    for (int j = 0; j < QR_HEADS; ++j) {
        const int h = h0 + j;
        if (h >= H) break;
        float v[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
        uint16_t* dst;
        if (h < a.Hq + a.Hkv) {
            const bool is_q = h < a.Hq;
            const float4 g = __ldg(reinterpret_cast<const float4*>(is_q ? a.q_norm : a.k_norm) + lane);
            const float ss = warp_sum(v[0] * v[0] + v[1] * v[1] + v[2] * v[2] + v[3] * v[3]);
            const float inv = rsqrtf(ss * (1.f / HEAD_DIM) + a.eps);
            v[0] *= inv * g.x;
            v[1] *= inv * g.y;
            v[2] *= inv * g.z;
            v[3] *= inv * g.w;
#pragma unroll
            for (int e = 0; e < 4; ++e) {   // lanes 0-15 hold i, lanes 16-31 the partners i + 64
                const float o = __shfl_xor_sync(0xFFFFFFFFu, v[e], 16);
                v[e] = lane < 16 ? v[e] * c[e] - o * s[e] : v[e] * c[e] + o * s[e];
            }
            dst = is_q ? a.q_out + (int64_t)row * a.q_stride + (int64_t)h * HEAD_DIM + 4 * lane
                       : kv.k + at + (int64_t)(h - a.Hq) * kv.head_stride;
        } else {
            dst = kv.v + at + (int64_t)(h - a.Hq - a.Hkv) * kv.head_stride;
        }
        *reinterpret_cast<uint2*>(dst) = make_uint2(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]));
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
