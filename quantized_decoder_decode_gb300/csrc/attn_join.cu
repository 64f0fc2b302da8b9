// Joins the partial results of attn_tiles.cu and attn_rows.cu where keys are split or come from two places:
//   out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,   M = max_i m_i.
// A kv head's G rows of a token are joined by G warps: a lane takes one row and four dims (one
// 16-byte load per partial result, eight in flight), so that a warp reads G x 32 bytes at a time
// from the chunked layout.  The reads are what it costs: it starts early (its index work overlaps
// the kernel before) and is short.  Up to four parts take the variant with four reads in flight, which
// fits an SM four times instead of twice: 10656 rows of three parts (16.7 MB) 5 us instead of 9 (the whole
// call 45.3 us instead of 49.3); more parts take eight at a time (17 to 20 parts of 512 rows: 3.2 us).

#include "attn_plan.h"
#include "attn.cuh"

namespace fq {

namespace {

constexpr int AJ_WARPS = 8;

template <class Args, int BATCH>
__global__ void __launch_bounds__(AJ_WARPS * 32) attn_join_kernel(const __grid_constant__ Args a) {
    const int lane = threadIdx.x & 31;
    const JoinEntry e = a.e[blockIdx.x];
    const int Hq = a.io.Hq, Hkv = a.io.Hkv, G = Hq / Hkv;
    const int idx = blockIdx.y * AJ_WARPS + (threadIdx.x >> 5);
    const int t = idx / Hq, kh = idx % Hq / G;
    const int gh = (lane >> 1) % G, row = t * G + gh;
    const int d = ((idx % G) * (16 / G) + (lane >> 1) / G) * 8 + (lane & 1) * 4;   // dims d .. d + 3
    const int n = e.nA + e.nB + e.nC;
    const float* a_o = a.part.a_o + ((int64_t)e.a0 * Hkv + kh) * TILE_ROWS * HEAD_DIM + ((d >> 3) * TILE_ROWS + e.a_row + row) * 8 + (d & 7);
    const float2* a_ml = a.part.a_ml + ((int64_t)e.a0 * Hkv + kh) * TILE_ROWS + e.a_row + row;
    const int64_t a_step = (int64_t)e.a_step * Hkv * TILE_ROWS;
    const int64_t b_blk = (int64_t)e.b0 * Hkv + kh, c_blk = (int64_t)e.c0 * Hkv + kh;
    // partial result i of this row: (m, l) and the values
    auto ml_at = [&](int i) -> const float2* {
        if (i < e.nA) return a_ml + i * a_step;
        i -= e.nA;
        return a.part.b_ml + (i < e.nB ? (b_blk + (int64_t)i * Hkv) * SMALL_ROWS + e.b_row
                                       : (c_blk + (int64_t)(i - e.nB) * Hkv) * SMALL_ROWS) + row;
    };
    auto o_at = [&](int i) -> const float4* {
        if (i < e.nA) return reinterpret_cast<const float4*>(a_o + i * a_step * HEAD_DIM);
        i -= e.nA;
        const int64_t blk = i < e.nB ? b_blk + (int64_t)i * Hkv : c_blk + (int64_t)(i - e.nB) * Hkv;
        const int r8 = row + (i < e.nB ? e.b_row : 0);
        return reinterpret_cast<const float4*>(a.part.b_o + blk * (SMALL_ROWS * HEAD_DIM) + ((d >> 3) * SMALL_ROWS + r8) * 8 + (d & 7));
    };
    pdl_wait();   // the partial results are written
    if (idx >= e.n_tok * Hq) return;
    // One pass: values and statistics of a batch of partial results are read together, what is
    // summed so far follows the maximum.
    float M = -INFINITY, L = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < n; i0 += BATCH) {
        float4 v[BATCH];
        float2 ml[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
            if (i0 + k < n) {
                ml[k] = *ml_at(i0 + k);
                v[k] = *o_at(i0 + k);
            }
        float top = M;
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
            if (i0 + k < n) top = fmaxf(top, ml[k].x);
        if (M != top) {
            const float f = ex2(M - top);   // (0 from -inf)
            L *= f;
            y.x *= f;
            y.y *= f;
            y.z *= f;
            y.w *= f;
            M = top;
        }
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
            if (i0 + k < n) {
                // (a part that saw no key, or only scores of -inf, weighs nothing; a NaN sum stays one)
                const float f = ml[k].x == -INFINITY && ml[k].y == 0.f ? 0.f : ml[k].x == M ? 1.f : ex2(ml[k].x - M);
                L = fmaf(ml[k].y, f, L);
                if (f == 0.f) continue;   // its values may not be finite
                y.x = fmaf(v[k].x, f, y.x);
                y.y = fmaf(v[k].y, f, y.y);
                y.z = fmaf(v[k].z, f, y.z);
                y.w = fmaf(v[k].w, f, y.w);
            }
    }
    if (min(e.k_len, t + e.off) > 0) {
        const float inv = 1.f / L;
        y.x *= inv;
        y.y *= inv;
        y.z *= inv;
        y.w *= inv;
    }
    const int64_t at = (int64_t)(e.q_row0 + t) * a.io.out_stride + (int64_t)(kh * G + gh) * HEAD_DIM + d;
    if (a.io.out_f32) *reinterpret_cast<float4*>((float*)a.io.out + at) = y;
    else *reinterpret_cast<uint2*>((uint16_t*)a.io.out + at) = make_uint2(bf16x2(y.x, y.y), bf16x2(y.z, y.w));
}

}  // namespace

template <class Args>
void launch_attn_join(const Args& a, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)a.n_entries, (unsigned)((a.max_tok * a.io.Hq + AJ_WARPS - 1) / AJ_WARPS));
    cfg.blockDim = dim3(AJ_WARPS * 32);
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, a.max_parts <= 4 ? attn_join_kernel<Args, 4> : attn_join_kernel<Args, 8>, a);
}
template void launch_attn_join<JoinArgsS>(const JoinArgsS&, cudaStream_t);
template void launch_attn_join<JoinArgsL>(const JoinArgsL&, cudaStream_t);

}  // namespace fq
