// Attention of few query rows over many keys: single tokens against their caches, the tails of a
// batch behind a shared prefix, short prompts.  And the kernel that joins partial results.
//
// Memory bound: every K and V row is read once per kv head for all G heads (x tokens) of the
// group, up to 16 packed rows, straight from global memory into the operand registers of
// mma.sync m16n8k16 (bf16, f32 sums): at 16 rows the tensor work is far below the memory time,
// and no shared memory or barrier stands between a load and its use.
//   S = Q K^T: the sum over the 128 dims may run in any order as long as Q and K agree, so a
//     thread's 16-byte piece of a K row (8 neighbouring dims) serves as the operand's pairs of
//     two k-steps.
//   O = P V: the weights leave S in the layout the second product takes them in; V rows 2c, 2c+1
//     (keys) are paired per dim by byte permutes, and the dims of a 16-byte piece go to eight
//     different n-tiles, so again every load is 16 bytes.
// A CTA of four warps takes a chunk of the keys of one (row group, kv head); the warps take
// blocks of 16 keys in turn with a running reference maximum (moved only when the maximum has
// grown by more than 2^8) and are joined in shared memory.
// Keys beyond the chunk are read as zeros with weight 0.  In blocks where some row does not see a
// key, V values that are not finite are set to zero for the product and added to the rows that
// see them.

#include "attn_plan.h"
#include "common.cuh"

namespace fq {

namespace {

constexpr int AR_WARPS = 4, AR_THREADS = AR_WARPS * 32;
constexpr int AR_OPAD = HEAD_DIM + 4;

FQ_DEV void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

FQ_DEV bool odd_pair(uint32_t w) { return (w & 0x7F800000u) == 0x7F800000u || (w & 0x7F80u) == 0x7F80u; }
FQ_DEV uint32_t finite_pair(uint32_t w) {
    if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
    if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
    return w;
}

__global__ void __launch_bounds__(AR_THREADS, 3) attn_rows_kernel(const __grid_constant__ RowsArgs a) {
    __shared__ float so[AR_WARPS][ROWS_MAX][AR_OPAD];
    __shared__ float2 sml[AR_WARPS][ROWS_MAX];
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int Hkv = a.io.Hkv, G = a.io.Hq / Hkv;
    const int item = blockIdx.x / Hkv, head = blockIdx.x % Hkv;
    int lo = 0, hi = a.n_groups;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.g[mid].item0 <= item) lo = mid;
        else hi = mid;
    }
    const RowGroup& g = a.g[lo];
    const KvRows& kv = a.kv[lo];
    const int rows = g.n_tok * G;
    const int c0 = (item - g.item0) * g.chunk;
    const int c1 = max(0, min(min(g.k_len, g.n_tok - 1 + g.off), c0 + g.chunk));
    const int first = max(0, min(g.k_len, g.off));   // keys that every row sees
    const int r = lane >> 2, c = lane & 3;
    int limit[2];
    const uint16_t* qrow[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int row = r + 8 * j, tok = row / G;
        limit[j] = row < rows ? max(0, min(g.k_len, tok + g.off)) : 0;
        qrow[j] = a.io.q + (int64_t)(g.q_row0 + tok) * a.io.q_stride + (int64_t)(head * G + row % G) * HEAD_DIM + 8 * c;
    }
    uint4 q[2][4];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[j][i] = r + 8 * j < rows ? __ldg(reinterpret_cast<const uint4*>(qrow[j] + 32 * i)) : make_uint4(0, 0, 0, 0);

    const uint16_t* kb = kv.k + (int64_t)g.k_row0 * kv.row_stride + (int64_t)head * kv.head_stride;
    const uint16_t* vb = kv.v + (int64_t)g.k_row0 * kv.row_stride + (int64_t)head * kv.head_stride;
    const int64_t rs = kv.row_stride;
    uint4 kr[2][4], vr[4][2];
    auto load_k = [&](int k0) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int key = k0 + 8 * j + r;
            const uint16_t* p = kb + (int64_t)key * rs + 8 * c;
#pragma unroll
            for (int i = 0; i < 4; ++i) kr[j][i] = key < c1 ? ld_stream16(p + 32 * i) : make_uint4(0, 0, 0, 0);
        }
    };
    auto load_v = [&](int k0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int key = k0 + 2 * c + (j & 1) + 8 * (j >> 1);
            const uint16_t* p = vb + (int64_t)key * rs + 8 * r;
#pragma unroll
            for (int h = 0; h < 2; ++h) vr[j][h] = key < c1 ? ld_stream16(p + 64 * h) : make_uint4(0, 0, 0, 0);
        }
    };
    float o[16][4];
#pragma unroll
    for (int t = 0; t < 16; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    int k0 = c0 + 16 * warp;
    if (k0 < c1) load_k(k0);
    for (; k0 < c1; k0 += 16 * AR_WARPS) {
        load_v(k0);
        float s[2][4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                mma16816(s[j], q[0][i].x, q[1][i].x, q[0][i].y, q[1][i].y, kr[j][i].x, kr[j][i].y);
                mma16816(s[j], q[0][i].z, q[1][i].z, q[0][i].w, q[1][i].w, kr[j][i].z, kr[j][i].w);
            }
        }
        if (k0 + 16 * AR_WARPS < c1) load_k(k0 + 16 * AR_WARPS);
        // scores of row r (s[j][0..1]) and r + 8 (s[j][2..3]), keys k0 + 8j + 2c + {0, 1}
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[j][e] = k0 + 8 * j + 2 * c + (e & 1) < min(limit[e >> 1], c1) ? s[j][e] * a.c : -INFINITY;
        float f[2];
        bool move = false;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float top = fmaxf(fmaxf(s[0][2 * j], s[0][2 * j + 1]), fmaxf(s[1][2 * j], s[1][2 * j + 1]));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            const bool mv = top - m[j] > 8.f;   // (not at -inf - -inf)
            f[j] = mv ? ex2(m[j] - top) : 1.f;
            if (mv) m[j] = top;
            move |= mv;
        }
        if (__any_sync(0xFFFFFFFFu, move)) {
            l[0] *= f[0];
            l[1] *= f[1];
#pragma unroll
            for (int t = 0; t < 16; ++t) {
                o[t][0] *= f[0];
                o[t][1] *= f[0];
                o[t][2] *= f[1];
                o[t][3] *= f[1];
            }
        }
        const float m0 = m[0] == -INFINITY ? 0.f : m[0], m1 = m[1] == -INFINITY ? 0.f : m[1];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            s[j][0] = ex2(s[j][0] - m0);
            s[j][1] = ex2(s[j][1] - m0);
            s[j][2] = ex2(s[j][2] - m1);
            s[j][3] = ex2(s[j][3] - m1);
            l[0] += s[j][0] + s[j][1];
            l[1] += s[j][2] + s[j][3];
        }
        const uint32_t p0 = bf16x2(s[0][0], s[0][1]), p1 = bf16x2(s[0][2], s[0][3]), p2 = bf16x2(s[1][0], s[1][1]),
                       p3 = bf16x2(s[1][2], s[1][3]);
        bool odd = false;
        if (k0 + 16 > first) {   // some row does not see all of these keys
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    odd |= odd_pair(vr[j][h].x) || odd_pair(vr[j][h].y) || odd_pair(vr[j][h].z) || odd_pair(vr[j][h].w);
            odd = __any_sync(0xFFFFFFFFu, odd);
            if (odd) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        vr[j][h] = make_uint4(finite_pair(vr[j][h].x), finite_pair(vr[j][h].y), finite_pair(vr[j][h].z),
                                              finite_pair(vr[j][h].w));
            }
        }
        // dim 64h + 8r + e of the pieces is column r of n-tile 8h + e
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t w0[4] = {vr[0][h].x, vr[0][h].y, vr[0][h].z, vr[0][h].w}, w1[4] = {vr[1][h].x, vr[1][h].y, vr[1][h].z, vr[1][h].w};
            const uint32_t w2[4] = {vr[2][h].x, vr[2][h].y, vr[2][h].z, vr[2][h].w}, w3[4] = {vr[3][h].x, vr[3][h].y, vr[3][h].z, vr[3][h].w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint32_t sel = e & 1 ? 0x7632u : 0x5410u;
                mma16816(o[8 * h + e], p0, p1, p2, p3, __byte_perm(w0[e >> 1], w1[e >> 1], sel), __byte_perm(w2[e >> 1], w3[e >> 1], sel));
            }
        }
        if (odd) {
            for (int k = 0; k < 16 && k0 + k < c1; ++k) {
                const uint16_t* p = vb + (int64_t)(k0 + k) * rs;
#pragma unroll
                for (int t = 0; t < 16; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint16_t b = p[64 * (t >> 3) + 8 * (2 * c + (e & 1)) + (t & 7)];
                        if ((b & 0x7F80u) == 0x7F80u && k0 + k < limit[e >> 1]) o[t][e] += bf2f(b);
                    }
            }
        }
    }
    // ---- join the warps
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        l[j] += __shfl_xor_sync(0xFFFFFFFFu, l[j], 1);
        l[j] += __shfl_xor_sync(0xFFFFFFFFu, l[j], 2);
        if (c == 0) sml[warp][r + 8 * j] = make_float2(m[j], l[j]);
        if (r + 8 * j < rows)
#pragma unroll
            for (int t = 0; t < 16; ++t) {
                so[warp][r + 8 * j][64 * (t >> 3) + 16 * c + (t & 7)] = o[t][2 * j];
                so[warp][r + 8 * j][64 * (t >> 3) + 16 * c + 8 + (t & 7)] = o[t][2 * j + 1];
            }
    }
    __syncthreads();
    for (int row = warp; row < rows; row += AR_WARPS) {
        float M = -INFINITY, L = 0.f;
#pragma unroll
        for (int w = 0; w < AR_WARPS; ++w) M = fmaxf(M, sml[w][row].x);
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < AR_WARPS; ++w) {
            const float2 ml = sml[w][row];
            const float f = ml.x == -INFINITY && M != -INFINITY ? 0.f : ml.x == M ? 1.f : ex2(ml.x - M);
            if (ml.x == -INFINITY && ml.y == 0.f) continue;   // saw no key (its sums are zero)
            const float4 v = *reinterpret_cast<const float4*>(&so[w][row][4 * lane]);
            L = fmaf(ml.y, f, L);
            y.x = fmaf(v.x, f, y.x);
            y.y = fmaf(v.y, f, y.y);
            y.z = fmaf(v.z, f, y.z);
            y.w = fmaf(v.w, f, y.w);
        }
        const int tok = row / G;
        if (g.slot0 >= 0) {
            const int64_t blk = ((int64_t)(g.slot0 + item - g.item0) * Hkv + head) * ROWS_MAX + row;
            reinterpret_cast<float4*>(a.part.b_o + blk * HEAD_DIM)[lane] = y;
            if (lane == 0) a.part.b_ml[blk] = make_float2(M, L);
        } else {
            const float inv = min(g.k_len, tok + g.off) > 0 ? 1.f / L : 0.f;
            if (min(g.k_len, tok + g.off) > 0) {
                y.x *= inv;
                y.y *= inv;
                y.z *= inv;
                y.w *= inv;
            }
            const int64_t at = (int64_t)(g.q_row0 + tok) * a.io.out_stride + (int64_t)(head * G + row % G) * HEAD_DIM;
            if (a.io.out_f32) reinterpret_cast<float4*>((float*)a.io.out + at)[lane] = y;
            else reinterpret_cast<uint2*>((uint16_t*)a.io.out + at)[lane] = make_uint2(bf16x2(y.x, y.y), bf16x2(y.z, y.w));
        }
    }
    pdl_wait();   // this grid ends after the one it may run beside, so what waits for it waits for both
}

// out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i over the partial results of the rows of an
// entry.  A kv head's G rows of a token are joined by G warps: a lane takes one row and four dims
// (one 16-byte load per partial result, eight in flight), so that a warp reads G x 32 bytes at a
// time from the chunked layout of the tiles and whole 32-byte sectors from the rows.  The reads
// are what it costs: it starts early (its index work overlaps the kernels before) and is short.
constexpr int AJ_WARPS = 8;

template <class Args>
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
    const int64_t b_blk = ((int64_t)e.b0 * Hkv + kh) * ROWS_MAX + e.b_row + row, c_blk = ((int64_t)e.c0 * Hkv + kh) * ROWS_MAX + row;
    const int64_t b_step = (int64_t)Hkv * ROWS_MAX;
    // partial result i of this row: (m, l) and the values
    auto ml_at = [&](int i) -> const float2* {
        if (i < e.nA) return a_ml + i * a_step;
        i -= e.nA;
        return a.part.b_ml + (i < e.nB ? b_blk + i * b_step : c_blk + (i - e.nB) * b_step);
    };
    auto o_at = [&](int i) -> const float4* {
        if (i < e.nA) return reinterpret_cast<const float4*>(a_o + i * a_step * HEAD_DIM);
        i -= e.nA;
        return reinterpret_cast<const float4*>(a.part.b_o + (i < e.nB ? b_blk + i * b_step : c_blk + (i - e.nB) * b_step) * HEAD_DIM + d);
    };
    pdl_wait();   // the partial results are written
    if (idx >= e.n_tok * Hq) return;
    float M = -INFINITY;
#pragma unroll 4
    for (int i = 0; i < n; ++i) M = fmaxf(M, ml_at(i)->x);
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
    float L = 0.f;
    constexpr int BATCH = 8;
    for (int i0 = 0; i0 < n; i0 += BATCH) {
        float4 v[BATCH];
        float2 ml[BATCH];
#pragma unroll
        for (int k = 0; k < BATCH; ++k)
            if (i0 + k < n) {
                v[k] = *o_at(i0 + k);
                ml[k] = *ml_at(i0 + k);
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

static cudaLaunchConfig_t config(dim3 grid, int threads, bool dependent, cudaLaunchAttribute* attr, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = dependent ? 1 : 0;
    return cfg;
}

void launch_attn_rows(const RowsArgs& a, bool dependent, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    const cudaLaunchConfig_t cfg = config(dim3((unsigned)((int64_t)a.n_items * a.io.Hkv)), AR_THREADS, dependent, attr, s);
    cudaLaunchKernelEx(&cfg, attn_rows_kernel, a);
}

template <class Args>
void launch_attn_join(const Args& a, cudaStream_t s) {
    cudaLaunchAttribute attr[1];
    const unsigned y = (unsigned)((a.max_tok * a.io.Hq + AJ_WARPS - 1) / AJ_WARPS);
    const cudaLaunchConfig_t cfg = config(dim3((unsigned)a.n_entries, y), AJ_WARPS * 32, true, attr, s);
    cudaLaunchKernelEx(&cfg, attn_join_kernel<Args>, a);
}
template void launch_attn_join<JoinArgsS>(const JoinArgsS&, cudaStream_t);
template void launch_attn_join<JoinArgsL>(const JoinArgsL&, cudaStream_t);

}  // namespace fq
