// Attention of few query rows over many keys: single tokens against their caches, the tails of a
// batch behind a shared prefix, short prompts.
//
// Memory bound: every K and V row is read once per kv head for all G heads (x tokens) of the
// group, up to 8 packed rows, straight from global memory into the operand registers of
// mma.sync m16n8k16 (bf16, f32 sums), with the query rows as the 8 columns: the tensor work is far
// below the memory time, and no shared memory or barrier stands between a load and its use.
//   S' = K Q' (16 keys x 8 rows): the sum over the 128 dims may run in any order as long as Q and
//     K agree, so a thread's 16-byte piece of a K row (8 neighbouring dims) serves as the
//     operand's pairs of two k-steps.
//   O' = V' P' (dims x 8 rows): the weights, rounded to bf16 pairs, are transposed between the
//     lanes (movmatrix); V rows 2c, 2c+1 (keys) are paired per dim by byte permutes, and the
//     dims of a thread's 16-byte pieces go to eight different tiles, so that every load is 16
//     bytes again and a thread ends up with 8 neighbouring dims of two rows.
// A CTA of four warps takes a chunk of the keys of one (row group, kv head); the warps take
// blocks of 16 keys in turn with a running reference maximum (moved only when the maximum has
// grown by more than 2^8; weights 2^-lift of the usual ones, as in attn_tiles.cu) and are joined in shared
// memory.
// Measured: 16 single tokens over 512 to 4097 rows (152 MB, 32 / 8 heads) 26 us, 5.8 TB/s; a block of 64
// keys of a CTA takes 1.9 us, of which its reads wait for memory all but 0.3.  The start of a CTA (its
// arguments, the first reads) is 2.5 us, the join in it 0.7 us.  CTAs of two warps, six per SM, balance better but
// leave twice the partial results: 32.8 us for the call instead of 31.0.
// Keys beyond the chunk are read as zeros with weight 0.  In blocks where some row does not see a
// key, V values that are not finite are set to zero for the product and added to the rows that
// see them.

#include "attn_plan.h"
#include "attn.cuh"

namespace fq {

namespace {

constexpr int AR_WARPS = 4, AR_THREADS = AR_WARPS * 32;
constexpr int AR_OPAD = HEAD_DIM + 4;

FQ_DEV void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 8 x 8 matrix of 16-bit values, two neighbours of row lane / 4 per lane, transposed
FQ_DEV uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

FQ_DEV bool odd_pair(uint32_t w) { return (w & 0x7F800000u) == 0x7F800000u || (w & 0x7F80u) == 0x7F80u; }
FQ_DEV uint32_t finite_pair(uint32_t w) {
    if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
    if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
    return w;
}
FQ_DEV float max_over_rows(float v) {   // over the lanes with the same lane % 4
    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
    v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
    return fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
}

__global__ void __launch_bounds__(AR_THREADS, ROWS_CTAS_SM) attn_rows_kernel(const __grid_constant__ RowsArgs a) {
    __shared__ float so[AR_WARPS][SMALL_ROWS][AR_OPAD];
    __shared__ float2 sml[AR_WARPS][SMALL_ROWS];
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int Hkv = a.io.Hkv, G = a.io.Hq / Hkv;
    const int item = blockIdx.x / Hkv, head = blockIdx.x % Hkv;
    const RowGroup& g = a.g[a.group[item]];
    const KvRows& kv = a.kv[a.group[item]];
    const int rows = g.n_tok * G;
    const int c0 = (item - g.item0) * g.chunk;
    const int c1 = max(0, min(min(g.k_len, g.n_tok - 1 + g.off), c0 + g.chunk));
    const int first = max(0, min(g.k_len, g.off));   // keys that every row sees
    const int r = lane >> 2, c = lane & 3;

    const int64_t rs = kv.row_stride;
    const uint16_t* kb = kv.k + (int64_t)g.k_row0 * rs + (int64_t)head * kv.head_stride + 8 * c;
    const uint16_t* vb = kv.v + (int64_t)g.k_row0 * rs + (int64_t)head * kv.head_stride;
    uint4 kr[2][4], vr[4][2];
    auto load_k = [&](int k0) {   // keys k0 + r, k0 + 8 + r: dims 32i + 8c ..
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int key = k0 + 8 * j + r;
            const uint16_t* p = kb + (int64_t)key * rs;
#pragma unroll
            for (int i = 0; i < 4; ++i) kr[j][i] = key < c1 ? ld_stream16(p + 32 * i) : make_uint4(0, 0, 0, 0);
        }
    };
    auto load_v = [&](int k0) {   // keys k0 + 2c, + 1, + 8, + 9: dims 64h + 8r ..
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int key = k0 + 2 * c + (j & 1) + 8 * (j >> 1);
            const uint16_t* p = vb + (int64_t)key * rs + 8 * r;
#pragma unroll
            for (int h = 0; h < 2; ++h) vr[j][h] = key < c1 ? ld_stream16(p + 64 * h) : make_uint4(0, 0, 0, 0);
        }
    };
    int k0 = c0 + 16 * warp;
    if (k0 < c1) {
        load_k(k0);
        load_v(k0);
    }
    uint4 q[4];   // packed row r: dims 32i + 8c ..
    {
        const uint16_t* p = a.io.q + (int64_t)(g.q_row0 + r / G) * a.io.q_stride + (int64_t)(head * G + r % G) * HEAD_DIM + 8 * c;
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = r < rows ? __ldg(reinterpret_cast<const uint4*>(p + 32 * i)) : make_uint4(0, 0, 0, 0);
    }
    int limit[2];   // keys of this chunk's range that rows 2c, 2c + 1 see
#pragma unroll
    for (int e = 0; e < 2; ++e) limit[e] = 2 * c + e < rows ? min(c1, max(0, (2 * c + e) / G + g.off)) : 0;
    float o[8][4];   // dims 8r + t (rows 2c, 2c + 1), 64 + 8r + t
#pragma unroll
    for (int t = 0; t < 8; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    for (; k0 < c1; k0 += 16 * AR_WARPS) {
        const bool more = k0 + 16 * AR_WARPS < c1;   // K and V of the next block come while this one is worked on
        float s[4] = {0.f, 0.f, 0.f, 0.f};   // (key r, rows 2c, 2c + 1), (key 8 + r, ..)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            mma16816(s, kr[0][i].x, kr[1][i].x, kr[0][i].y, kr[1][i].y, q[i].x, q[i].y);
            mma16816(s, kr[0][i].z, kr[1][i].z, kr[0][i].w, kr[1][i].w, q[i].z, q[i].w);
        }
        if (more) load_k(k0 + 16 * AR_WARPS);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[e] = k0 + 8 * (e >> 1) + r < limit[e & 1] ? s[e] * a.c : -INFINITY;
        float f[2];
        bool move = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float top = max_over_rows(fmaxf(s[e], s[2 + e]));
            const bool mv = top - m[e] > 8.f;   // (not at -inf - -inf)
            f[e] = mv ? ex2(m[e] - top) : 1.f;
            if (mv) m[e] = top;
            move |= mv;
        }
        if (__any_sync(0xFFFFFFFFu, move)) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[e] *= f[e];
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    o[t][e] *= f[e];
                    o[t][2 + e] *= f[e];
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float mm = m[e] == -INFINITY ? 0.f : m[e] + a.io.lift;
            s[e] = ex2(s[e] - mm);
            s[2 + e] = ex2(s[2 + e] - mm);
            l[e] += s[e] + s[2 + e];
        }
        const uint32_t p0 = transpose8(bf16x2(s[0], s[1])), p1 = transpose8(bf16x2(s[2], s[3]));
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
        {
            const uint32_t w[4][2][4] = {
                {{vr[0][0].x, vr[0][0].y, vr[0][0].z, vr[0][0].w}, {vr[0][1].x, vr[0][1].y, vr[0][1].z, vr[0][1].w}},
                {{vr[1][0].x, vr[1][0].y, vr[1][0].z, vr[1][0].w}, {vr[1][1].x, vr[1][1].y, vr[1][1].z, vr[1][1].w}},
                {{vr[2][0].x, vr[2][0].y, vr[2][0].z, vr[2][0].w}, {vr[2][1].x, vr[2][1].y, vr[2][1].z, vr[2][1].w}},
                {{vr[3][0].x, vr[3][0].y, vr[3][0].z, vr[3][0].w}, {vr[3][1].x, vr[3][1].y, vr[3][1].z, vr[3][1].w}}};
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const uint32_t sel = t & 1 ? 0x7632u : 0x5410u;
                mma16816(o[t], __byte_perm(w[0][0][t >> 1], w[1][0][t >> 1], sel), __byte_perm(w[0][1][t >> 1], w[1][1][t >> 1], sel),
                         __byte_perm(w[2][0][t >> 1], w[3][0][t >> 1], sel), __byte_perm(w[2][1][t >> 1], w[3][1][t >> 1], sel), p0, p1);
            }
        }
        if (more) load_v(k0 + 16 * AR_WARPS);
        if (odd) {
            for (int k = 0; k < 16 && k0 + k < c1; ++k) {
                const uint16_t* p = vb + (int64_t)(k0 + k) * rs + 8 * r;
#pragma unroll
                for (int t = 0; t < 8; ++t)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint16_t b = p[64 * (e >> 1) + t];
                        if ((b & 0x7F80u) == 0x7F80u && k0 + k < limit[e & 1]) o[t][e] += bf2f(b);
                    }
            }
        }
    }
    // ---- join the warps
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 4);
        l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 8);
        l[e] += __shfl_xor_sync(0xFFFFFFFFu, l[e], 16);
        if (r == 0) sml[warp][2 * c + e] = make_float2(m[e], l[e]);
        if (2 * c + e < rows)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float4* d = reinterpret_cast<float4*>(&so[warp][2 * c + e][64 * h + 8 * r]);
                d[0] = make_float4(o[0][2 * h + e], o[1][2 * h + e], o[2][2 * h + e], o[3][2 * h + e]);
                d[1] = make_float4(o[4][2 * h + e], o[5][2 * h + e], o[6][2 * h + e], o[7][2 * h + e]);
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
            if (ml.x == -INFINITY && ml.y == 0.f) continue;   // saw no key, or only scores of -inf
            const float f = ml.x == M ? 1.f : ex2(ml.x - M);
            const float4 v = *reinterpret_cast<const float4*>(&so[w][row][4 * lane]);
            L = fmaf(ml.y, f, L);
            y.x = fmaf(v.x, f, y.x);
            y.y = fmaf(v.y, f, y.y);
            y.z = fmaf(v.z, f, y.z);
            y.w = fmaf(v.w, f, y.w);
        }
        const int tok = row / G;
        if (g.slot0 >= 0) {
            const int64_t blk = (int64_t)(g.slot0 + item - g.item0) * Hkv + head;
            float* to = a.part.b_o + blk * (SMALL_ROWS * HEAD_DIM) + (lane >> 1) * (SMALL_ROWS * 8) + row * 8 + (lane & 1) * 4;
            *reinterpret_cast<float4*>(to) = y;
            if (lane == 0) a.part.b_ml[blk * SMALL_ROWS + row] = make_float2(M, L);
        } else {
            if (min(g.k_len, tok + g.off) > 0) {
                const float inv = 1.f / L;
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

}  // namespace

// What is in flight from memory (12 warps x 8 KB per SM) is held in the L1 cache, which is what shared
// memory leaves of 256 KB: behind attn_tiles.cu, with its 227 KB, a block of keys took 3.2 us
// instead of 1.9 (64 tails behind a shared prefix 45 -> 39 us) until the split was asked for.
cudaError_t attn_rows_prepare() {
    constexpr int SHARED_PERCENT = 25;   // 57 KB: three CTAs
    return cudaFuncSetAttribute(attn_rows_kernel, cudaFuncAttributePreferredSharedMemoryCarveout, SHARED_PERCENT);
}

void launch_attn_rows(const RowsArgs& a, bool beside, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3((unsigned)((int64_t)a.n_items * a.io.Hkv));
    cfg.blockDim = dim3(AR_THREADS);
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = beside ? 1 : 0;
    cudaLaunchKernelEx(&cfg, attn_rows_kernel, a);
}

}  // namespace fq
