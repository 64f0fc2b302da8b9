// Attention of packed prompts and of batches behind a shared prefix: the plain first form.
// One CTA of four warps per (query row, query head): each warp takes every fourth key, keeps a
// running maximum, sum and value vector (4 dims per lane), and the four are joined at the end.

#include "common.cuh"
#include "kernels.h"

namespace fq {

namespace {

struct Span {
    const uint16_t *k, *v;
    int64_t stride;
    int n;
};

FQ_DEV void attend(const Span& sp, int warp, int lane, const float q[4], float& m, float& l, float o[4]) {
    for (int j = warp; j < sp.n; j += 4) {
        const uint2 kw = *reinterpret_cast<const uint2*>(sp.k + (int64_t)j * sp.stride + 4 * lane);
        const uint2 vw = *reinterpret_cast<const uint2*>(sp.v + (int64_t)j * sp.stride + 4 * lane);
        float s = q[0] * bf_lo(kw.x) + q[1] * bf_hi(kw.x) + q[2] * bf_lo(kw.y) + q[3] * bf_hi(kw.y);
        s = warp_sum(s);
        const float mn = fmaxf(m, s);
        const float r = m == mn ? 1.f : exp2f(m - mn), p = exp2f(s - (mn == -INFINITY ? 0.f : mn));
        l = l * r + p;
        o[0] = o[0] * r + p * bf_lo(vw.x);
        o[1] = o[1] * r + p * bf_hi(vw.x);
        o[2] = o[2] * r + p * bf_lo(vw.y);
        o[3] = o[3] * r + p * bf_hi(vw.y);
        m = mn;
    }
}

FQ_DEV void row_out(const AttnIo& io, int row, int h, const Span* sp, int n_sp) {
    __shared__ float sm[4], sl[4], so[4][HEAD_DIM];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint2 qw = *reinterpret_cast<const uint2*>(io.q + (int64_t)row * io.q_stride + (int64_t)h * HEAD_DIM + 4 * lane);
    const float f = io.scale * 1.4426950408889634f;
    const float q[4] = {bf_lo(qw.x) * f, bf_hi(qw.x) * f, bf_lo(qw.y) * f, bf_hi(qw.y) * f};
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    int keys = 0;
    for (int i = 0; i < n_sp; ++i) {
        attend(sp[i], warp, lane, q, m, l, o);
        keys += sp[i].n;
    }
    for (int e = 0; e < 4; ++e) so[warp][4 * lane + e] = o[e];
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
    __syncthreads();
    const int d = threadIdx.x;
    const float M = fmaxf(fmaxf(sm[0], sm[1]), fmaxf(sm[2], sm[3]));
    float L = 0.f, O = 0.f;
    for (int w = 0; w < 4; ++w) {
        const float r = sm[w] == M ? 1.f : exp2f(sm[w] - M);
        L += sl[w] * r;
        O += so[w][d] * r;
    }
    const float y = keys ? O / L : 0.f;
    const int64_t at = (int64_t)row * io.out_stride + (int64_t)h * HEAD_DIM + d;
    if (io.out_f32) ((float*)io.out)[at] = y;
    else ((__nv_bfloat16*)io.out)[at] = __float2bfloat16_rn(y);
}

__global__ void __launch_bounds__(128) prompt_kernel(const __grid_constant__ PromptArgs a) {
    const int row = blockIdx.x, h = blockIdx.y;
    int s = 0;
    while (s + 1 < a.n_seq && a.seq[s + 1].q_row0 <= row) ++s;
    const PromptSeq& q = a.seq[s];
    const int kh = h / (a.io.Hq / a.io.Hkv);
    const int64_t base = (int64_t)q.k_row0 * a.kv[s].row_stride + (int64_t)kh * a.kv[s].head_stride;
    const int i = row - q.q_row0;
    const Span sp{a.kv[s].k + base, a.kv[s].v + base, a.kv[s].row_stride, max(0, i + q.k_len - q.q_len + 1)};
    row_out(a.io, row, h, &sp, 1);
}

__global__ void __launch_bounds__(128) shared_kernel(const __grid_constant__ SharedArgs a) {
    const int s = blockIdx.x, h = blockIdx.y;
    const int kh = h / (a.io.Hq / a.io.Hkv);
    const int64_t p0 = (int64_t)kh * a.prefix.head_stride, t0 = (int64_t)kh * a.tail[s].head_stride;
    const Span sp[2] = {{a.prefix.k + p0, a.prefix.v + p0, a.prefix.row_stride, a.prefix_len},
                        {a.tail[s].k + t0, a.tail[s].v + t0, a.tail[s].row_stride, a.tail_len[s]}};
    row_out(a.io, s, h, sp, 2);
}

}  // namespace

void launch_prompt(const PromptArgs& a, cudaStream_t s) {
    prompt_kernel<<<dim3(a.q_rows, a.io.Hq), 128, 0, s>>>(a);
}

void launch_shared(const SharedArgs& a, cudaStream_t s) {
    shared_kernel<<<dim3(a.n_seq, a.io.Hq), 128, 0, s>>>(a);
}

}  // namespace fq
