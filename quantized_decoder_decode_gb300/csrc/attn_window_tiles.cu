// The tile kernel of attention with windows and sinks, over views and over pages (attn_tiles.cuh).

#include "attn_tiles.cuh"

namespace fq {

namespace {

__device__ uint32_t g_bad_pages;   // table entries that named no page of their pool

}  // namespace

cudaError_t attn_page_word(uint32_t** word) { return cudaGetSymbolAddress((void**)word, g_bad_pages); }

cudaError_t attn_window_tiles_prepare() {
    cudaError_t e = prepare_t<WindowArgs1S>();
    if (e == cudaSuccess) e = prepare_t<WindowArgs1>();
    if (e == cudaSuccess) e = prepare_t<WindowArgsN>();
    if (e == cudaSuccess) e = prepare_t<PagedArgsS>();
    return e != cudaSuccess ? e : prepare_t<PagedArgsL>();
}

template void launch_tiles<WindowArgs1S>(const WindowArgs1S&, cudaStream_t);
template void launch_tiles<WindowArgs1>(const WindowArgs1&, cudaStream_t);
template void launch_tiles<WindowArgsN>(const WindowArgsN&, cudaStream_t);
template void launch_tiles<PagedArgsS>(const PagedArgsS&, cudaStream_t);
template void launch_tiles<PagedArgsL>(const PagedArgsL&, cudaStream_t);

}  // namespace fq
