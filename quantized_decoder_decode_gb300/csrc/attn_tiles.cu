// The tile kernel of prompt and shared-prompt attention (attn_tiles.cuh): rows that see every key up to their own.

#include "attn_tiles.cuh"

namespace fq {

namespace {

__device__ uint32_t g_attn_waits;   // CTAs that gave up, of calls that name no other record

}  // namespace

cudaError_t attn_tiles_prepare() {
    cudaError_t e = prepare_t<TileArgs1S>();
    if (e == cudaSuccess) e = prepare_t<TileArgs1>();
    if (e == cudaSuccess) e = prepare_t<TileArgsNS>();
    return e != cudaSuccess ? e : prepare_t<TileArgsN>();
}

template void launch_tiles<TileArgs1S>(const TileArgs1S&, cudaStream_t);
template void launch_tiles<TileArgs1>(const TileArgs1&, cudaStream_t);
template void launch_tiles<TileArgsNS>(const TileArgsNS&, cudaStream_t);
template void launch_tiles<TileArgsN>(const TileArgsN&, cudaStream_t);

cudaError_t attn_wait_word(uint32_t** word) { return cudaGetSymbolAddress((void**)word, g_attn_waits); }

}  // namespace fq
