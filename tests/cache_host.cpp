// The host side of the operators on windows, pages and caches made shorter (csrc/attn_cache_api.cu: checks, work
// lists, launches) with launches that are only written down, for tests without a GPU: nothing here touches a device,
// whatever the addresses.  Every launch becomes a list of numbers, read by cache_host_launch.

#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <vector>

#include "attn_cache_api.cu"

namespace {

char g_error[512];
std::vector<std::vector<long long>> g_launches;
uint32_t g_word, g_bad;

template <class... T>
void put(std::vector<long long>& v, T... x) {
    (v.push_back((long long)x), ...);
}
void put_seqs(std::vector<long long>& v, const AttnSeq* s, int n) {
    for (int i = 0; i < n; ++i) put(v, s[i].q_row0, s[i].q_len, s[i].k_row0, s[i].k_len, s[i].off, s[i].view);
}

}  // namespace

namespace fq {

fq_status fail(fq_status s, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_error, sizeof g_error, fmt, ap);
    va_end(ap);
    return s;
}

bool encode_bf16_tiles(void* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides, const uint32_t*) {
    // what a tensor map wants of these: 16-byte aligned, extents below 2^32, strides below 2^40
    bool ok = (reinterpret_cast<uintptr_t>(base) & 15) == 0;
    for (int i = 0; i < rank; ++i) ok = ok && dims[i] >= 1 && dims[i] <= 1ull << 32 && (i == 0 || (strides[i] % 16 == 0 && strides[i] < 1ull << 40));
    memset(map, ok ? 1 : 0, 128);
    return ok;
}

// 0, entries of the type, views of the type, paged, Hq, Hkv, window, sinks, n, n x (tok0, info, j0, j1), 64 sequences
template <class Args>
void launch_tiles(const Args& a, cudaStream_t) {
    std::vector<long long> v;
    put(v, 0, Args::ENTRIES, Args::VIEWS, Args::PAGED, a.io.Hq, a.io.Hkv, a.mask.window, a.mask.sinks, a.n_entries);
    for (int i = 0; i < a.n_entries; ++i) put(v, a.e[i].tok0, a.e[i].info, a.e[i].j0, a.e[i].j1);
    put_seqs(v, a.seq, MAX_SEQ);
    g_launches.push_back(v);
}
template void launch_tiles<WindowArgs1S>(const WindowArgs1S&, cudaStream_t);
template void launch_tiles<WindowArgs1>(const WindowArgs1&, cudaStream_t);
template void launch_tiles<WindowArgsN>(const WindowArgsN&, cudaStream_t);
template void launch_tiles<PagedArgsS>(const PagedArgsS&, cudaStream_t);
template void launch_tiles<PagedArgsL>(const PagedArgsL&, cudaStream_t);

// 1, beside, Hq, Hkv, window, sinks, n, n x (q_row0, n_tok, k_row0, k_len, off, first key number, keys, partial block or -1, sequence)
template <bool PAGED>
void rows(const WindowRowsArgs<PAGED>& a, bool beside) {
    std::vector<long long> v;
    put(v, 1, beside, a.io.Hq, a.io.Hkv, a.mask.window, a.mask.sinks, 0);
    if (a.n_items > MAX_ITEMS) abort();
    for (int i = 0; i < a.n_items; ++i)
        for (int n = a.group[i], c0, c1; rows_part(a, i, n, c0, c1); ++n, ++v[6]) {
            const RowGroup& g = a.g[n];
            put(v, g.q_row0, g.n_tok, g.k_row0, g.k_len, g.off, c0, c1 - c0, g.slot0 < 0 ? -1 : g.slot0 + i - g.item0, g.seq);
        }
    g_launches.push_back(v);
}
void launch_attn_window_rows(const WindowRowsArgs<false>& a, bool beside, cudaStream_t) { rows(a, beside); }
void launch_attn_window_rows(const WindowRowsArgs<true>& a, bool beside, cudaStream_t) { rows(a, beside); }

// 2, n, n x (q_row0, n_tok, k_len, off, a0, nA, a_step, a_row, b0, nB, b_row, c0, nC)
template <class Args>
void launch_attn_join(const Args& a, cudaStream_t) {
    std::vector<long long> v;
    put(v, 2, a.n_entries);
    for (int i = 0; i < a.n_entries; ++i) {
        const JoinEntry& e = a.e[i];
        put(v, e.q_row0, e.n_tok, e.k_len, e.off, e.a0, e.nA, e.a_step, e.a_row, e.b0, e.nB, e.b_row, e.c0, e.nC);
    }
    g_launches.push_back(v);
}
template void launch_attn_join<JoinArgsS>(const JoinArgsS&, cudaStream_t);
template void launch_attn_join<JoinArgsL>(const JoinArgsL&, cudaStream_t);

void launch_qk_paged(const QkPagedArgs& a, cudaStream_t) { g_launches.push_back({3, a.rows, a.pages.shift, a.pages.n_pages, a.pages.table_stride}); }

// 4, entries of the type, views of the type, Hq, Hkv, window, sinks, thread blocks, entries, units, units x (sequence, head, kind,
// more, j0, j1, b0, b1, slot), 64 sequences
template <class Args>
void launch_key_weights(const Args& a, int grid, cudaStream_t) {
    std::vector<long long> v;
    put(v, 4, Args::ENTRIES, Args::VIEWS, a.Hq, a.Hkv, a.mask.window, a.mask.sinks, grid, a.n_entries, 0);
    for (int c = 0; c < grid; ++c) {
        KwUnit u;
        for (KwLine l = kw_line(a, c); kw_next(a, l, u); ++v[9])
            put(v, u.seq, u.head, u.kind >> 7, (int)u.more, u.j0, u.j1, u.b0, u.b1, u.slot);
    }
    put_seqs(v, a.seq, MAX_SEQ);
    g_launches.push_back(v);
}
template void launch_key_weights<KwArgs1S>(const KwArgs1S&, int, cudaStream_t);
template void launch_key_weights<KwArgs1M>(const KwArgs1M&, int, cudaStream_t);
template void launch_key_weights<KwArgs1>(const KwArgs1&, int, cudaStream_t);
template void launch_key_weights<KwArgsN>(const KwArgsN&, int, cudaStream_t);
// 5, n, n x (sequence, head, more, j0, j1, first slot, first of the others' slots, others: two slots apart) of the sums that are joined
template <class Args>
void launch_key_weights_join(const Args& a, cudaStream_t) {
    std::vector<long long> v;
    put(v, 5, 0);
    for (int i = 0; i < a.n_entries; ++i)
        for (int h = 0; h < a.Hkv && !(a.e[i].info & (KW_ROWS | KW_NONE)); ++h) {
            int c0, c1;
            kw_parts(a, i, h, c0, c1);
            if (c0 == c1) continue;
            put(v, a.e[i].info & 127, h, (a.e[i].info & KW_MORE) != 0, a.e[i].j0, a.e[i].j1, 2 * c0 + 1, 2 * (c0 + 1), c1 - c0);
            ++v[1];
        }
    g_launches.push_back(v);
}
template void launch_key_weights_join<KwArgs1S>(const KwArgs1S&, cudaStream_t);
template void launch_key_weights_join<KwArgs1M>(const KwArgs1M&, cudaStream_t);
template void launch_key_weights_join<KwArgs1>(const KwArgs1&, cudaStream_t);
template void launch_key_weights_join<KwArgsN>(const KwArgsN&, cudaStream_t);
// 6, longest, blocks, n, n x (rows, rows that stay, first number, first block)
void launch_evict(const EvictArgs& a, int max_len, int blocks, cudaStream_t) {
    std::vector<long long> v;
    put(v, 6, max_len, blocks, a.n_seq);
    for (int i = 0; i < a.n_seq; ++i) put(v, a.s[i].len, a.s[i].n, a.s[i].kept0, a.s[i].block0);
    g_launches.push_back(v);
}

cudaError_t attn_window_tiles_prepare() { return cudaSuccess; }
cudaError_t attn_window_rows_prepare() { return cudaSuccess; }
cudaError_t key_weights_prepare() { return cudaSuccess; }
cudaError_t attn_page_word(uint32_t** word) {
    *word = &g_bad;
    return cudaSuccess;
}
fq_status attn_device(int* dev, uint32_t** waits) {
    *dev = 0;
    *waits = &g_word;
    return FQ_OK;
}
void attn_set_page_word(int, uint32_t*) {}

}  // namespace fq

extern "C" {

const char* fq_last_error(void) { return g_error; }
int cache_host_launches(int clear) {
    const int n = (int)g_launches.size();
    if (clear) g_launches.clear();
    return n;
}
int cache_host_launch(int i, long long* out, int room) {
    const std::vector<long long>& v = g_launches[i];
    for (int k = 0; k < (int)v.size() && k < room; ++k) out[k] = v[k];
    return (int)v.size();
}
cudaError_t CUDARTAPI cudaGetLastError(void) { return cudaSuccess; }
const char* CUDARTAPI cudaGetErrorString(cudaError_t) { return "no error"; }

}  // extern "C"
