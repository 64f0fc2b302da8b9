// The host side of the attention operators (csrc/attn_api.cu: checks, work lists, launches) with launches that
// are only written down, for tests without a GPU: nothing here touches a device, whatever the addresses.
// Every launch becomes a list of numbers, read by attn_host_launch.

#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <vector>

#include "attn_api.cu"

namespace {

char g_error[512];
std::vector<std::vector<long long>> g_launches;
uint32_t g_word;

struct FakeMap {   // what encode_bf16_tiles notes in place of a tensor map
    unsigned long long base, rank, dims[4], strides[4];
};
static_assert(sizeof(FakeMap) <= 128, "a tensor map");

template <class... T>
void put(std::vector<long long>& v, T... x) {
    (v.push_back((long long)x), ...);
}
void put_map(std::vector<long long>& v, const void* map) {   // base, rows, row and head stride in bytes
    FakeMap m;
    memcpy(&m, map, sizeof m);
    put(v, m.base, m.dims[1], m.strides[1], m.strides[2]);
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

bool encode_bf16_tiles(void* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides_bytes, const uint32_t*) {
    FakeMap m = {};
    m.base = (unsigned long long)base;
    m.rank = rank;
    for (int i = 0; i < rank; ++i) {
        m.dims[i] = dims[i];
        m.strides[i] = strides_bytes[i];
    }
    memcpy(map, &m, sizeof m);
    return true;
}

// 0, entries of the type, views of the type, Hq, Hkv, n, n x (tok0, info, j0, j1), per sequence (q_row0, q_len, k_row0,
// k_len, off, view) with those that no entry names left at 0, and per view of the type the K and V maps
// (base, rows, strides) with those that no sequence names left at 0
template <class Args>
void launch_tiles(const Args& a, cudaStream_t) {
    std::vector<long long> v;
    put(v, 0, Args::ENTRIES, Args::VIEWS, a.io.Hq, a.io.Hkv, a.n_entries);
    bool seq[MAX_SEQS] = {}, view[MAX_SEQS] = {};
    for (int i = 0; i < a.n_entries; ++i) {
        put(v, a.e[i].tok0, a.e[i].info, a.e[i].j0, a.e[i].j1);
        seq[a.e[i].info & 127] = true;
    }
    for (int i = 0; i < MAX_SEQS; ++i) {
        const AttnSeq s = seq[i] ? a.seq[i] : AttnSeq{0, 0, 0, 0, 0, 0};
        put(v, s.q_row0, s.q_len, s.k_row0, s.k_len, s.off, s.view);
        if (seq[i] && s.k_len) view[s.view] = true;
    }
    for (int i = 0; i < Args::VIEWS; ++i)
        if (view[i]) {
            put_map(v, a.map_k[i]);
            put_map(v, a.map_v[i]);
        } else {
            put(v, 0, 0, 0, 0, 0, 0, 0, 0);
        }
    g_launches.push_back(v);
}
template void launch_tiles<TileArgs1S>(const TileArgs1S&, cudaStream_t);
template void launch_tiles<TileArgs1>(const TileArgs1&, cudaStream_t);
template void launch_tiles<TileArgsNS>(const TileArgsNS&, cudaStream_t);
template void launch_tiles<TileArgsN>(const TileArgsN&, cudaStream_t);

// 1, beside, Hq, Hkv, n, n x (q_row0, n_tok, k_row0, k_len, off, first key, keys, partial block or -1, k, v)
void launch_attn_rows(const RowsArgs& a, bool beside, cudaStream_t) {
    std::vector<long long> v;
    put(v, 1, beside, a.io.Hq, a.io.Hkv, a.n_items);
    for (int i = 0; i < a.n_items; ++i) {
        const RowGroup& g = a.g[a.group[i]];
        const KvRows& kv = a.kv[a.group[i]];
        const int c = i - g.item0;
        put(v, g.q_row0, g.n_tok, g.k_row0, g.k_len, g.off, (long long)c * g.chunk, g.chunk, g.slot0 < 0 ? -1 : g.slot0 + c, kv.k, kv.v);
    }
    g_launches.push_back(v);
}

// 2, entries of the type, n, max_tok, max_parts, n x (q_row0, n_tok, k_len, off, a0, nA, a_step, a_row, b0, nB, b_row, c0, nC)
template <class Args>
void launch_attn_join(const Args& a, cudaStream_t) {
    std::vector<long long> v;
    put(v, 2, Args::ENTRIES, a.n_entries, a.max_tok, a.max_parts);
    for (int i = 0; i < a.n_entries; ++i) {
        const JoinEntry& e = a.e[i];
        put(v, e.q_row0, e.n_tok, e.k_len, e.off, e.a0, e.nA, e.a_step, e.a_row, e.b0, e.nB, e.b_row, e.c0, e.nC);
    }
    g_launches.push_back(v);
}
template void launch_attn_join<JoinArgsS>(const JoinArgsS&, cudaStream_t);
template void launch_attn_join<JoinArgsL>(const JoinArgsL&, cudaStream_t);

void launch_qk_rows(const QkRowsArgs& a, cudaStream_t) { g_launches.push_back({3, a.rows}); }

cudaError_t attn_tiles_prepare() { return cudaSuccess; }
cudaError_t attn_rows_prepare() { return cudaSuccess; }
cudaError_t attn_wait_word(uint32_t** word) {
    *word = &g_word;
    return cudaSuccess;
}

}  // namespace fq

extern "C" {

const char* fq_last_error(void) { return g_error; }

// the number of launches written down; launch i: its length, and its numbers where `out` has room for them
int attn_host_launches(int clear) {
    const int n = (int)g_launches.size();
    if (clear) g_launches.clear();
    return n;
}
int attn_host_launch(int i, long long* out, int room) {
    const std::vector<long long>& v = g_launches[i];
    for (int k = 0; k < (int)v.size() && k < room; ++k) out[k] = v[k];
    return (int)v.size();
}

// the runtime calls of the host side
cudaError_t CUDARTAPI cudaGetDevice(int* dev) {
    *dev = 0;
    return cudaSuccess;
}
cudaError_t CUDARTAPI cudaGetLastError(void) { return cudaSuccess; }
const char* CUDARTAPI cudaGetErrorString(cudaError_t) { return "no error"; }
cudaError_t CUDARTAPI cudaMemcpyAsync(void* dst, const void* src, size_t n, cudaMemcpyKind, cudaStream_t) {
    memcpy(dst, src, n);
    return cudaSuccess;
}
cudaError_t CUDARTAPI cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }

}  // extern "C"
