// routing_api.hip -- host side of the operators around the experts' products
// and the shared projection (declared in include/fp8gemm.h): the router's
// choice, tokens sorted by expert and back with their gradients, low-rank
// adapters.
//
// As in fp8gemm_api.hip every entry point validates on the host, enqueues
// nothing on an error, launches on the caller's stream, and neither
// allocates, frees nor synchronizes.
#include <algorithm>

#include "host_common.h"
#include "kernels_adapter.h"
#include "kernels_expert.h"
#include "kernels_route.h"

namespace {

using namespace fp8h;

// Workgroups of a launch: a grid has fewer than 2^32 threads.
constexpr int64_t max_grid(int threads) { return 0xFFFFFFFFll / threads; }

bool row_type_ok(int32_t t) { return t == FP8_TYPE_F32 || t == FP8_TYPE_BF16; }
size_t type_size(int32_t t) { return t == FP8_TYPE_F32 ? 4 : 2; }
bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// ---------------------------------------------------------------------------
// The router.
// ---------------------------------------------------------------------------
constexpr int kMaxRouteE = 1024, kMaxRouteK = 64;

fp8_status check_route(int64_t T, int32_t E, int32_t k, int32_t type) {
    if (!dims_ok(T) || E < 1 || k < 1 || !row_type_ok(type)) return FP8_ERR_INVALID_ARG;
    if (k > E) return FP8_ERR_SHAPE;
    if (E > kMaxRouteE || k > kMaxRouteK || cdiv(T, 4) > max_grid(256)) return FP8_ERR_UNSUPPORTED;
    return FP8_OK;
}

template <typename T, bool GRAD>
void launch_route(fp8k::RouteParams& p, hipStream_t s) {
    const dim3 grid((unsigned)cdiv(p.T, 4)), block(256);
    auto go = [&](auto kernel, int per) {
        // a lane's `per` logits in one load: rows and lanes at multiples of it
        const size_t bytes = std::min<size_t>(per * sizeof(T), 16);
        p.vec = p.E % per == 0 && aligned(p.logits, bytes) && (!GRAD || aligned(p.dlogits, bytes));
        hipLaunchKernelGGL(kernel, grid, block, 0, s, p);
    };
    auto pick = [&](auto choice, auto grad, int per) {
        if constexpr (GRAD) go(grad, per);
        else go(choice, per);
    };
    if (p.E <= 64) pick(fp8k::route_topk_kernel<T, 1>, fp8k::route_grad_kernel<T, 1>, 1);
    else if (p.E <= 128) pick(fp8k::route_topk_kernel<T, 2>, fp8k::route_grad_kernel<T, 2>, 2);
    else if (p.E <= 256) pick(fp8k::route_topk_kernel<T, 4>, fp8k::route_grad_kernel<T, 4>, 4);
    else if (p.E <= 512) pick(fp8k::route_topk_kernel<T, 8>, fp8k::route_grad_kernel<T, 8>, 8);
    else pick(fp8k::route_topk_kernel<T, 16>, fp8k::route_grad_kernel<T, 16>, 16);
}

// ---------------------------------------------------------------------------
// The sort.
// ---------------------------------------------------------------------------
// One workgroup counts and places alone while its pairs are few; then chunks
// are counted by a first kernel, at most kMaxSortChunks, since every workgroup
// adds up all chunks' counts.  One MI355X, both kernels, us: 2048 pairs of 256
// experts alone 8.4, two chunks 8.9; 4096 of 64 alone 9.1, four chunks 7.8;
// 65536 of 256 in chunks of 1024 9.8, of 2048 11.7, of 4096 15.9.
constexpr int64_t kSortAlone = 2048, kSortChunk = 1024, kMaxSortChunks = 256;

int64_t sort_chunk(int64_t pairs) {
    if (pairs <= kSortAlone) return std::max<int64_t>(pairs, 1);
    return std::max(kSortChunk, cdiv(cdiv(pairs, kMaxSortChunks), 1024) * 1024);
}
int64_t sort_chunks(int64_t pairs) { return std::max<int64_t>(cdiv(pairs, sort_chunk(pairs)), 1); }
size_t sort_bytes(int64_t pairs, int64_t bins) {
    const int64_t chunks = sort_chunks(pairs);
    return chunks > 1 ? (size_t)(cdiv(chunks, 4) * 4 * bins) * sizeof(int32_t) : 0;
}

fp8_status check_sort(int64_t pairs, int32_t E, int32_t id_bytes) {
    if (!dims_ok(pairs) || E < 1 || !(id_bytes == 4 || id_bytes == 8)) return FP8_ERR_INVALID_ARG;
    if (E > fp8k::kSortMaxExperts || pairs > kMaxDim / 2) return FP8_ERR_UNSUPPORTED;
    return FP8_OK;
}

fp8_status run_sort(fp8k::SortParams& p, void* ws, size_t ws_bytes, hipStream_t s) {
    if (ws_bytes && !ws) return FP8_ERR_INVALID_ARG;
    if (!aligned16(ws)) return FP8_ERR_ALIGNMENT;
    if (ws_bytes < sort_bytes(p.pairs, p.bins)) return FP8_ERR_SCRATCH;
    int cus = 0;
    const fp8_status st = current_device_cus(&cus);
    if (st != FP8_OK) return st;
    p.chunk = sort_chunk(p.pairs);
    p.chunks = (int32_t)sort_chunks(p.pairs);
    p.chunks4 = (int32_t)cdiv(p.chunks, 4) * 4;
    p.hist = static_cast<int32_t*>(ws);
    const dim3 grid((unsigned)p.chunks);
    if (p.chunks > 1) {
        hipLaunchKernelGGL(fp8k::expert_count_kernel, grid, dim3(1024), 0, s, p);
        const fp8_status run = launch_status();
        if (run != FP8_OK) return run;
    }
    if (p.chunk <= 512) hipLaunchKernelGGL((fp8k::expert_place_kernel<4, 2>), grid, dim3(256), 0, s, p);
    else if (p.chunk <= 1024) hipLaunchKernelGGL((fp8k::expert_place_kernel<16, 1>), grid, dim3(1024), 0, s, p);
    else if (p.chunk <= 2048) hipLaunchKernelGGL((fp8k::expert_place_kernel<16, 2>), grid, dim3(1024), 0, s, p);
    else if (p.chunk <= 4096) hipLaunchKernelGGL((fp8k::expert_place_kernel<16, 4>), grid, dim3(1024), 0, s, p);
    else hipLaunchKernelGGL((fp8k::expert_place_kernel<16, 0>), grid, dim3(1024), 0, s, p);
    return launch_status();
}

// ---------------------------------------------------------------------------
// Rows.
// ---------------------------------------------------------------------------
fp8_status check_rows(int64_t T, int32_t k, int64_t rows, int64_t W, int32_t type) {
    if (!dims_ok(T) || !dims_ok(rows) || !dims_ok(W) || k < 1 || !row_type_ok(type)) return FP8_ERR_INVALID_ARG;
    if (T * k >= kMaxDim) return FP8_ERR_UNSUPPORTED;
    return FP8_OK;
}

// Codes of more bytes than the last-level cache holds are stored past the caches.
constexpr int64_t kCacheBytes = (int64_t)256 << 20;
// Rows of whole cache lines, which no other row shares.
constexpr size_t kLine = 128;
bool whole_lines(int64_t W, int32_t type, const void* p) { return W * (int64_t)type_size(type) % kLine == 0 && aligned(p, kLine); }

// Waves (4 a workgroup) that move rows, and those that look for rows to clear;
// workgroups in whole `step`s.
fp8_status rows_grid(fp8k::RowsParams& p, int64_t per_seg, dim3* grid, int64_t step = 1) {
    p.segs = cdiv(p.W, per_seg);
    p.work = p.T * p.segs;
    const int64_t waves = p.work + (p.src ? cdiv(p.rows, fp8k::kClearRows) : 0);
    const int64_t wgs = cdiv(cdiv(waves, 4), step) * step;
    if (wgs > max_grid(256)) return FP8_ERR_UNSUPPORTED;
    *grid = dim3((unsigned)wgs);
    return FP8_OK;
}

// ---------------------------------------------------------------------------
// Adapters.
// ---------------------------------------------------------------------------
struct AdapterPlan {
    int whole;                  // one kernel, with as many workgroups per tile; 0: two kernels
    int group;                  // tiles per workgroup of the two: 1 or 4
    int64_t tiles, groups, splits, k_range, n_range;
    size_t bytes(int64_t R) const { return whole ? 0 : (size_t)(splits * tiles * 16 * R) * sizeof(float); }
};

// One kernel where tiles hold few tokens (tokens times R up to 64 per tile of the
// table) and four workgroups per tile are about one per compute unit: a table's
// tiles are those it has room for, of which a quarter or more is empty in most
// batches.  One MI355X, one kernel / two, us, tiles in use x tokens of each:
// K 7168, N 2048: 1 x 1 R 16 6.2 / 7.4, R 64 12.1 / 11.8; 64 x 1 R 16 6.9 / 9.2, R 64
// 17.4 / 19.1; 64 x 4 R 16 9.5 / 9.8; K 2048, N 7168: 1 x 1 R 16 5.9 / 6.8; 64 x 1 7.7 /
// 11.4; and a launch less.  The other side, K 7168, N 2048: 24 x 16 R 16 11.4 / 8.5, R 64
// 25.3 / 16.2; 96 x 1 with four workgroups each 12.5 / 11.2, with two 8.3, but
// with two a tile of 16 tokens takes 14.0 / 7.9.  Parts of N of 256 columns or more (1 x 1,
// R 16: N 2048 8 parts 6.2, 16 6.1, N 300 2 parts 5.7, 16 6.2).
int adapter_whole_parts(int64_t T, int64_t tiles, int64_t N, int64_t R, int cus) {
    if (R > 64 || T * R > 64 * tiles || 3 * tiles > cus) return 0;
    int parts = 1;
    while (parts < 16 && 2 * parts * 256 < N + 256 && 2 * parts * tiles * 3 <= 4 * (int64_t)cus) parts *= 2;
    return parts;
}

// Groups of four tiles where adapters have tokens enough to share their loads
// and the work outweighs the longer way of a workgroup.  One MI355X, tiles /
// groups, us: 8 adapters, K 7168, N 2048: 1000 tokens R 16 14.2 / 15.4, R 64 33.9 / 23.1;
// 2000 R 16 17.0 / 18.8, R 32 26.7 / 20.4; 8192 R 16 50.9 / 41.8, R 64 108.7 / 56.0; K
// 4096, N 2048: 8 adapters R 128, 300 tokens 21.3 / 29.3, 600 35.8 / 29.6.  Around 24
// tokens per adapter the two are about even where the tokens are spread over all
// adapters (R 64, of 255 adapters, K 7168, N 2048: 16 each 91 / 104, 20 115 / 113, 24 120 /
// 119; K 4096: 10 each 49 / 54, 20 64 / 58, 32 106 / 92; K 2048, N 5000, of 60: 16 29 / 37,
// 24 33 / 32; R 16, K 4096: 16 28.7 / 32.7, 23 40.5 / 39.9, 32 47.8 / 47.7).
// The count is that of the table's adapters: which of them occur the host does
// not know.  Few long runs of tokens over a large table therefore keep to tiles
// (7 runs, 255 adapters, K 4096, N 2048: R 64, 4000 tokens 38.8 / 33.6, 6000 55.9 / 45.4;
// at R 16, 21.1 / 25.6 and 27.7 / 35.9, tiles are the faster ones).
// Workgroups per compute unit of the table: along K eight (tiles: most of a
// table may be empty, and a full one loses little; 256 tiles, R 64, K 7168, first
// kernel, 2 splits / 8, us: 14 in use 17.5 / 6.3, all 34 / 35; R 16 8.1 / 3.7, 10.8 / 11.6)
// or four (groups; 8192 tokens, K 7168, N 2048, both kernels: R 64 3 splits 54.6 us, 5
// 52.7, 7 51.8, 8 53.8, 10 56.4; R 16 44.4, 42.3, 39.5, 40.2, 41.2), along N four or eight,
// and parts of at most 1024 of N (440 and 631 tiles, R 16, K 2048, N 7168, both kernels, 2
// or 1 parts / 7: 64 in use 25.7 / 15.2, 256 49.6 / 40.4); parts of K of 512 and parts
// of N of 256 at least.  A single tile has 8 splits at most, whose sums are
// loaded at once (K 7168, N 2048, 14 splits of 512 / 8 of 896: one token R 104 21.1 / 18.8;
// 200 of 3 adapters R 64 15.9 / 14.9).
AdapterPlan adapter_plan(int64_t T, int64_t L, int64_t rows, int64_t N, int64_t K, int64_t R, int cus) {
    AdapterPlan pl{};
    pl.tiles = rows / 16;
    pl.whole = adapter_whole_parts(T, pl.tiles, N, R, cus);
    pl.group = T >= 24 * (L + 1) && T * R >= 48 << 10 ? 4 : 1;
    pl.groups = std::max<int64_t>(cdiv(pl.tiles, pl.group), 1);
    auto share = [&](int64_t len, int64_t most, int64_t step, int64_t wgs) {
        const int64_t parts = std::clamp(wgs / pl.groups, (int64_t)1, std::max<int64_t>(most, 1));
        return std::max(cdiv(cdiv(len, parts), step), (int64_t)1) * step;
    };
    const int64_t k_most = cdiv(K, 512);
    pl.k_range = share(K, pl.group == 1 ? std::min<int64_t>(k_most, 8) : k_most, 128, (pl.group == 1 ? 8 : 4) * cus);
    pl.splits = cdiv(K, pl.k_range);
    const int64_t n_step = pl.group == 4 && R > 32 ? 512 : 256;       // 64 columns per wave
    pl.n_range = share(N, cdiv(N, n_step), n_step, (pl.group == 1 ? 4 : 8) * cus);
    if (pl.group == 1) pl.n_range = std::min<int64_t>(pl.n_range, 1024);
    return pl;
}

// Both launches fit, found before the first one is enqueued.  The grids of groups
// are whole 8s, and their second kernel has up to 512 threads.
bool adapter_grids_ok(const AdapterPlan& pl, int64_t N) {
    const int64_t wgs = pl.groups * std::max(pl.splits, cdiv(N, pl.n_range));
    return pl.group == 1 ? wgs <= max_grid(256) : cdiv(wgs, 8) * 8 <= max_grid(512);
}

fp8_status check_adapters(int64_t T, int64_t N, int64_t K, int32_t L, int32_t R, int64_t rows) {
    if (!dims_ok(T) || !dims_ok(N) || !dims_ok(K) || !dims_ok(rows) || L < 1 || R < 1) return FP8_ERR_INVALID_ARG;
    if (K % 128 || K == 0 || R % 8 || rows % 16) return FP8_ERR_SHAPE;
    if (R > fp8k::kAdapterMaxR || K > kMaxGemmK) return FP8_ERR_UNSUPPORTED;
    return FP8_OK;
}

// Grids of groups in whole 8s: a workgroup's die is its index modulo 8.
template <int RT, int G>
void launch_adapter_down(const fp8k::AdapterParams& p, const AdapterPlan& pl, hipStream_t s) {
    const int64_t wgs = pl.groups * p.splits;
    if (pl.group == 1) hipLaunchKernelGGL((fp8k::adapter_down_kernel<RT, G>), dim3((unsigned)wgs), dim3(256), 0, s, p);
    else hipLaunchKernelGGL((fp8k::adapter_down_group_kernel<RT, RT <= 4 ? 128 : 64, RT == 4 ? 3 : 2>), dim3((unsigned)(cdiv(wgs, 8) * 8)), dim3(256), 0, s, p, pl.groups);
}
template <int RS>
void launch_adapter_up(const fp8k::AdapterParams& p, const AdapterPlan& pl, hipStream_t s) {
    const int64_t wgs = pl.groups * p.parts;
    if (pl.group == 1) hipLaunchKernelGGL((fp8k::adapter_up_kernel<RS>), dim3((unsigned)wgs), dim3(256), 0, s, p);
    else {
        const dim3 grid((unsigned)(cdiv(wgs, 8) * 8)), block(64 * fp8k::adapter_up_waves(RS));
        const bool lines = whole_lines(p.N, FP8_TYPE_BF16, p.y) && aligned(p.out, kLine);
        if (lines) hipLaunchKernelGGL((fp8k::adapter_up_group_kernel<RS, true>), grid, block, 0, s, p, pl.groups);
        else hipLaunchKernelGGL((fp8k::adapter_up_group_kernel<RS, false>), grid, block, 0, s, p, pl.groups);
    }
}

}  // namespace

extern "C" {

fp8_status fp8_route_topk(const void* logits, int64_t T, int32_t E, int32_t k, int32_t type, int32_t renormalize,
                          float scale, float* weights, int32_t* ids, void* stream) {
    const fp8_status st = check_route(T, E, k, type);
    if (st != FP8_OK) return st;
    if (T == 0) return FP8_OK;
    if (!logits || !weights || !ids) return FP8_ERR_INVALID_ARG;
    if (!aligned(logits, type_size(type)) || !aligned(weights, 4) || !aligned(ids, 4)) return FP8_ERR_ALIGNMENT;
    int cus = 0;
    const fp8_status dev = current_device_cus(&cus);
    if (dev != FP8_OK) return dev;
    fp8k::RouteParams p{};
    p.logits = logits; p.w = weights; p.ids = ids;
    p.T = T; p.E = E; p.k = k; p.scale = scale; p.renorm = renormalize != 0;
    if (type == FP8_TYPE_F32) launch_route<float, false>(p, (hipStream_t)stream);
    else launch_route<uint16_t, false>(p, (hipStream_t)stream);
    return launch_status();
}

fp8_status fp8_route_topk_grad(const float* dweights, const void* logits, const int32_t* ids, int64_t T, int32_t E,
                               int32_t k, int32_t type, int32_t renormalize, float scale, void* dlogits,
                               void* stream) {
    const fp8_status st = check_route(T, E, k, type);
    if (st != FP8_OK) return st;
    if (T == 0) return FP8_OK;
    if (!dweights || !logits || !ids || !dlogits) return FP8_ERR_INVALID_ARG;
    if (!aligned(logits, type_size(type)) || !aligned(dlogits, type_size(type)) || !aligned(dweights, 4) || !aligned(ids, 4))
        return FP8_ERR_ALIGNMENT;
    int cus = 0;
    const fp8_status dev = current_device_cus(&cus);
    if (dev != FP8_OK) return dev;
    fp8k::RouteParams p{};
    p.logits = logits; p.ids = const_cast<int32_t*>(ids); p.dw = dweights; p.dlogits = dlogits;
    p.T = T; p.E = E; p.k = k; p.scale = scale; p.renorm = renormalize != 0;
    if (type == FP8_TYPE_F32) launch_route<float, true>(p, (hipStream_t)stream);
    else launch_route<uint16_t, true>(p, (hipStream_t)stream);
    return launch_status();
}

int64_t fp8_expert_rows(int64_t pairs, int32_t E, int32_t align) {
    if (pairs < 0 || pairs > kMaxDim / 2 || E < 1 || align < 1) return -1;
    return (pairs + std::min<int64_t>(E, pairs) * (align - 1)) / align * align;
}

size_t fp8_expert_sort_workspace_size(int64_t pairs, int32_t E) {
    if (check_sort(pairs, E, 4) != FP8_OK) return 0;
    return sort_bytes(pairs, E + 1);
}

fp8_status fp8_expert_sort_contiguous(const void* ids, int32_t id_bytes, int64_t pairs, int32_t E, int32_t align,
                                      int64_t rows, int32_t keep, int32_t* pos, int32_t* src, int32_t* m_indices,
                                      int32_t* counts, void* workspace, size_t workspace_bytes, void* stream) {
    const fp8_status st = check_sort(pairs, E, id_bytes);
    if (st != FP8_OK) return st;
    if (!dims_ok(rows) || align < 1 || align > 1024 || (align & (align - 1))) return FP8_ERR_INVALID_ARG;
    if ((pairs && !ids) || (rows && (!src || !m_indices))) return FP8_ERR_INVALID_ARG;
    for (const void* q : {(const void*)pos, (const void*)src, (const void*)m_indices, (const void*)counts})
        if (!aligned(q, 4)) return FP8_ERR_ALIGNMENT;
    if (!aligned(ids, id_bytes)) return FP8_ERR_ALIGNMENT;
    fp8k::SortParams p{};
    p.ids = ids; p.pos = pos; p.src = src; p.m_indices = m_indices; p.counts = counts; p.contiguous = true;
    p.pairs = pairs; p.rows = rows; p.E = E; p.bins = keep ? E + 1 : E; p.align = align; p.wide = id_bytes == 8;
    return run_sort(p, workspace, workspace_bytes, (hipStream_t)stream);
}

fp8_status fp8_expert_sort_masked(const void* ids, int32_t id_bytes, int64_t pairs, int32_t E, int64_t max_m,
                                  int32_t* pos, int32_t* src, int32_t* masked_m, void* workspace,
                                  size_t workspace_bytes, void* stream) {
    const fp8_status st = check_sort(pairs, E, id_bytes);
    if (st != FP8_OK) return st;
    if (!dims_ok(max_m)) return FP8_ERR_INVALID_ARG;
    if (E * max_m > kMaxDim / 2) return FP8_ERR_UNSUPPORTED;
    if ((pairs && !ids) || (max_m && !src) || !masked_m) return FP8_ERR_INVALID_ARG;
    for (const void* q : {(const void*)pos, (const void*)src, (const void*)masked_m})
        if (!aligned(q, 4)) return FP8_ERR_ALIGNMENT;
    if (!aligned(ids, id_bytes)) return FP8_ERR_ALIGNMENT;
    fp8k::SortParams p{};
    p.ids = ids; p.pos = pos; p.src = src; p.counts = masked_m;
    p.pairs = pairs; p.rows = E * max_m; p.E = E; p.bins = E; p.align = 1; p.max_m = max_m; p.wide = id_bytes == 8;
    return run_sort(p, workspace, workspace_bytes, (hipStream_t)stream);
}

fp8_status fp8_expert_dispatch(const void* x, const int32_t* pos, const int32_t* src, void* xs, int64_t T, int32_t k,
                               int64_t rows, int64_t K, int32_t type, void* stream) {
    const fp8_status st = check_rows(T, k, rows, K, type);
    if (st != FP8_OK) return st;
    if (rows == 0 || K == 0 || (T == 0 && !src)) return FP8_OK;
    fp8k::RowsParams p{};
    p.x = x; p.out = xs; p.pos = pos; p.src = src; p.T = T; p.rows = rows; p.W = K; p.k = k;
    dim3 grid;
    const fp8_status g = rows_grid(p, 64 * fp8k::kRowVecs * 16 / (int64_t)type_size(type), &grid);
    if (g != FP8_OK) return g;
    if ((T && (!x || !pos)) || !xs) return FP8_ERR_INVALID_ARG;
    if (!aligned(x, type_size(type)) || !aligned(xs, type_size(type)) || !aligned(pos, 4) || !aligned(src, 4))
        return FP8_ERR_ALIGNMENT;
    int cus = 0;
    const fp8_status dev = current_device_cus(&cus);
    if (dev != FP8_OK) return dev;
    if (type == FP8_TYPE_F32) hipLaunchKernelGGL(fp8k::expert_dispatch_kernel<float>, grid, dim3(256), 0, (hipStream_t)stream, p);
    else hipLaunchKernelGGL(fp8k::expert_dispatch_kernel<uint16_t>, grid, dim3(256), 0, (hipStream_t)stream, p);
    return launch_status();
}

fp8_status fp8_expert_dispatch_quant(const void* x, const int32_t* pos, uint8_t* xq, float* sa, int64_t T, int32_t k,
                                     int64_t rows, int64_t K, int32_t type, uint32_t flags, void* stream) {
    const fp8_status st = check_rows(T, k, rows, K, type);
    if (st != FP8_OK) return st;
    if (flags & ~FP8_FLAG_UE8M0) return FP8_ERR_INVALID_ARG;
    if (K % 128) return FP8_ERR_SHAPE;
    if (T == 0 || rows == 0 || K == 0) return FP8_OK;
    fp8k::RowsParams p{};
    p.x = x; p.out = xq; p.sa = sa; p.pos = pos; p.T = T; p.rows = rows; p.W = K; p.k = k;
    dim3 grid;
    const fp8_status g = rows_grid(p, 1024, &grid, 8);
    if (g != FP8_OK) return g;
    if (!x || !pos || !xq || !sa) return FP8_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(xq) || !aligned16(sa) || !aligned(pos, 4)) return FP8_ERR_ALIGNMENT;
    int cus = 0;
    const fp8_status dev = current_device_cus(&cus);
    if (dev != FP8_OK) return dev;
    const hipStream_t s = (hipStream_t)stream;
    const bool pow2 = flags & FP8_FLAG_UE8M0;
    const bool past = T * k * K > kCacheBytes;
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, p); };
    if (type == FP8_TYPE_F32) {
        if (past) pow2 ? go(fp8k::expert_dispatch_quant_kernel<float, true, true>) : go(fp8k::expert_dispatch_quant_kernel<float, false, true>);
        else pow2 ? go(fp8k::expert_dispatch_quant_kernel<float, true, false>) : go(fp8k::expert_dispatch_quant_kernel<float, false, false>);
    } else {
        if (past) pow2 ? go(fp8k::expert_dispatch_quant_kernel<uint16_t, true, true>) : go(fp8k::expert_dispatch_quant_kernel<uint16_t, false, true>);
        else pow2 ? go(fp8k::expert_dispatch_quant_kernel<uint16_t, true, false>) : go(fp8k::expert_dispatch_quant_kernel<uint16_t, false, false>);
    }
    return launch_status();
}

fp8_status fp8_expert_combine(const void* y, const int32_t* pos, const float* weights, void* out, int64_t T,
                              int32_t k, int64_t rows, int64_t N, int32_t type, void* stream) {
    const fp8_status st = check_rows(T, k, rows, N, type);
    if (st != FP8_OK) return st;
    if (T == 0 || N == 0) return FP8_OK;
    fp8k::RowsParams p{};
    p.x = y; p.out = out; p.pos = pos; p.w = weights; p.T = T; p.rows = rows; p.W = N; p.k = k;
    dim3 grid;
    const fp8_status g = rows_grid(p, 64 * fp8k::kCombineVecs * 16 / (int64_t)type_size(type), &grid);
    if (g != FP8_OK) return g;
    if ((rows && !y) || !pos || !out) return FP8_ERR_INVALID_ARG;
    if (!aligned(y, type_size(type)) || !aligned(out, type_size(type)) || !aligned(pos, 4) || !aligned(weights, 4))
        return FP8_ERR_ALIGNMENT;
    int cus = 0;
    const fp8_status dev = current_device_cus(&cus);
    if (dev != FP8_OK) return dev;
    const bool lines = whole_lines(N, type, y);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, (hipStream_t)stream, p); };
    if (type == FP8_TYPE_F32) lines ? go(fp8k::expert_combine_kernel<float, true>) : go(fp8k::expert_combine_kernel<float, false>);
    else lines ? go(fp8k::expert_combine_kernel<uint16_t, true>) : go(fp8k::expert_combine_kernel<uint16_t, false>);
    return launch_status();
}

fp8_status fp8_expert_combine_grad(const void* dout, const void* y, const int32_t* pos, const float* weights,
                                   const int32_t* src, void* dy, float* dweights, int64_t T, int32_t k, int64_t rows,
                                   int64_t N, int32_t type, void* stream) {
    const fp8_status st = check_rows(T, k, rows, N, type);
    if (st != FP8_OK) return st;
    if (!dy && !dweights) return FP8_OK;
    if (T == 0 && (!dy || !src || rows == 0 || N == 0)) return FP8_OK;
    const int64_t wgs = T + (dy && src ? cdiv(rows, 4 * fp8k::kClearRows) : 0);
    if (wgs > max_grid(256)) return FP8_ERR_UNSUPPORTED;
    if ((T && (!pos || (N && !dout))) || (T && rows && N && dweights && !y)) return FP8_ERR_INVALID_ARG;
    for (const void* q : {dout, y, (const void*)dy})
        if (!aligned(q, type_size(type))) return FP8_ERR_ALIGNMENT;
    for (const void* q : {(const void*)pos, (const void*)weights, (const void*)src, (const void*)dweights})
        if (!aligned(q, 4)) return FP8_ERR_ALIGNMENT;
    int cus = 0;
    const fp8_status dev = current_device_cus(&cus);
    if (dev != FP8_OK) return dev;
    fp8k::RowsParams p{};
    p.x = dout; p.y = y; p.out = dy; p.dw = dweights; p.pos = pos; p.w = weights; p.src = dy ? src : nullptr;
    p.T = T; p.rows = rows; p.W = N; p.k = k;
    p.work = T;
    const dim3 grid((unsigned)wgs);
    const bool few = k <= 4, lines = whole_lines(N, type, y) && aligned(dy, kLine);
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, (hipStream_t)stream, p); };
    if (type == FP8_TYPE_F32) {
        if (lines) few ? go(fp8k::expert_combine_grad_kernel<float, 4, true>) : go(fp8k::expert_combine_grad_kernel<float, 8, true>);
        else few ? go(fp8k::expert_combine_grad_kernel<float, 4, false>) : go(fp8k::expert_combine_grad_kernel<float, 8, false>);
    } else {
        if (lines) few ? go(fp8k::expert_combine_grad_kernel<uint16_t, 4, true>) : go(fp8k::expert_combine_grad_kernel<uint16_t, 8, true>);
        else few ? go(fp8k::expert_combine_grad_kernel<uint16_t, 4, false>) : go(fp8k::expert_combine_grad_kernel<uint16_t, 8, false>);
    }
    return launch_status();
}

size_t fp8_adapters_workspace_size(int64_t T, int32_t L, int64_t rows, int64_t N, int64_t K, int32_t R) {
    if (check_adapters(T, N, K, L, R, rows) != FP8_OK) return 0;
    int cus = 0;
    if (current_device_cus(&cus) != FP8_OK) return 0;
    const AdapterPlan pl = adapter_plan(T, L, rows, N, K, R, cus);
    return adapter_grids_ok(pl, N) ? pl.bytes(R) : 0;
}

fp8_status fp8_adapters_plan(int64_t T, int32_t L, int64_t rows, int64_t N, int64_t K, int32_t R, int32_t compute_units,
                             fp8_adapters_plan_t* plan) {
    if (!plan || compute_units <= 0) return FP8_ERR_INVALID_ARG;
    const fp8_status st = check_adapters(T, N, K, L, R, rows);
    if (st != FP8_OK) return st;
    const AdapterPlan pl = adapter_plan(T, L, rows, N, K, R, compute_units);
    if (!adapter_grids_ok(pl, N)) return FP8_ERR_UNSUPPORTED;
    *plan = fp8_adapters_plan_t{};
    plan->tiles = pl.tiles;
    plan->group = pl.group;
    plan->k_splits = pl.splits;
    plan->k_range = pl.k_range;
    plan->n_range = pl.n_range;
    plan->workspace_bytes = pl.bytes(R);
    plan->whole = pl.whole;
    return FP8_OK;
}

fp8_status fp8_add_adapters(const uint16_t* x, const uint16_t* a, const uint16_t* b, const float* scale,
                            const int32_t* src, const int32_t* index, const uint16_t* y, uint16_t* out, int64_t T,
                            int64_t N, int64_t K, int32_t L, int32_t R, int64_t rows, void* workspace,
                            size_t workspace_bytes, void* stream) {
    const fp8_status st = check_adapters(T, N, K, L, R, rows);
    if (st != FP8_OK) return st;
    if (T == 0 || N == 0 || rows == 0) return FP8_OK;
    if (!x || !a || !b || !scale || !src || !index || !y || !out || (workspace_bytes && !workspace)) return FP8_ERR_INVALID_ARG;
    if (!aligned16(x) || !aligned16(a) || !aligned16(b) || !aligned16(workspace)) return FP8_ERR_ALIGNMENT;
    if (!aligned(scale, 4) || !aligned(src, 4) || !aligned(index, 4) || !aligned(y, 2) || !aligned(out, 2))
        return FP8_ERR_ALIGNMENT;
    int cus = 0;
    const fp8_status dev = current_device_cus(&cus);
    if (dev != FP8_OK) return dev;
    const AdapterPlan pl = adapter_plan(T, L, rows, N, K, R, cus);
    if (!adapter_grids_ok(pl, N)) return FP8_ERR_UNSUPPORTED;
    if (workspace_bytes < pl.bytes(R)) return FP8_ERR_SCRATCH;
    fp8k::AdapterParams p{};
    p.x = x; p.a = a; p.b = b; p.scale = scale; p.src = src; p.index = index; p.y = y; p.out = out;
    p.z = static_cast<float*>(workspace);
    p.T = T; p.N = N; p.K = K; p.tiles = pl.tiles; p.k_range = pl.k_range; p.n_range = pl.n_range;
    p.L = L; p.R = R; p.splits = (int32_t)pl.splits; p.parts = (int32_t)cdiv(N, pl.n_range);
    const hipStream_t s = (hipStream_t)stream;
    if (pl.whole) {
        p.parts = pl.whole;
        const dim3 grid((unsigned)(cdiv(pl.tiles, 8) * 8 * pl.whole)), block(64 * fp8k::kWholeWaves);
        if (R <= 32) hipLaunchKernelGGL(fp8k::adapter_whole_kernel<1>, grid, block, 0, s, p);
        else hipLaunchKernelGGL(fp8k::adapter_whole_kernel<2>, grid, block, 0, s, p);
        return launch_status();
    }
    // (one tile: as many steps of K in flight as two chunks leave registers for)
    if (R <= 16) launch_adapter_down<1, 4>(p, pl, s);
    else if (R <= 32) launch_adapter_down<2, 4>(p, pl, s);
    else if (R <= 64) launch_adapter_down<4, 2>(p, pl, s);
    else launch_adapter_down<8, 1>(p, pl, s);
    const fp8_status run = launch_status();
    if (run != FP8_OK) return run;
    if (R <= 32) launch_adapter_up<1>(p, pl, s);
    else if (R <= 64) launch_adapter_up<2>(p, pl, s);
    else launch_adapter_up<4>(p, pl, s);
    return launch_status();
}

}  // extern "C"
