// api.cu -- the exported C ABI (include/q4.h): host-side argument checks,
// plan selection and launches.  Nothing here allocates or synchronises except
// q4_check.  Every product call names its weight layout and the weight
// buffer's byte count, checked against each other before anything runs.
#include <stdio.h>
#include <string.h>

#include <cmath>
#include <mutex>

#include "serve.cuh"
#include "tcgen05.cuh"

__device__ unsigned int g_q4_error = 0u;

namespace q4 {

static thread_local char t_last_error[256] = "";

q4_status cuda_fail(cudaError_t e)
{
    snprintf(t_last_error, sizeof(t_last_error), "%s: %s", cudaGetErrorName(e),
             cudaGetErrorString(e));
    return Q4_ERR_CUDA;
}

static inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static inline bool valid_dtype(q4_dtype t) { return t == Q4_F32 || t == Q4_BF16 || t == Q4_F16; }

// Per-device cached facts.
struct DevInfo {
    int sm_count = 0;
    unsigned int *err = nullptr;
};
static std::mutex g_mu;
static DevInfo g_dev[64];

static const DevInfo *dev_info()
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    std::lock_guard<std::mutex> lock(g_mu);
    DevInfo &d = g_dev[dev];
    if (d.sm_count == 0) {
        int sms = 0;
        if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return nullptr;
        void *p = nullptr;
        if (cudaGetSymbolAddress(&p, g_q4_error) != cudaSuccess) return nullptr;
        d.err = static_cast<unsigned int *>(p);
        d.sm_count = sms;
    }
    return &d;
}

unsigned int *device_error_word()
{
    const DevInfo *d = dev_info();
    return d ? d->err : nullptr;
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                             &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// The error word for the store checks of the packing kernels: looked up
// only in debug builds, so release calls stay free of the device query.
static inline unsigned int *debug_err() { return kDebugBounds ? device_error_word() : nullptr; }

// Stores i + 1 into byte i of a 32-byte buffer through the store check,
// declaring an extent of 16.
__global__ void k_bounds_selftest(uint8_t *buf, unsigned int *err)
{
    const int i = threadIdx.x;
    if (i < 32 && store_ok(i, 16, err)) buf[i] = static_cast<uint8_t>(i + 1);
}

static inline bool sizes_ok(int64_t N, int64_t K)
{
    return N >= 1 && K >= G && K % G == 0 && N <= (1LL << 30) && K <= (1LL << 30) &&
           N * K <= (1LL << 40);
}

size_t weight_bytes(int64_t N, int64_t K, q4_layout layout)
{
    if (!sizes_ok(N, K)) return 0;
    const size_t tile = layout == Q4_LAYOUT_TILED ? TILE_BYTES
                        : layout == Q4_LAYOUT_COMPACT ? CMP_TILE_BYTES
                                                      : 0;
    return static_cast<size_t>((N + TILE_ROWS - 1) / TILE_ROWS) * static_cast<size_t>(K / G) * tile;
}

// The weight buffer matches its declared layout and shape byte for byte.
static inline bool weights_ok(int64_t N, int64_t K, q4_layout layout, size_t qw_bytes)
{
    const size_t need = weight_bytes(N, K, layout);
    return need != 0 && qw_bytes == need;
}

static q4_status gemv_common(const void *x, q4_dtype xt, int64_t M, int64_t N, int64_t K,
                             const void *qw, q4_layout layout, size_t qw_bytes, void *y,
                             q4_dtype yt, void *workspace, size_t workspace_bytes,
                             cudaStream_t stream, int path, int debug_no_copy, uint64_t wait_ns)
{
    if (!x || !qw || !y) return Q4_ERR_INVALID_ARG;
    if (!sizes_ok(N, K) || N > (1LL << 28)) return Q4_ERR_INVALID_ARG;
    if (!weights_ok(N, K, layout, qw_bytes)) return Q4_ERR_INVALID_ARG;
    const bool cmp = layout == Q4_LAYOUT_COMPACT;
    if (M < 1 || M > Q4_GEMV_MAX_M) return Q4_ERR_UNSUPPORTED;
    if (!valid_dtype(xt) || !valid_dtype(yt)) return Q4_ERR_UNSUPPORTED;
    if (path == PATH_FMA && (M != 1 || cmp)) return Q4_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(qw) || !aligned16(y) || !aligned16(workspace))
        return Q4_ERR_MISALIGNED;
    const DevInfo *d = dev_info();
    if (!d) return cuda_fail(cudaGetLastError());
    const GemvPlan plan = gemv_plan(static_cast<int>(M), static_cast<int>(N), static_cast<int>(K),
                                    xt, path, d->sm_count, cmp);
    if (plan.workspace > 0 && (!workspace || workspace_bytes < plan.workspace))
        return Q4_ERR_INVALID_ARG;
    GemvArgs a{};
    a.x = x;
    a.xt = xt;
    a.M = static_cast<int>(M);
    a.N = static_cast<int>(N);
    a.K = static_cast<int>(K);
    a.qw = static_cast<const uint8_t *>(qw);
    a.y = y;
    a.yt = yt;
    a.maxc = plan.maxc;
    if (plan.maxc > 1) {
        const size_t counters = gemv_counter_bytes(N);
        a.count = static_cast<unsigned int *>(workspace);
        a.partial = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + counters);
        // store checks use the plan's own extents (inside the caller's buffer)
        a.count_len = plan.nrb;
        a.partial_len = static_cast<int64_t>((plan.workspace - counters) / sizeof(float));
    }
    a.wait_ns = wait_ns;
    a.err = d->err;
    a.debug_no_copy = debug_no_copy;
    const cudaError_t e = gemv_launch(plan, a, stream);
    return e == cudaSuccess ? Q4_OK : cuda_fail(e);
}


// ------------------------------------------------------- serving operators
constexpr int64_t INT_MOST = 2147483647;

// The cache's fields, in the order that decides which status is returned.
static q4_status cache_ok(const q4_kv_cache *c)
{
    if (!c || !c->k || !c->v || c->blocks < 1 || c->heads < 1 || c->block_size < 1 || c->head_dim < 1)
        return Q4_ERR_INVALID_ARG;
    if (c->type != Q4_BF16 && c->type != Q4_F16) return Q4_ERR_UNSUPPORTED;
    if (c->blocks > INT_MOST || c->heads > 65536 || c->block_size > 65536 || c->block_size % 16 ||
        c->head_dim > 128 || c->head_dim % 8)
        return Q4_ERR_UNSUPPORTED;
    constexpr int64_t most = 1LL << 40;  // elements; keeps every offset far inside 64 bits
    if (c->block_stride < 0 || c->head_stride < 0 || c->token_stride < c->head_dim ||
        c->block_stride > most || c->head_stride > most || c->token_stride > most)
        return Q4_ERR_INVALID_ARG;
    // Of several blocks, heads or tokens none may share its elements with
    // another: sorted by stride, each dimension steps over the ones inside.
    struct {
        int64_t n, stride;
    } d[3] = {{c->block_size, c->token_stride}, {c->heads, c->head_stride}, {c->blocks, c->block_stride}};
    std::sort(d, d + 3, [](const auto &x, const auto &y) { return x.stride < y.stride; });
    int64_t extent = c->head_dim;
    for (const auto &x : d) {
        if (x.n == 1) continue;
        if (x.stride < extent) return Q4_ERR_INVALID_ARG;
        if (x.stride >= (1LL << 39) || x.stride > (1LL << 60) / x.n) return Q4_ERR_UNSUPPORTED;
        extent += (x.n - 1) * x.stride;
    }
    if (!aligned16(c->k) || !aligned16(c->v) || c->block_stride % 8 || c->head_stride % 8 ||
        c->token_stride % 8)
        return Q4_ERR_MISALIGNED;
    return Q4_OK;
}

}  // namespace q4

using namespace q4;

extern "C" {

static q4_status quantize_common(const float *w, int64_t N, int64_t K, uint8_t *packed,
                                 float *scale, uint8_t *zero, bool symmetric, q4_stream_t stream)
{
    if (!w || !packed || !scale || !zero || !sizes_ok(N, K)) return Q4_ERR_INVALID_ARG;
    if (!aligned16(w)) return Q4_ERR_MISALIGNED;
    const cudaError_t e = quantize_launch(w, N, K, packed, scale, zero, symmetric, debug_err(),
                                          reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? Q4_OK : cuda_fail(e);
}

q4_status q4_quantize(const float *w, int64_t N, int64_t K, uint8_t *packed, float *scale,
                      uint8_t *zero, q4_stream_t stream)
{
    return quantize_common(w, N, K, packed, scale, zero, false, stream);
}

q4_status q4_quantize_sym(const float *w, int64_t N, int64_t K, uint8_t *packed, float *scale,
                          uint8_t *zero, q4_stream_t stream)
{
    return quantize_common(w, N, K, packed, scale, zero, true, stream);
}

size_t q4_weight_bytes(int64_t N, int64_t K, q4_layout layout)
{
    return weight_bytes(N, K, layout);
}

q4_status q4_repack(const uint8_t *packed, const float *scale, const uint8_t *zero, int64_t N,
                    int64_t K, void *qw, q4_stream_t stream)
{
    if (!packed || !scale || !zero || !qw || !sizes_ok(N, K)) return Q4_ERR_INVALID_ARG;
    if (!aligned16(qw)) return Q4_ERR_MISALIGNED;
    const cudaError_t e = repack_launch(packed, scale, zero, N, K, static_cast<uint8_t *>(qw),
                                        debug_err(), reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? Q4_OK : cuda_fail(e);
}

q4_status q4_unpack(const void *qw, int64_t N, int64_t K, uint8_t *packed, float *scale,
                    uint8_t *zero, q4_stream_t stream)
{
    if (!packed || !scale || !zero || !qw || !sizes_ok(N, K)) return Q4_ERR_INVALID_ARG;
    if (!aligned16(qw)) return Q4_ERR_MISALIGNED;
    const cudaError_t e = unpack_launch(static_cast<const uint8_t *>(qw), N, K, packed, scale,
                                        zero, debug_err(), reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? Q4_OK : cuda_fail(e);
}

q4_status q4_repack_compact(const uint8_t *packed, const float *scale, const uint8_t *zero,
                            int64_t N, int64_t K, void *qw, q4_stream_t stream)
{
    if (!packed || !scale || !zero || !qw || !sizes_ok(N, K)) return Q4_ERR_INVALID_ARG;
    if (!aligned16(qw)) return Q4_ERR_MISALIGNED;
    const cudaError_t e = repack_compact_launch(packed, scale, zero, N, K,
                                                static_cast<uint8_t *>(qw), debug_err(),
                                                reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? Q4_OK : cuda_fail(e);
}

q4_status q4_unpack_compact(const void *qw, int64_t N, int64_t K, uint8_t *packed,
                            uint16_t *scale16, uint8_t *zero, q4_stream_t stream)
{
    if (!packed || !scale16 || !zero || !qw || !sizes_ok(N, K)) return Q4_ERR_INVALID_ARG;
    if (!aligned16(qw)) return Q4_ERR_MISALIGNED;
    const cudaError_t e = unpack_compact_launch(static_cast<const uint8_t *>(qw), N, K, packed,
                                                scale16, zero, debug_err(),
                                                reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? Q4_OK : cuda_fail(e);
}

q4_status q4_xsum(const void *x, q4_dtype xt, int64_t M, int64_t K, float *xsum,
                  q4_stream_t stream)
{
    if (!x || !xsum || M < 1 || !sizes_ok(M, K)) return Q4_ERR_INVALID_ARG;
    if (!valid_dtype(xt)) return Q4_ERR_UNSUPPORTED;
    const cudaError_t e = xsum_launch(x, xt, M, K, xsum, debug_err(),
                                      reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? Q4_OK : cuda_fail(e);
}

size_t q4_gemv_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    if (M < 1 || M > Q4_GEMV_MAX_M || !sizes_ok(N, K)) return 0;
    const DevInfo *d = dev_info();
    if (!d) return 0;
    // the largest need over activation types and paths, so one buffer serves
    // every call with this shape
    size_t need = 0;
    const q4_dtype types[3] = {Q4_BF16, Q4_F16, Q4_F32};
    const int paths[3] = {PATH_AUTO, PATH_MMA, PATH_FMA};
    for (int cmp = 0; cmp < 2; ++cmp)
        for (q4_dtype t : types)
            for (int p : paths) {
                if (p == PATH_FMA && (M != 1 || cmp)) continue;
                const GemvPlan g = gemv_plan(static_cast<int>(M), static_cast<int>(N),
                                             static_cast<int>(K), t, p, d->sm_count, cmp != 0);
                need = std::max(need, g.workspace);
            }
    return need;
}

q4_status q4_gemv(const void *x, q4_dtype xt, int64_t M, int64_t N, int64_t K, const void *qw,
                  q4_layout layout, size_t qw_bytes, void *y, q4_dtype yt, void *workspace,
                  size_t workspace_bytes, q4_stream_t stream)
{
    return gemv_common(x, xt, M, N, K, qw, layout, qw_bytes, y, yt, workspace, workspace_bytes,
                       reinterpret_cast<cudaStream_t>(stream), PATH_AUTO, 0, 1000000000ull);
}

q4_status q4_gemv_path(const void *x, q4_dtype xt, int64_t M, int64_t N, int64_t K,
                       const void *qw, q4_layout layout, size_t qw_bytes, void *y, q4_dtype yt,
                       void *workspace, size_t workspace_bytes, int path, q4_stream_t stream)
{
    if (path != PATH_AUTO && path != PATH_FMA && path != PATH_MMA) return Q4_ERR_UNSUPPORTED;
    return gemv_common(x, xt, M, N, K, qw, layout, qw_bytes, y, yt, workspace, workspace_bytes,
                       reinterpret_cast<cudaStream_t>(stream), path, 0, 1000000000ull);
}

q4_status q4_gemv_timeout_selftest(const void *x, q4_dtype xt, int64_t M, int64_t N, int64_t K,
                                   const void *qw, q4_layout layout, size_t qw_bytes, void *y,
                                   q4_dtype yt, void *workspace, size_t workspace_bytes,
                                   q4_stream_t stream)
{
    return gemv_common(x, xt, M, N, K, qw, layout, qw_bytes, y, yt, workspace, workspace_bytes,
                       reinterpret_cast<cudaStream_t>(stream), PATH_AUTO, 1, 20000000ull);
}

static q4_status gemm_common(const void *x, q4_dtype xt, int64_t M, int64_t N, int64_t K,
                             const void *qw, q4_layout layout, size_t qw_bytes, void *y,
                             q4_dtype yt, void *workspace, size_t workspace_bytes,
                             q4_stream_t stream, int debug_no_copy, uint64_t wait_ns)
{
    if (!x || !qw || !y) return Q4_ERR_INVALID_ARG;
    if (M < 1 || M > (1LL << 30) || !sizes_ok(N, K) || N > (1LL << 30)) return Q4_ERR_INVALID_ARG;
    if (!weights_ok(N, K, layout, qw_bytes)) return Q4_ERR_INVALID_ARG;
    if ((xt != Q4_BF16 && xt != Q4_F16) || !valid_dtype(yt)) return Q4_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(qw) || !aligned16(y) || !aligned16(workspace))
        return Q4_ERR_MISALIGNED;
    const DevInfo *d = dev_info();
    if (!d) return cuda_fail(cudaGetLastError());
    const GemmPlan plan = gemm_plan(M, N, K, d->sm_count);
    if (plan.workspace > 0 && (!workspace || workspace_bytes < plan.workspace))
        return Q4_ERR_INVALID_ARG;
    cudaError_t e = cudaSuccess;
    const q4_status st = gemm_run(plan, x, xt, M, N, K, static_cast<const uint8_t *>(qw),
                                  layout == Q4_LAYOUT_COMPACT, y, yt, workspace, d->err, wait_ns,
                                  debug_no_copy, reinterpret_cast<cudaStream_t>(stream), &e);
    if (st == Q4_ERR_CUDA) return cuda_fail(e);
    return st;
}

q4_status q4_gemm(const void *x, q4_dtype xt, int64_t M, int64_t N, int64_t K, const void *qw,
                  q4_layout layout, size_t qw_bytes, void *y, q4_dtype yt, void *workspace,
                  size_t workspace_bytes, q4_stream_t stream)
{
    return gemm_common(x, xt, M, N, K, qw, layout, qw_bytes, y, yt, workspace, workspace_bytes,
                       stream, 0, 2000000000ull);
}

size_t q4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    if (M < 1 || M > (1LL << 30) || !sizes_ok(N, K) || N > (1LL << 30)) return 0;
    const DevInfo *d = dev_info();
    if (!d) return 0;
    return gemm_plan(M, N, K, d->sm_count).workspace;
}

q4_status q4_gemm_timeout_selftest(const void *x, q4_dtype xt, int64_t M, int64_t N, int64_t K,
                                   const void *qw, q4_layout layout, size_t qw_bytes, void *y,
                                   q4_dtype yt, void *workspace, size_t workspace_bytes,
                                   q4_stream_t stream)
{
    return gemm_common(x, xt, M, N, K, qw, layout, qw_bytes, y, yt, workspace, workspace_bytes,
                       stream, 1, 20000000ull);
}

q4_status q4_cache_plan(const int32_t *cached, const int32_t *fresh, int64_t B, int64_t block_size,
                        int32_t *table, int64_t table_stride, int64_t width,
                        const int32_t *free_blocks, const int32_t *free_count,
                        int64_t free_capacity, int64_t T, int32_t *q_start, int32_t *kv_len,
                        int32_t *position, int64_t *slot, int32_t *counts, q4_stream_t stream)
{
    if (!cached || !fresh || !table || !free_blocks || !free_count || !q_start || !kv_len ||
        !position || !slot || !counts)
        return Q4_ERR_INVALID_ARG;
    if (B < 1 || block_size < 1 || width < 1 || table_stride < width || free_capacity < 1 || T < 1)
        return Q4_ERR_INVALID_ARG;
    if (B > Q4_PLAN_MAX_REQUESTS || T > INT_MOST || free_capacity > INT_MOST ||
        table_stride > (1LL << 40) || width > INT_MOST / block_size)
        return Q4_ERR_UNSUPPORTED;
    // What is written (the first six) may lie over nothing else: every CTA
    // reads the lengths, some after others have written.
    const struct {
        const void *p;
        int64_t bytes;
    } arrays[] = {{table, ((B - 1) * table_stride + width) * 4}, {q_start, (B + 1) * 4}, {kv_len, B * 4},
                  {position, T * 4}, {slot, T * 8}, {counts, 16}, {cached, B * 4}, {fresh, B * 4},
                  {free_blocks, free_capacity * 4}, {free_count, 4}};
    for (int i = 0; i < 6; ++i)
        for (int j = i + 1; j < 10; ++j) {
            const uintptr_t x = reinterpret_cast<uintptr_t>(arrays[i].p), y = reinterpret_cast<uintptr_t>(arrays[j].p);
            if (x >= y + arrays[j].bytes || y >= x + arrays[i].bytes) continue;
            // between the table's rows there is room
            const int64_t step = table_stride * 4, at = static_cast<int64_t>(y - x);
            if (i > 0 || y < x || at % step < width * 4 || at % step + arrays[j].bytes > step) return Q4_ERR_INVALID_ARG;
        }
    PlanArgs a{};
    a.cached = cached;
    a.fresh = fresh;
    a.B = static_cast<int>(B);
    a.S = static_cast<int>(block_size);
    a.table = table;
    a.table_stride = table_stride;
    a.width = static_cast<int>(width);
    a.free_blocks = free_blocks;
    a.free_count = free_count;
    a.free_capacity = static_cast<int>(free_capacity);
    a.T = static_cast<int>(T);
    a.q_start = q_start;
    a.kv_len = kv_len;
    a.position = position;
    a.slot = slot;
    a.counts = counts;
    a.err = debug_err();
    const cudaError_t e = cache_plan_launch(a, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? Q4_OK : cuda_fail(e);
}

q4_status q4_rope_append(const void *qkv, int64_t qkv_stride, int64_t T, int64_t Hq, int64_t rot,
                         q4_rope_style style, const double *freq, float factor,
                         const int32_t *position, const int64_t *slot, void *q_out,
                         int64_t q_stride, const q4_kv_cache *cache, q4_stream_t stream)
{
    if (!qkv || !position || !slot || !q_out) return Q4_ERR_INVALID_ARG;
    const q4_status st = cache_ok(cache);
    if (st != Q4_OK) return st;
    if (T < 1 || Hq < 1 || rot < 0 || rot > cache->head_dim || rot % 2 || (rot > 0 && !freq))
        return Q4_ERR_INVALID_ARG;
    if (style != Q4_ROPE_HALF && style != Q4_ROPE_INTERLEAVED) return Q4_ERR_INVALID_ARG;
    if (T > INT_MOST || Hq > 65536) return Q4_ERR_UNSUPPORTED;
    if (qkv_stride < (Hq + 2 * cache->heads) * cache->head_dim || q_stride < Hq * cache->head_dim)
        return Q4_ERR_INVALID_ARG;
    if (qkv_stride > (1LL << 30) || q_stride > (1LL << 30)) return Q4_ERR_UNSUPPORTED;
    if (!aligned16(qkv) || !aligned16(q_out) || qkv_stride % 8 || q_stride % 8)
        return Q4_ERR_MISALIGNED;
    RopeArgs a{};
    a.qkv = static_cast<const uint16_t *>(qkv);
    a.qkv_stride = qkv_stride;
    a.T = static_cast<int>(T);
    a.Hq = static_cast<int>(Hq);
    a.Hkv = static_cast<int>(cache->heads);
    a.D = static_cast<int>(cache->head_dim);
    a.rot = static_cast<int>(rot);
    a.freq = freq;
    a.factor = factor;
    a.position = position;
    a.slot = slot;
    a.q_out = static_cast<uint16_t *>(q_out);
    a.q_stride = q_stride;
    a.k = static_cast<uint16_t *>(cache->k);
    a.v = static_cast<uint16_t *>(cache->v);
    a.block_stride = cache->block_stride;
    a.head_stride = cache->head_stride;
    a.token_stride = cache->token_stride;
    a.blocks = static_cast<int>(cache->blocks);
    a.S = static_cast<int>(cache->block_size);
    a.err = debug_err();
    const cudaError_t e = rope_append_launch(a, cache->type == Q4_F16, style == Q4_ROPE_INTERLEAVED,
                                             reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? Q4_OK : cuda_fail(e);
}

// Rows (tokens times heads) of a call: their indices run on to the end of a
// tile of 256 rows, in 32 bits.
constexpr int64_t ATTN_MOST_ROWS = INT_MOST - 1023;

static bool attention_sizes_ok(int64_t max_fresh, int64_t Hq, int64_t heads, int64_t head_dim)
{
    return max_fresh >= 1 && max_fresh <= INT_MOST && heads >= 1 && Hq >= heads && Hq % heads == 0 &&
           Hq <= 65536 && head_dim >= 8 && head_dim <= 128 && head_dim % 8 == 0;
}

size_t q4_attention_workspace_bytes(int64_t max_fresh, int64_t Hq, int64_t heads, int64_t head_dim)
{
    if (!attention_sizes_ok(max_fresh, Hq, heads, head_dim)) return 0;
    const DevInfo *d = dev_info();
    if (!d) return 0;
    return attention_plan(max_fresh, Hq / heads, head_dim, d->sm_count).workspace;
}

static q4_status attention_common(const void *q, int64_t q_stride, int64_t T, int64_t Hq,
                                  const q4_kv_cache *cache, const int32_t *table,
                                  int64_t table_stride, int64_t width, const int32_t *q_start,
                                  const int32_t *kv_len, int64_t B, int64_t max_fresh, float scale,
                                  int64_t window, void *o, q4_dtype ot, int64_t o_stride, float *lse,
                                  void *workspace, size_t workspace_bytes, q4_stream_t stream,
                                  int debug_no_copy, uint64_t wait_ns)
{
    if (!q || !table || !q_start || !kv_len || !o) return Q4_ERR_INVALID_ARG;
    const q4_status st = cache_ok(cache);
    if (st != Q4_OK) return st;
    if (T < 1 || B < 1 || Hq < 1 || Hq % cache->heads || max_fresh < 1 || width < 1 ||
        table_stride < width || window < 0 || !std::isfinite(scale))
        return Q4_ERR_INVALID_ARG;
    if (ot != Q4_F32 && ot != cache->type) return Q4_ERR_UNSUPPORTED;
    if (!attention_sizes_ok(max_fresh, Hq, cache->heads, cache->head_dim) || T > ATTN_MOST_ROWS / Hq ||
        B > INT_MOST || table_stride > (1LL << 40) || width > (INT_MOST >> 1) / cache->block_size)
        return Q4_ERR_UNSUPPORTED;
    const int64_t row = Hq * cache->head_dim;
    if (q_stride < row || o_stride < row) return Q4_ERR_INVALID_ARG;
    if (q_stride > (1LL << 30) || o_stride > (1LL << 30)) return Q4_ERR_UNSUPPORTED;
    if (!aligned16(q) || !aligned16(o) || !aligned16(workspace) || q_stride % 8 || o_stride % 8 ||
        (reinterpret_cast<uintptr_t>(lse) & 3u))
        return Q4_ERR_MISALIGNED;
    const DevInfo *d = dev_info();
    if (!d) return cuda_fail(cudaGetLastError());
    const AttnPlan plan = attention_plan(max_fresh, Hq / cache->heads, cache->head_dim, d->sm_count);
    if (debug_no_copy && !plan.tc) return Q4_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < plan.workspace) return Q4_ERR_INVALID_ARG;
    AttnArgs a{};
    a.q = static_cast<const uint16_t *>(q);
    a.k = static_cast<const uint16_t *>(cache->k);
    a.v = static_cast<const uint16_t *>(cache->v);
    a.o = o;
    a.ot = ot;
    a.lse = lse;
    a.q_stride = q_stride;
    a.o_stride = o_stride;
    a.block_stride = cache->block_stride;
    a.head_stride = cache->head_stride;
    a.token_stride = cache->token_stride;
    a.table = table;
    a.table_stride = table_stride;
    a.q_start = q_start;
    a.kv_len = kv_len;
    a.T = static_cast<int>(T);
    a.B = static_cast<int>(B);
    a.Hq = static_cast<int>(Hq);
    a.Hkv = static_cast<int>(cache->heads);
    a.GQ = static_cast<int>(Hq / cache->heads);
    a.D = static_cast<int>(cache->head_dim);
    a.S = static_cast<int>(cache->block_size);
    a.by_GQ.set(a.GQ);
    a.by_S.set(a.S);
    a.blocks = static_cast<int>(cache->blocks);
    a.width = static_cast<int>(width);
    a.scale_log2 = scale * 1.4426950408889634f;
    // a window that no length reaches hides nothing
    a.window = window > INT_MOST ? 0 : static_cast<int>(window);
    a.count = static_cast<unsigned int *>(workspace);
    a.part = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + ATTN_COUNTER_BYTES);
    a.count_len = ATTN_COUNTER_BYTES / sizeof(unsigned int);
    a.wait_ns = wait_ns;
    a.debug_no_copy = debug_no_copy;
    a.part_len = static_cast<int64_t>((plan.workspace - ATTN_COUNTER_BYTES) / sizeof(float));
    a.err = d->err;
    const cudaError_t e = attention_launch(plan, a, cache->type == Q4_F16,
                                           reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? Q4_OK : cuda_fail(e);
}

q4_status q4_attention(const void *q, int64_t q_stride, int64_t T, int64_t Hq,
                       const q4_kv_cache *cache, const int32_t *table, int64_t table_stride,
                       int64_t width, const int32_t *q_start, const int32_t *kv_len, int64_t B,
                       int64_t max_fresh, float scale, int64_t window, void *o, q4_dtype ot,
                       int64_t o_stride, float *lse, void *workspace, size_t workspace_bytes,
                       q4_stream_t stream)
{
    return attention_common(q, q_stride, T, Hq, cache, table, table_stride, width, q_start, kv_len, B,
                            max_fresh, scale, window, o, ot, o_stride, lse, workspace, workspace_bytes,
                            stream, 0, 2000000000ull);
}

q4_status q4_attention_timeout_selftest(const void *q, int64_t q_stride, int64_t T, int64_t Hq,
                                        const q4_kv_cache *cache, const int32_t *table,
                                        int64_t table_stride, int64_t width, const int32_t *q_start,
                                        const int32_t *kv_len, int64_t B, int64_t max_fresh,
                                        float scale, int64_t window, void *o, q4_dtype ot,
                                        int64_t o_stride, float *lse, void *workspace,
                                        size_t workspace_bytes, q4_stream_t stream)
{
    return attention_common(q, q_stride, T, Hq, cache, table, table_stride, width, q_start, kv_len, B,
                            max_fresh, scale, window, o, ot, o_stride, lse, workspace, workspace_bytes,
                            stream, 1, 20000000ull);
}

q4_status q4_check(q4_stream_t stream)
{
    cudaError_t e = cudaStreamSynchronize(reinterpret_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e);
    unsigned int word = 0;
    e = cudaMemcpyFromSymbol(&word, g_q4_error, sizeof(word));
    if (e != cudaSuccess) return cuda_fail(e);
    if (word) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_q4_error, &zero, sizeof(zero));
        if (e != cudaSuccess) return cuda_fail(e);
        return (word & ERR_BOUNDS) ? Q4_ERR_BOUNDS : Q4_ERR_TIMEOUT;
    }
    return Q4_OK;
}

const char *q4_status_str(q4_status status)
{
    switch (status) {
    case Q4_OK: return "ok";
    case Q4_ERR_INVALID_ARG: return "invalid argument";
    case Q4_ERR_UNSUPPORTED: return "unsupported shape or dtype";
    case Q4_ERR_MISALIGNED: return "pointer not 16-byte aligned";
    case Q4_ERR_CUDA: return "CUDA error";
    case Q4_ERR_TIMEOUT: return "a bounded device wait timed out";
    case Q4_ERR_BOUNDS: return "a store outside its buffer was skipped (debug build)";
    }
    return "unknown status";
}

const char *q4_last_cuda_error(void) { return t_last_error; }

q4_status q4_debug_bounds_selftest(uint8_t *buf, q4_stream_t stream)
{
    if (!kDebugBounds) return Q4_ERR_UNSUPPORTED;
    if (!buf) return Q4_ERR_INVALID_ARG;
    const DevInfo *d = dev_info();
    if (!d) return cuda_fail(cudaGetLastError());
    k_bounds_selftest<<<1, 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(buf, d->err);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? Q4_OK : cuda_fail(e);
}

}  // extern "C"
