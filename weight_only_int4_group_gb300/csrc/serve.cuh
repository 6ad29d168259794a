// serve.cuh -- internal declarations of the serving operators (cache plan,
// rotary append, attention over the blocked cache).
#pragma once

#include "common.cuh"

namespace q4 {

// Division of 0 <= n < 2^31 by a divisor fixed for the launch: with
// 2^(s - 32) < d <= 2^(s - 31), n / d = n * (floor(2^s / d) + 1) >> s exactly
// (Granlund and Montgomery 1994, for 31-bit n).
struct FastDiv {
    uint32_t mul, shift;
    int d;
    void set(int divisor)
    {
        d = divisor;
        int l = 0;
        while ((1ll << l) < divisor) ++l;
        shift = 31 + l;
        mul = static_cast<uint32_t>((1ull << shift) / static_cast<unsigned>(divisor) + 1);
    }
    __host__ __device__ __forceinline__ int div(int n) const
    {
        return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * mul) >> shift);
    }
};

// CTAs that take n (up to 2^31 - 1) things, `per` each.
inline int ctas_for(int64_t n, int per) { return static_cast<int>((n + per - 1) / per); }

// One q4_attention call as its kernels see it.
struct AttnArgs {
    const uint16_t *q, *k, *v;  // 16-bit elements, bf16 or f16
    void *o;
    q4_dtype ot;
    float *lse;  // or null
    int64_t q_stride, o_stride;
    int64_t block_stride, head_stride, token_stride;
    const int *table;
    int64_t table_stride;
    const int *q_start, *kv_len;
    int T, B, Hq, Hkv, GQ;  // GQ: query heads per KV head
    FastDiv by_GQ, by_S;
    int D, S, blocks, width;
    float scale_log2;  // scale * log2(e): scores in units of log 2
    int window;        // 0: none
    unsigned int *count;  // arrival counters
    float *part;          // partial results: four per CTA, or two per warp
    int64_t count_len, part_len;  // their extents, for the store checks
    uint64_t wait_ns;
    int debug_no_copy;
    unsigned int *err;
};

constexpr size_t ATTN_COUNTER_BYTES = 131072;

struct AttnPlan {
    bool tc;         // tensor-core kernel (many rows per KV head)
    int grid;
    size_t workspace;
};
AttnPlan attention_plan(int64_t max_fresh, int64_t GQ, int64_t D, int sm_count);
size_t attention_tc_part_bytes(int64_t D, int grid);
cudaError_t attention_tc_launch(int grid, const AttnArgs &a, bool f16, cudaStream_t s);
cudaError_t attention_launch(const AttnPlan &p, const AttnArgs &a, bool f16, cudaStream_t s);

struct PlanArgs {
    const int *cached, *fresh;
    int B, S;
    int *table;
    int64_t table_stride;
    int width;
    const int *free_blocks, *free_count;
    int free_capacity, T;
    int *q_start, *kv_len, *position;
    int64_t *slot;
    int *counts;
    unsigned int *err;
};
cudaError_t cache_plan_launch(const PlanArgs &a, cudaStream_t s);

struct RopeArgs {
    const uint16_t *qkv;
    int64_t qkv_stride;
    int T, Hq, Hkv, D, rot;
    const double *freq;
    float factor;
    const int *position;
    const int64_t *slot;
    uint16_t *q_out;
    int64_t q_stride;
    uint16_t *k, *v;
    int64_t block_stride, head_stride, token_stride;
    int blocks, S;
    unsigned int *err;
};
cudaError_t rope_append_launch(const RopeArgs &a, bool f16, bool interleaved, cudaStream_t s);

// Launch with programmatic stream serialization: the kernel may become
// resident while the previous one drains, and waits (grid_dep_wait) before it
// touches memory.  It lets its own dependents go only behind that wait, so
// that whatever they read early (a product its weights) was complete before
// this kernel began to work.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kern)(P...), dim3 grid, int threads, size_t smem,
                             cudaStream_t s, A... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

// Raises a kernel's dynamic shared memory limit once per device.
template <typename K>
cudaError_t allow_smem(K kern, size_t bytes, std::atomic<bool> (&done)[64])
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(bytes));
    if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
    return e;
}

}  // namespace q4
