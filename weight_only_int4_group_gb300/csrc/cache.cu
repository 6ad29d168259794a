// cache.cu -- the step's plan over the blocked KV cache, and the rotary
// positions with the cache append.
#include "serve.cuh"

namespace q4 {
namespace {

// ------------------------------------------------------------------- plan
// Everything follows from two running sums over the requests: of the new
// tokens (first row of each request) and of the blocks they need (which
// entries of the free stack each request takes).  The data are a few bytes
// per request and 12 bytes per token, so the call is a launch and three
// dependent memory round trips (measured, in a graph: 3.5 us for 8 requests,
// 5.5 us for 1024 with 16000 tokens); every CTA repeats the sums over all requests
// (8 bytes each, from L2 after the first CTA) instead of a second launch,
// then finds the request of each of its tokens by bisection in shared memory.
constexpr int PLAN_THREADS = 512;

struct Need {
    int64_t n;   // new tokens (negative lengths: none)
    int64_t nb;  // new blocks
    bool fits;   // lengths valid and within the table's width
};
__device__ __forceinline__ Need need_of(const PlanArgs &a, int b)
{
    const int64_t c = a.cached[b], f = a.fresh[b];
    Need r;
    r.n = f < 0 || c < 0 ? 0 : f;
    r.fits = f >= 0 && c >= 0 && c + f <= static_cast<int64_t>(a.width) * a.S;
    // c + f < 2^32: unsigned 32-bit divisions
    const uint32_t S = a.S;
    r.nb = r.fits ? static_cast<int64_t>((static_cast<uint32_t>(c + f) + S - 1) / S) -
                        static_cast<int64_t>((static_cast<uint32_t>(c) + S - 1) / S)
                  : 0;
    return r;
}

__global__ void __launch_bounds__(PLAN_THREADS) k_cache_plan(const PlanArgs a)
{
    extern __shared__ int plan_smem[];
    int *start = plan_smem;           // [B + 1]
    int *first = plan_smem + a.B + 1; // [B] first entry of the free stack taken; -1: not served
    __shared__ int64_t wsum[2][PLAN_THREADS / 32];
    __shared__ unsigned int tally[3];  // blocks taken, tokens served, requests not served
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool lead = blockIdx.x == 0;

    grid_dep_wait();
    grid_dep_launch_dependents();
    if (tid < 3) tally[tid] = 0;
    const int64_t avail = max(0, min(*a.free_count, a.free_capacity));

    // contiguous requests per thread, then an exclusive scan over the threads
    const int per = (a.B + PLAN_THREADS - 1) / PLAN_THREADS;
    const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    int64_t sn = 0, sb = 0;
    for (int b = b0; b < b1; ++b) {
        const Need r = need_of(a, b);
        sn += r.n;
        sb += r.nb;
    }
    int64_t in = sn, ib = sb;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t pn = __shfl_up_sync(0xffffffffu, in, d), pb = __shfl_up_sync(0xffffffffu, ib, d);
        if (lane >= d) {
            in += pn;
            ib += pb;
        }
    }
    if (lane == 31) {
        wsum[0][warp] = in;
        wsum[1][warp] = ib;
    }
    __syncthreads();
    int64_t rn = in - sn, rb = ib - sb;
    for (int w = 0; w < warp; ++w) {
        rn += wsum[0][w];
        rb += wsum[1][w];
    }
    unsigned int mine[3] = {0, 0, 0};  // at most avail, T and B in all
    for (int b = b0; b < b1; ++b) {
        const Need r = need_of(a, b);
        const bool served = r.fits && rn + r.n <= a.T && (r.nb == 0 || rb + r.nb <= avail);
        start[b] = static_cast<int>(min(rn, static_cast<int64_t>(a.T)));
        first[b] = !served ? -1 : r.nb ? static_cast<int>(rb) : 0;
        if (lead) {
            if (store_ok(b, static_cast<int64_t>(a.B) + 1, a.err)) a.q_start[b] = start[b];
            if (store_ok(b, a.B, a.err)) a.kv_len[b] = served ? a.cached[b] + a.fresh[b] : 0;
            if (served) {
                mine[0] += static_cast<unsigned int>(r.nb);
                mine[1] += static_cast<unsigned int>(r.n);
            } else {
                ++mine[2];
            }
        }
        rn += r.n;
        // rb past avail stays past it: later requests in need are not served
        rb += r.nb;
    }
    if (b1 == a.B && b0 < b1) {
        start[a.B] = static_cast<int>(min(rn, static_cast<int64_t>(a.T)));
        if (lead && store_ok(a.B, static_cast<int64_t>(a.B) + 1, a.err)) a.q_start[a.B] = start[a.B];
    }
    if (lead) {
#pragma unroll
        for (int i = 0; i < 3; ++i) {
            const unsigned int s = __reduce_add_sync(0xffffffffu, mine[i]);
            if (lane == 0 && s) atomicAdd(&tally[i], s);
        }
    }
    __syncthreads();
    if (lead && tid < 4 && store_ok(tid, 4, a.err))
        a.counts[tid] = tid == 0   ? start[a.B]
                        : tid == 1 ? static_cast<int>(tally[1])
                        : tid == 2 ? static_cast<int>(avail) - static_cast<int>(tally[0])
                                   : static_cast<int>(tally[2]);

    // the requests' new table entries, requests dealt over the grid's warps
    const int nwarp = gridDim.x * (PLAN_THREADS / 32);
    for (int b = blockIdx.x * (PLAN_THREADS / 32) + warp; b < a.B; b += nwarp) {
        if (first[b] < 0) continue;
        const uint32_t S = a.S, c = a.cached[b], l = c + static_cast<uint32_t>(a.fresh[b]);
        const int have = static_cast<int>((c + S - 1) / S), need = static_cast<int>((l + S - 1) / S);
        for (int j = have + lane; j < need; j += 32) {
            const int64_t at = b * a.table_stride + j;
            if (store_ok(at, static_cast<int64_t>(a.B) * a.table_stride, a.err))
                a.table[at] = a.free_blocks[avail - 1 - (first[b] + (j - have))];
        }
    }

    // the tokens
    for (int64_t t = static_cast<int64_t>(blockIdx.x) * PLAN_THREADS + tid; t < a.T;
         t += static_cast<int64_t>(gridDim.x) * PLAN_THREADS) {
        int pos = 0;
        int64_t slot = -1;
        if (t < start[a.B]) {
            int lo = 0, hi = a.B;  // start[lo] <= t < start[hi]
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (start[mid] <= t)
                    lo = mid;
                else
                    hi = mid;
            }
            if (first[lo] >= 0) {
                const uint32_t c = a.cached[lo], S = a.S, p = c + static_cast<uint32_t>(t - start[lo]);
                pos = static_cast<int>(p);
                const int j = static_cast<int>(p / S), have = static_cast<int>((c + S - 1) / S);
                const int blk = j < have ? a.table[lo * a.table_stride + j]
                                         : a.free_blocks[avail - 1 - (first[lo] + (j - have))];
                if (blk >= 0) slot = static_cast<int64_t>(blk) * S + p % S;
            }
        }
        if (store_ok(t, a.T, a.err)) {
            a.position[t] = pos;
            a.slot[t] = slot;
        }
    }
}

}  // namespace

cudaError_t cache_plan_launch(const PlanArgs &a, cudaStream_t s)
{
    static std::atomic<bool> done[64];
    constexpr size_t most = (2 * Q4_PLAN_MAX_REQUESTS + 1) * sizeof(int);
    const cudaError_t e = allow_smem(k_cache_plan, most, done);
    if (e != cudaSuccess) return e;
    const size_t smem = (2 * static_cast<size_t>(a.B) + 1) * sizeof(int);
    const int grid = std::min(128, ctas_for(a.T, PLAN_THREADS));
    return launch_dependent(k_cache_plan, dim3(grid), PLAN_THREADS, smem, s, a);
}

// ------------------------------------------------------- rotary and append
// Memory-bound: every qkv element is read once and written once.  A CTA takes
// TOK tokens; its threads first compute the cosines and sines of the tokens'
// angles (one each, shared by all heads of the token through shared memory),
// then move the heads: a thread handles VEC rotated pairs (two VEC-element
// loads a half head apart, or one load of interleaved pairs) or a VEC-element
// copy (the unrotated part of a head, the values).  VEC is the widest vector
// that the pair layout allows, 8 elements (16 bytes) for the usual sizes.
// Measured: 8192 rows of 80 heads of 128 in 58.3 us, 5.8 TB/s read and
// written, 0.85 of the measured copy bandwidth (the cache rows are 256-byte
// pieces at random places).  Several units per thread in flight were slower
// (74 us and more): the registers cost more warps than the loads gain.
namespace {

constexpr int ROPE_THREADS = 256;

template <bool F16>
__device__ __forceinline__ float to_f32(uint16_t b)
{
    if (!F16) return __uint_as_float(static_cast<uint32_t>(b) << 16);
    __half_raw h;
    h.x = b;
    return __half2float(__half(h));
}
template <bool F16>
__device__ __forceinline__ uint16_t from_f32(float f)
{
    if (!F16) return __bfloat16_as_ushort(__float2bfloat16_rn(f));
    return __half_as_ushort(__float2half_rn(f));
}

template <int VEC>
struct alignas(VEC * 2) Vec {
    uint16_t e[VEC];
};

template <bool F16, bool INTER, int VEC>
__global__ void __launch_bounds__(ROPE_THREADS) k_rope_append(const RopeArgs a, int tok)
{
    using V = Vec<VEC>;
    extern __shared__ float2 rope_cs[];  // [tok][rot / 2] (factor * cos, factor * sin)
    __shared__ int64_t dst_off[8];       // element offset of the token's cache row, or -1
    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * tok, nt = min(tok, a.T - t0);
    const int half = a.rot / 2;

    grid_dep_wait();
    grid_dep_launch_dependents();
    for (int i = tid; i < nt * half; i += ROPE_THREADS) {
        const int t = i / half;
        // whole turns drop out in 64 bits; what is left fits f32
        double turns = a.position[t0 + t] * (a.freq[i - t * half] * 0.15915494309189535);
        turns -= rint(turns);
        float sn, cs;
        sincospif(2.0f * static_cast<float>(turns), &sn, &cs);
        rope_cs[i] = make_float2(cs * a.factor, sn * a.factor);
    }
    if (tid < nt) {
        const int64_t slot = a.slot[t0 + tid];
        const bool in = slot >= 0 && slot < static_cast<int64_t>(a.blocks) * a.S;
        const int64_t blk = !in ? 0 : slot >> 32 ? slot / a.S : static_cast<uint32_t>(slot) / static_cast<uint32_t>(a.S);
        dst_off[tid] = in ? blk * a.block_stride + (slot - blk * a.S) * a.token_stride : -1;
    }
    __syncthreads();

    // units per rotated head: pairs, then copies of the rest
    const int pair_units = INTER ? a.rot / VEC : half / VEC;
    const int units = pair_units + (a.D - a.rot) / VEC;
    const int heads = a.Hq + a.Hkv;
    const int64_t cache_len = static_cast<int64_t>(a.blocks - 1) * a.block_stride +
                              static_cast<int64_t>(a.Hkv - 1) * a.head_stride +
                              static_cast<int64_t>(a.S - 1) * a.token_stride + a.D;
    const int64_t q_len = static_cast<int64_t>(a.T - 1) * a.q_stride + static_cast<int64_t>(a.Hq) * a.D;
    const int per = ROPE_THREADS / units;  // heads in flight
    const int u = tid % units, h0 = tid / units;
    if (h0 < per) {
        const bool pair = u < pair_units;
        for (int w = blockIdx.y * per + h0; w < nt * heads; w += gridDim.y * per) {
            const int t = w / heads, h = w - t * heads;
            const uint16_t *x = a.qkv + (t0 + t) * a.qkv_stride + static_cast<int64_t>(h) * a.D;
            uint16_t *y;
            int64_t at;
            if (h < a.Hq) {
                at = (t0 + t) * a.q_stride + static_cast<int64_t>(h) * a.D;
                y = a.q_out + at;
                if (!store_ok(at + a.D - 1, q_len, a.err)) continue;
            } else {
                if (dst_off[t] < 0) continue;
                at = dst_off[t] + (h - a.Hq) * a.head_stride;
                y = a.k + at;
                if (!store_ok(at + a.D - 1, cache_len, a.err)) continue;
            }
            if (pair && INTER) {
                V v = *reinterpret_cast<const V *>(x + u * VEC);
                const float2 *cs = rope_cs + t * half + u * (VEC / 2);
#pragma unroll
                for (int i = 0; i < VEC / 2; ++i) {
                    const float p = to_f32<F16>(v.e[2 * i]), q = to_f32<F16>(v.e[2 * i + 1]);
                    v.e[2 * i] = from_f32<F16>(p * cs[i].x - q * cs[i].y);
                    v.e[2 * i + 1] = from_f32<F16>(p * cs[i].y + q * cs[i].x);
                }
                *reinterpret_cast<V *>(y + u * VEC) = v;
            } else if (pair) {
                V lo = *reinterpret_cast<const V *>(x + u * VEC);
                V hi = *reinterpret_cast<const V *>(x + half + u * VEC);
                const float2 *cs = rope_cs + t * half + u * VEC;
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float p = to_f32<F16>(lo.e[i]), q = to_f32<F16>(hi.e[i]);
                    lo.e[i] = from_f32<F16>(p * cs[i].x - q * cs[i].y);
                    hi.e[i] = from_f32<F16>(p * cs[i].y + q * cs[i].x);
                }
                *reinterpret_cast<V *>(y + u * VEC) = lo;
                *reinterpret_cast<V *>(y + half + u * VEC) = hi;
            } else {
                const int e = a.rot + (u - pair_units) * VEC;
                *reinterpret_cast<V *>(y + e) = *reinterpret_cast<const V *>(x + e);
            }
        }
    }
    // values: 16-byte copies
    const int vu = a.D / 8, vper = ROPE_THREADS / vu, vc = tid % vu, vh = tid / vu;
    if (vh < vper) {
        for (int w = blockIdx.y * vper + vh; w < nt * a.Hkv; w += gridDim.y * vper) {
            const int t = w / a.Hkv, h = w - t * a.Hkv;
            if (dst_off[t] < 0) continue;
            const int64_t at = dst_off[t] + h * a.head_stride;
            if (!store_ok(at + a.D - 1, cache_len, a.err)) continue;
            *reinterpret_cast<uint4 *>(a.v + at + vc * 8) = *reinterpret_cast<const uint4 *>(
                a.qkv + (t0 + t) * a.qkv_stride + static_cast<int64_t>(heads + h) * a.D + vc * 8);
        }
    }
}

template <bool F16, bool INTER>
cudaError_t rope_launch(const RopeArgs &a, cudaStream_t s)
{
    // Tokens per CTA and CTAs per token (us, 64 + 2 * 8 heads of 128): few
    // tokens are latency, shared out finer (T = 4: 2.7 by four CTAs each, 3.7
    // by one; T = 152: 3.7 by two, 4.0 by four); many are bandwidth, where
    // more tokens per CTA spare beginnings (T = 8192: 57.7 by four tokens in
    // two halves, 64.1 by one; T = 2048: 18.2 and 16.9).  The rule goes by
    // tokens alone: with 32 + 2 * 32 heads T = 2999 takes 28.9 and 3000 30.5,
    // with 8 + 2 8.9 and 7.4.
    const bool many = a.T >= 3000;
    const int tok = many ? 4 : 1;
    const int split = many ? 2 : a.T <= 64 ? 4 : a.T <= 152 ? 2 : 1;
    const dim3 grid(ctas_for(a.T, tok), split);
    const size_t smem = static_cast<size_t>(tok) * (a.rot / 2) * sizeof(float2);
    // the widest vector that divides the pair layout and both parts of the head
    const int m = (INTER ? a.rot : a.rot / 2) | (a.D - a.rot);
    if (m % 8 == 0) return launch_dependent(k_rope_append<F16, INTER, 8>, grid, ROPE_THREADS, smem, s, a, tok);
    if (m % 4 == 0) return launch_dependent(k_rope_append<F16, INTER, 4>, grid, ROPE_THREADS, smem, s, a, tok);
    if (m % 2 == 0) return launch_dependent(k_rope_append<F16, INTER, 2>, grid, ROPE_THREADS, smem, s, a, tok);
    return launch_dependent(k_rope_append<F16, false, 1>, grid, ROPE_THREADS, smem, s, a, tok);
}

}  // namespace

cudaError_t rope_append_launch(const RopeArgs &a, bool f16, bool interleaved, cudaStream_t s)
{
    if (f16) return interleaved ? rope_launch<true, true>(a, s) : rope_launch<true, false>(a, s);
    return interleaved ? rope_launch<false, true>(a, s) : rope_launch<false, false>(a, s);
}

}  // namespace q4
