// attention8.cu -- attention over the 8-bit blocked cache.
#include "attention.cuh"
#include "cache8.cuh"

namespace q4 {
namespace {

// A warp per (token row, query head): 32 keys at a time, a key per lane for the
// scores, 4 dims per lane for the weighted values; one pass with the running
// maximum and sum.
template <int CODE, bool F16>
__global__ void __launch_bounds__(256) k_attn8(const AttnArgs a, const Codes c)
{
    using X = Exponents<CODE, F16>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ float qs[8][128];
    grid_dep_wait();
    grid_dep_launch_dependents();
    const int64_t w = static_cast<int64_t>(blockIdx.x) * 8 + warp;
    if (w >= static_cast<int64_t>(a.T) * a.Hq) return;
    const int t = static_cast<int>(w / a.Hq), h = static_cast<int>(w - static_cast<int64_t>(t) * a.Hq), kvh = h / a.GQ;
    const int b = request_of(a.q_start, a.B, t);
    int t0, n, kv;
    request(a, b, t0, n, kv);
    if (t < t0 || t >= t0 + n) return;
    const int place = kv - n + (t - t0);
    for (int d = lane; d < 128; d += 32)
        qs[warp][d] = d < a.D ? bits_to_f32<F16>(a.q[t * a.q_stride + static_cast<int64_t>(h) * a.D + d]) : 0.0f;
    __syncwarp();
    float m = -INFINITY, l = 0.0f, o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j0 = window_start(a, place) & ~15; j0 <= place; j0 += 32) {
        const int j = j0 + lane;
        const bool seen = j <= place && (a.window == 0 || j > place - a.window);
        int64_t at = -1;
        float fk = 0.0f, fv = 0.0f, s = -INFINITY;
        if (seen) {
            s = 0.0f;
            const int col = a.by_S.div(j), blk = a.table[b * a.table_stride + col];
            if (static_cast<unsigned>(blk) < static_cast<unsigned>(c.blocks)) {
                at = blk * c.block_stride + (j - col * a.S) * c.token_stride + kvh * c.head_stride;
                fk = pow2(X::of(c.k_exp[static_cast<int64_t>(blk) * c.heads + kvh]));
                fv = pow2(X::of(c.v_exp[static_cast<int64_t>(blk) * c.heads + kvh]));
                for (int d = 0; d < a.D; d += 4) {
                    float x[4];
                    codes_to_f32<CODE>(*reinterpret_cast<const uint32_t *>(c.k + at + d), x);
#pragma unroll
                    for (int e = 0; e < 4; ++e) s = fmaf(x[e], qs[warp][d + e], s);
                }
            }
            s *= fk * a.scale_log2;
        }
        float mx = s;
        for (int d = 16; d; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
        const float mn = fmaxf(m, mx);
        const float ref = mn == -INFINITY ? 0.0f : mn, f = ex2(m - ref), p = ex2(s - ref);
        m = mn;
        l = l * f + p;
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] *= f;
        for (int i = 0; i < 32; ++i) {
            const int64_t from = __shfl_sync(0xffffffffu, at, i);
            const float pv = __shfl_sync(0xffffffffu, p * fv, i);
            if (from >= 0 && lane * 4 < a.D) {
                float x[4];
                codes_to_f32<CODE>(*reinterpret_cast<const uint32_t *>(c.v + from + lane * 4), x);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = fmaf(pv, x[e], o[e]);
            }
        }
    }
    for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    const float inv = inverse(l);
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] *= inv;
    if (lane * 4 < a.D) store_dims<F16, 4>(a, t, h, lane * 4, o);
    if (lane == 0) store_lse(a, t, h, m, l);
}

template <int CODE, bool F16>
cudaError_t launch(const AttnArgs &a, const Codes &c, cudaStream_t s)
{
    const dim3 grid(ctas_for(static_cast<int64_t>(a.T) * a.Hq, 8));
    return launch_dependent(k_attn8<CODE, F16>, grid, 256, 0, s, a, c);
}

}  // namespace

AttnPlan attention8_plan(int64_t, int64_t, int64_t, int sm_count)
{
    AttnPlan p{};
    p.grid = sm_count;
    p.workspace = ATTN_COUNTER_BYTES;
    return p;
}

cudaError_t attention8_launch(const AttnPlan &, const AttnArgs &a, const Codes &c, q4_code code, bool f16, cudaStream_t s)
{
    if (code == Q4_I8) return f16 ? launch<I8, true>(a, c, s) : launch<I8, false>(a, c, s);
    return f16 ? launch<E4M3, true>(a, c, s) : launch<E4M3, false>(a, c, s);
}

}  // namespace q4
