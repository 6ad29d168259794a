// attention.cu -- attention over the blocked KV cache, few rows per KV head:
// the decode kernel.
//
// Rows.  The n new tokens of a request and the GQ query heads that share a
// KV head form n * GQ rows (token-major) that all read the same keys, in row
// tiles of 16 = the m of mma.sync m16n8k16.  Bound: with n * GQ <= 16 the
// keys and values are read once and each byte feeds 16 multiply-adds, so HBM
// bounds the call as long as loads are kept in flight.
//
// Work.  (request, row tile, KV head) are the items, a unit is 16 keys of
// one item.  All units of the call form one sequence, request-major, cut into
// equal contiguous ranges, one per CTA (one CTA per SM): every SM streams the
// same number of bytes whatever the lengths.  A CTA finds its range from the
// lengths on the device (locate()), so no host plan and no second launch is
// needed.  Within a piece of an item the CTA's 8 warps take its units in
// turn; each warp has its own ring of STAGES units in shared memory filled by
// cp.async (16 bytes per lane; keys past the request's end, blocks outside
// the cache and the padding of head_dim are filled with zeros, so nothing
// stale is ever multiplied), its own running maximum, sum and f32
// accumulator, and no barrier with the others until the piece ends, where the
// warps' results meet in shared memory.  An item cut by a range boundary
// leaves its pieces in the workspace; the last CTA to arrive adds them in CTA
// order, so results do not depend on timing.
#include "serve.cuh"
#include "attention.cuh"

namespace q4 {
namespace {

constexpr int R = 16;        // rows per tile
constexpr int TK = 16;       // keys per unit
constexpr int NW = 8;        // warps
constexpr int STAGES = 3;    // units in flight per warp
constexpr int THREADS = NW * 32;

template <int DP>
struct Sizes {
    static constexpr int ROW = DP * 2;             // bytes of a key
    static constexpr int TILE = TK * ROW;          // bytes of a unit's keys
    static constexpr int RING = NW * STAGES * 2 * TILE;
    static constexpr int MERGE = NW * R * (DP + 2) * 4;  // aliases the ring
    static constexpr int SMEM = RING > MERGE ? RING : MERGE;
    static constexpr int SLOT = R * (DP + 2);      // floats of a partial result
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <bool TRANS>
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr)
{
    if (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(addr)
                     : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(addr)
                     : "memory");
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool F16, int DP>
__global__ void __launch_bounds__(THREADS, 1) k_attn_stream(const AttnArgs a)
{
    using Z = Sizes<DP>;
    constexpr int KS = DP / 16, NO = DP / 8, CH = DP / 8;  // k steps, output n tiles, 16-byte chunks
    constexpr int LPT = TK * CH / 32;                      // 16-byte loads per lane per operand
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ LocateScratch ls;
    __shared__ int last_s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    grid_dep_launch_dependents();
    grid_dep_wait();
    const Range rng = cta_range<R, TK, NW, 1, 0>(a, ls);
    if (rng.u0 >= rng.u1) return;

    const uint32_t ring = smem_u32(smem) + warp * (STAGES * 2 * Z::TILE);
    Item it = rng.first;
    int64_t u = rng.u0;
    int kt = rng.kt;  // first unit of the piece within the item
    while (u < rng.u1) {
        const Span<R, TK> sp(a, it.b, it.rt);
        const int nu = static_cast<int>(min(static_cast<int64_t>(sp.units - kt), rng.u1 - u));

        // ---- this warp's units of the piece: kt + warp, kt + warp + NW, ...
        const int mine = nu > warp ? (nu - warp + NW - 1) / NW : 0;
        const uint16_t *kbase = a.k + it.head * a.head_stride, *vbase = a.v + it.head * a.head_stride;
        const int *trow = a.table + it.b * a.table_stride;
        auto block_of = [&](int i) {  // table entry of this warp's i-th unit
            const int key = (sp.kt0 + kt + warp + i * NW) * TK;
            return i < mine && key < sp.kv ? __ldg(trow + a.by_S.div(key)) : -1;
        };
        int next_block = block_of(0);
        auto issue = [&](int i) {
            if (i < mine) {
                const int blk = next_block;
                const int key = (sp.kt0 + kt + warp + i * NW) * TK;
                const bool in = static_cast<unsigned>(blk) < static_cast<unsigned>(a.blocks);
                const int64_t off = in ? blk * a.block_stride + (key - a.by_S.div(key) * a.S) * a.token_stride : 0;
                const uint32_t dst = ring + (i % STAGES) * 2 * Z::TILE;
#pragma unroll
                for (int l = 0; l < LPT; ++l) {
                    const int e = l * 32 + lane, row = e / CH, c = e % CH;
                    const bool ok = in && key + row < sp.kv && c * 8 < a.D;
                    const int64_t at = ok ? off + row * a.token_stride + c * 8 : 0;
                    const uint32_t d = dst + row * Z::ROW + ((c ^ (row & 7)) << 4);
                    cp_async16(d, kbase + at, ok);
                    cp_async16(d + Z::TILE, vbase + at, ok);
                }
                next_block = block_of(i + 1);
            }
            cp_async_commit();
        };
#pragma unroll
        for (int i = 0; i < STAGES - 1; ++i) issue(i);

        // ---- queries as A fragments: rows lane / 4 and + 8
        uint32_t qf[KS][4];
        const uint16_t *qrow[2];
        int place[2];  // the row's place in its request (its last visible key)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = sp.row0 + lane / 4 + 8 * j;
            const bool in = r < sp.row1;
            const int t = in ? a.by_GQ.div(r) : 0, g = in ? r - t * a.GQ : 0;
            place[j] = in ? sp.base + t : -1;
            qrow[j] = in ? a.q + (sp.t0 + t) * a.q_stride + static_cast<int64_t>(it.head * a.GQ + g) * a.D
                         : nullptr;
        }
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int c = s * 16 + (j >> 1) * 8 + (lane & 3) * 2;
                qf[s][j] = qrow[j & 1] && c < a.D ? *reinterpret_cast<const uint32_t *>(qrow[j & 1] + c) : 0u;
            }

        float o[NO][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < NO; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;

        for (int i = 0; i < mine; ++i) {
            cp_async_wait<STAGES - 2>();
            __syncwarp();  // the other lanes' copies too; and all lanes are done with the slot below
            issue(i + STAGES - 1);
            const uint32_t ks = ring + (i % STAGES) * 2 * Z::TILE, vs = ks + Z::TILE;
            float sc[2][4];
#pragma unroll
            for (int n = 0; n < 2; ++n) sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
                // matrices: keys 0-7 / 8-15 (lane bit 4), dims 16s.. / 16s + 8.. (lane bit 3)
                uint32_t b[4];
                const int row = (lane & 7) + ((lane >> 4) << 3), c = s * 2 + ((lane >> 3) & 1);
                ldsm4<false>(b, ks + row * Z::ROW + ((c ^ (row & 7)) << 4));
                mma16816<F16>(sc[0], qf[s], b[0], b[1]);
                mma16816<F16>(sc[1], qf[s], b[2], b[3]);
            }
            // ---- mask and softmax in units of log 2
            const int key0 = (sp.kt0 + kt + warp + i * NW) * TK + (lane & 3) * 2;
            uint32_t p[4];
            float f[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = key0 + (e >> 1) * 8 + (e & 1);
                    const bool seen = key <= place[j] && (a.window == 0 || key > place[j] - a.window);
                    v[e] = seen ? sc[e >> 1][2 * j + (e & 1)] * a.scale_log2 : -INFINITY;
                }
                float mx = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                const float mn = fmaxf(m[j], mx);
                const float ref = mn == -INFINITY ? 0.0f : mn;  // nothing seen yet
                f[j] = ex2(m[j] - ref);
                m[j] = mn;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = ex2(v[e] - ref);
                l[j] = l[j] * f[j] + ((v[0] + v[1]) + (v[2] + v[3]));
                // A fragment of the second product: keys are its k
                p[j] = pack2<F16>(v[0], v[1]);
                p[2 + j] = pack2<F16>(v[2], v[3]);
            }
            if (__any_sync(0xffffffffu, f[0] != 1.0f || f[1] != 1.0f)) {
#pragma unroll
                for (int n = 0; n < NO; ++n) {
                    o[n][0] *= f[0];
                    o[n][1] *= f[0];
                    o[n][2] *= f[1];
                    o[n][3] *= f[1];
                }
            }
#pragma unroll
            for (int n = 0; n < NO; n += 2) {
                // matrices: keys 0-7 / 8-15 (lane bit 3), dims 8n.. / 8n + 8.. (lane bit 4)
                uint32_t b[4];
                const int row = (lane & 7) + (((lane >> 3) & 1) << 3), c = n + (lane >> 4);
                ldsm4<true>(b, vs + row * Z::ROW + ((c ^ (row & 7)) << 4));
                mma16816<F16>(o[n], p, b[0], b[1]);
                mma16816<F16>(o[n + 1], p, b[2], b[3]);
            }
        }
        cp_async_wait<0>();
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            l[j] += __shfl_xor_sync(0xffffffffu, l[j], 1);
            l[j] += __shfl_xor_sync(0xffffffffu, l[j], 2);
        }

        // ---- the warps' results meet: [warp][row][DP + 2]
        __syncthreads();  // every warp is done with the rings
        float *mg = reinterpret_cast<float *>(smem);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float *w = mg + (warp * R + lane / 4 + 8 * j) * (DP + 2);
#pragma unroll
            for (int n = 0; n < NO; ++n)
                *reinterpret_cast<float2 *>(w + n * 8 + (lane & 3) * 2) = make_float2(o[n][2 * j], o[n][2 * j + 1]);
            if ((lane & 3) == 0) {
                w[DP] = m[j];
                w[DP + 1] = l[j];
            }
        }
        __syncthreads();
        const bool whole = kt == 0 && nu == sp.units;
        const int rows = sp.row1 - sp.row0;
        // a thread takes 4 dims of a row; warps without a unit hold nothing
        const bool use[NW] = {nu > 0, nu > 1, nu > 2, nu > 3, nu > 4, nu > 5, nu > 6, nu > 7};
        for (int e = tid; e < rows * (DP / 4); e += THREADS) {
            const int r = e / (DP / 4), d = e % (DP / 4) * 4;
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < NW; ++w)
                if (use[w]) top = fmaxf(top, mg[(w * R + r) * (DP + 2) + DP]);
            const float ref = top == -INFINITY ? 0.0f : top;
            float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f}, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                if (!use[w]) continue;
                const float *x = mg + (w * R + r) * (DP + 2);
                const float g = ex2(x[DP] - ref);
                sum += g * x[DP + 1];
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[c] += g * x[d + c];
            }
            if (whole) {
                finish_row<F16>(a, it, sp.t0, sp.row0 + r, d, acc, top, sum);
            } else {
                float *ps = a.part + (2 * static_cast<int64_t>(blockIdx.x) + (kt == 0)) * Z::SLOT + r * (DP + 2);
                if (store_ok(ps + DP + 1 - a.part, a.part_len, a.err)) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) ps[d + c] = acc[c];
                    if (d == 0) {
                        ps[DP] = top;
                        ps[DP + 1] = sum;
                    }
                }
            }
        }
        if (!whole) {
            // CTAs holding pieces of this item, in order
            const int64_t i0 = u - kt, i1 = i0 + sp.units;
            const int c0 = owner_of(i0, rng.total, rng.G), c1 = owner_of(i1 - 1, rng.total, rng.G);
            __syncthreads();
            if (tid == 0) {
                last_s = store_ok(c0, a.count_len, a.err) &&
                         atomic_add_acq_rel_gpu(a.count + c0, 1u) == static_cast<unsigned>(c1 - c0);
                if (last_s) a.count[c0] = 0u;
            }
            __syncthreads();
            if (last_s) {
                for (int e = tid; e < rows * (DP / 4); e += THREADS) {
                    const int r = e / (DP / 4), d = e % (DP / 4) * 4;
                    float top = -INFINITY, sum = 0.0f, acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    for (int c = c0; c <= c1; ++c) {
                        const float *x = a.part + (2 * static_cast<int64_t>(c) + (c == c0)) * Z::SLOT + r * (DP + 2);
                        const float mx = __ldcg(x + DP), ls2 = __ldcg(x + DP + 1);
                        const float mn = fmaxf(top, mx), ref = mn == -INFINITY ? 0.0f : mn;
                        const float g0 = ex2(top - ref), g1 = ex2(mx - ref);
                        top = mn;
                        sum = sum * g0 + ls2 * g1;
#pragma unroll
                        for (int k = 0; k < 4; ++k) acc[k] = acc[k] * g0 + __ldcg(x + d + k) * g1;
                    }
                    finish_row<F16>(a, it, sp.t0, sp.row0 + r, d, acc, top, sum);
                }
            }
        }
        __syncthreads();  // the merge buffer becomes the rings again
        u += nu;
        kt = 0;
        it.next(a, R);
    }
}

template <bool F16, int DP>
cudaError_t launch(const AttnPlan &p, const AttnArgs &a, cudaStream_t s)
{
    static std::atomic<bool> done[64];
    auto kern = k_attn_stream<F16, DP>;
    const cudaError_t e = allow_smem(kern, Sizes<DP>::SMEM, done);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3(p.grid), THREADS, Sizes<DP>::SMEM, s, a);
}

}  // namespace

AttnPlan attention_plan(int64_t max_fresh, int64_t GQ, int64_t D, int sm_count)
{
    AttnPlan p{};
    p.grid = std::min<int>(sm_count, ATTN_COUNTER_BYTES / sizeof(unsigned int) / 2);
    p.tc = max_fresh > R / GQ;
    const size_t slot = R * ((D > 64 ? 128 : 64) + 2) * sizeof(float);
    const size_t part = p.tc ? attention_tc_part_bytes(D, p.grid) : 2 * static_cast<size_t>(p.grid) * slot;
    p.workspace = ATTN_COUNTER_BYTES + part;
    return p;
}

cudaError_t attention_launch(const AttnPlan &p, const AttnArgs &a, bool f16, cudaStream_t s)
{
    if (p.tc) return attention_tc_launch(p.grid, a, f16, s);
    if (a.D > 64) return f16 ? launch<true, 128>(p, a, s) : launch<false, 128>(p, a, s);
    return f16 ? launch<true, 64>(p, a, s) : launch<false, 64>(p, a, s);
}

}  // namespace q4
