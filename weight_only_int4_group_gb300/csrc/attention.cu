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
// equal contiguous ranges, one per warp (8 warps per SM): every warp streams
// the same number of bytes whatever the lengths, finds its range from the
// lengths on the device (no host plan, no second launch), and shares nothing
// with its neighbours, so that one that finishes an item does not hold up the
// others' loads.  Each warp has a ring of STAGES units in shared memory filled
// by cp.async (16 bytes per lane; keys past the request's end or before every
// row's window, blocks outside the cache and the padding of head_dim are
// filled with zeros, so nothing stale is ever multiplied); the loads run ahead
// through the ends of items.
// An item cut by range boundaries leaves its pieces in the workspace, in the
// lanes' own order; the last warp to arrive adds them (eight at a time, in a
// tree, when there are many), always in sequence order, so results do not
// depend on timing.
//
// Measured (64 query / 8 KV heads of 128, bf16): 48 requests of 1001..24576
// keys 384 us, 6.5 TB/s (0.96 of the measured copy bandwidth); 32 of
// 101..8192 keys 96 us (0.83); one of 65536 55 us (0.72); one of 777 keys 13 us,
// which is latency.
#include "serve.cuh"
#include "attention.cuh"

namespace q4 {
namespace {

constexpr int R = 16;        // rows per tile
constexpr int TK = 16;       // keys per unit
constexpr int NW = 8;        // warps
constexpr int STAGES = 3;    // units in flight per warp
constexpr int THREADS = NW * 32;
// Places that an item takes beside its units (its beginning and end), and the
// least that a warp gets (one request of 777 keys: 14.1 us by 4 and 14.7 by 8;
// 16 with drafted tokens: 16.3 and 18.0).
constexpr int PAD = 4, MIN_UNITS = 4;
// Weights are taken under a reference this many powers of two below the row's
// maximum: they are rounded to the cache's type for the second product, and
// binary16 ends at 2^16 and 2^-25 (under the maximum itself, 65536 keys of
// weight 2^-25 beside a large one would vanish from the output while their
// row's sum counts them).  bf16 has the exponents of f32.
template <bool F16>
constexpr float LIFT = F16 ? 15.0f : 0.0f;
// Parts that are added at a time where an item is split; 4 levels hold 4096
// workers, of 2048 at most.
constexpr int MERGE = 8, LEVELS = 4, MOST_CTAS = 256;
static_assert(MERGE * MERGE * MERGE * MERGE >= NW * MOST_CTAS, "levels");
static_assert(LEVELS * 2 * NW * MOST_CTAS * sizeof(unsigned int) <= ATTN_COUNTER_BYTES, "counters");

template <int DP>
struct Sizes {
    static constexpr int ROW = DP * 2;             // bytes of a key
    static constexpr int TILE = TK * ROW;          // bytes of a unit's keys
    static constexpr int SMEM = NW * STAGES * 2 * TILE;
    static constexpr int SLOT = R * (DP + 8);      // floats of a partial result: sums, (reference, sum) per lane and row
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

// Adds n parts, the first at x and the others 2 * stride slots on each (a first
// piece of an item lies in the odd slot of its worker), to the row halves
// 0..J - 1 of the empty sums o, m, l; AHEAD parts' loads are in flight.
template <int J, int AHEAD, int NO>
__device__ __forceinline__ void add_parts(const float2 *x, int stride, int n, bool odd, int slot, float (&o)[NO][4],
                                          float (&m)[2], float (&l)[2])
{
    const float2 *even = x - (odd ? slot / 2 : 0);
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += AHEAD) {
        float2 y[AHEAD][J][NO], ml[AHEAD][J];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const bool in = i0 + i < n;
            const float2 *p = i0 + i == 0 ? x : even + static_cast<int64_t>(i0 + i) * stride * slot;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                ml[i][j] = in ? __ldcg(p + (NO * 2 + j) * 32) : make_float2(-INFINITY, 0.0f);
#pragma unroll
                for (int k = 0; k < NO; ++k) y[i][j][k] = in ? __ldcg(p + (k * 2 + j) * 32) : make_float2(0.0f, 0.0f);
            }
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const float mn = fmaxf(m[j], ml[i][j].x), ref = mn == -INFINITY ? 0.0f : mn;
                const float g0 = ex2(m[j] - ref), g1 = ex2(ml[i][j].x - ref);
                m[j] = mn;
                l[j] = l[j] * g0 + ml[i][j].y * g1;
#pragma unroll
                for (int k = 0; k < NO; ++k) {
                    o[k][2 * j] = o[k][2 * j] * g0 + y[i][j][k].x * g1;
                    o[k][2 * j + 1] = o[k][2 * j + 1] * g0 + y[i][j][k].y * g1;
                }
            }
    }
}

template <bool F16, int DP>
__global__ void __launch_bounds__(THREADS, 1) k_attn_stream(const AttnArgs a)
{
    using Z = Sizes<DP>;
    constexpr int KS = DP / 16, NO = DP / 8, CH = DP / 8;  // k steps, output n tiles, 16-byte chunks
    constexpr int LPT = TK * CH / 32;                      // 16-byte loads per lane per operand
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ LocateScratch ls;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    grid_dep_wait();
    grid_dep_launch_dependents();
    sum_slabs<R, TK, NW, PAD>(a, ls);
    // neighbours in the sequence on different SMs: few units use many SMs
    const int me = warp * gridDim.x + blockIdx.x;
    const Range rng = find_share<R, TK, NW, MIN_UNITS, PAD>(a, ls, me, NW * gridDim.x);
    if (rng.u0 >= rng.u1) return;

    using Pieces = Walk<R, TK, PAD>;
    Pieces k(a, rng), ld = k;  // being summed; being loaded
    const uint32_t ring = smem_u32(smem) + warp * (STAGES * 2 * Z::TILE);
    int ld_i = 0, ld_slot = 0;  // unit of ld, ring slot
    auto block_of = [&]() {  // table entry of the unit to load
        const int key = (ld.kt0 + ld.kt + ld_i) * TK;
        return ld.more(rng) && key < ld.kv ? a.table[ld.it.b * a.table_stride + a.by_S.div(key)] : -1;
    };
    int blk = block_of();
    auto issue = [&]() {
        if (ld.more(rng)) {
            const int key = (ld.kt0 + ld.kt + ld_i) * TK;
            const bool in = static_cast<unsigned>(blk) < static_cast<unsigned>(a.blocks);
            const uint32_t dst = ring + ld_slot * 2 * Z::TILE;
            // lane: 16-byte piece c of rows hi, hi + RPI, ..
            constexpr int RPI = 32 / CH;
            const int c = lane % CH, hi = lane / CH;
            int64_t at = in ? blk * a.block_stride + (key - a.by_S.div(key) * a.S + hi) * a.token_stride +
                                  ld.it.head * a.head_stride + c * 8
                            : 0;
            const int rows = in && c * 8 < a.D ? ld.kv - key : 0;  // keys that exist
            // and those that the window leaves to some row
            const int row0 = a.window > 0 && ld.kt + ld_i == 0 ? ld.first_key(a) - key : 0;
#pragma unroll
            for (int l = 0; l < LPT; ++l) {
                const int row = l * RPI + hi;
                const bool ok = row >= row0 && row < rows;
                const uint32_t d = dst + row * Z::ROW + ((c ^ (row & 7)) << 4);
                cp_async16(d, a.k + (ok ? at : 0), ok);
                cp_async16(d + Z::TILE, a.v + (ok ? at : 0), ok);
                at += RPI * a.token_stride;
            }
            ld_slot = ld_slot + 1 == STAGES ? 0 : ld_slot + 1;
            if (++ld_i == ld.nu) {
                ld.next(a, rng);
                ld_i = 0;
            }
            blk = block_of();
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) issue();

    int slot = 0;
    for (; k.more(rng); k.next(a, rng)) {
        // ---- queries as A fragments: rows lane / 4 and + 8
        uint32_t qf[KS][4];
        const uint16_t *qrow[2];
        int place[2];  // the row's place in its request (its last visible key)
        int64_t trow[2];
        int hrow[2];
        const bool two = k.row1 - k.row0 > 8;  // rows 8..15 are there
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = k.row0 + lane / 4 + 8 * j;
            const bool in = r < k.row1;
            const int t = in ? a.by_GQ.div(r) : 0, g = in ? r - t * a.GQ : 0;
            place[j] = in ? k.base + t : -1;
            trow[j] = in ? k.t0 + t : -1;
            hrow[j] = k.it.head * a.GQ + g;
            qrow[j] = in ? a.q + trow[j] * a.q_stride + static_cast<int64_t>(hrow[j]) * a.D : nullptr;
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

        for (int i = 0; i < k.nu; ++i) {
            cp_async_wait<STAGES - 2>();
            __syncwarp();  // the other lanes' copies too; and all lanes are done with the slot below
            issue();
            const uint32_t ks = ring + slot * 2 * Z::TILE, vs = ks + Z::TILE;
            slot = slot + 1 == STAGES ? 0 : slot + 1;
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
            const int key0 = (k.kt0 + k.kt + i) * TK + (lane & 3) * 2;
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
                for (int e = 0; e < 4; ++e) v[e] = ex2((v[e] - ref) + LIFT<F16>);  // no rounding of a large ref
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
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            l[j] += __shfl_xor_sync(0xffffffffu, l[j], 1);
            l[j] += __shfl_xor_sync(0xffffffffu, l[j], 2);
        }

        bool store = k.whole();
        if (!store) {
            // the item's pieces are the leaves of a tree of MERGE-fold nodes
            // over the workers that hold them; whoever completes a node adds
            // its parts in order, leaves the sum in the first part's place and
            // goes on to the next level.  A node's counter goes by its first
            // worker, which may also hold the end of another item.
            int w0, w1;
            k.holders(rng, w0, w1);
            // [dim pair][row half][lane], then (reference, sum) [row half][lane]
            auto part = [&](int w) {
                return reinterpret_cast<float2 *>(a.part + (2 * static_cast<int64_t>(w) + (w == w0)) * Z::SLOT) + lane;
            };
            int at = me;            // where this warp's sum goes
            int nodes = w1 - w0 + 1, idx = me - w0, stride = 1;  // of the level
            unsigned int *count = a.count;
            for (;;) {
                float2 *ps = part(at);
                if (store_ok(reinterpret_cast<float *>(ps - lane) + Z::SLOT - 1 - a.part, a.part_len, a.err)) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (j == 1 && !two) break;
#pragma unroll
                        for (int n = 0; n < NO; ++n) ps[(n * 2 + j) * 32] = make_float2(o[n][2 * j], o[n][2 * j + 1]);
                        ps[(NO * 2 + j) * 32] = make_float2(m[j], l[j]);
                    }
                }
                __threadfence();
                __syncwarp();
                const int first = idx / MERGE * MERGE, n_parts = min(MERGE, nodes - first);
                at = w0 + first * stride;
                int last = 0;
                if (lane == 0) {
                    unsigned int *c = count + 2 * at + (first == 0);
                    last = store_ok(c - a.count, a.count_len, a.err) &&
                           atomic_add_acq_rel_gpu(c, 1u) == static_cast<unsigned>(n_parts - 1);
                    if (last) *c = 0u;
                }
                if (!__shfl_sync(0xffffffffu, last, 0)) break;
                __syncwarp();  // lane 0's acquire holds for the other lanes' reads too: a shuffle orders no memory
                m[0] = m[1] = -INFINITY;
                l[0] = l[1] = 0.0f;
#pragma unroll
                for (int i = 0; i < NO; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
                if (two)
                    add_parts<2, 2, NO>(part(at), stride, n_parts, w0 == at, Z::SLOT, o, m, l);
                else
                    add_parts<1, 4, NO>(part(at), stride, n_parts, w0 == at, Z::SLOT, o, m, l);
                idx = first / MERGE;
                nodes = (nodes + MERGE - 1) / MERGE;
                stride *= MERGE;
                count += 2 * NW * gridDim.x;
                if (nodes == 1) {
                    store = true;
                    break;
                }
            }
        }
        if (store) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (trow[j] < 0) continue;
                const float inv = inverse(l[j]);
                const int64_t at = trow[j] * a.o_stride + static_cast<int64_t>(hrow[j]) * a.D + (lane & 3) * 2;
                const int64_t o_len = static_cast<int64_t>(a.T - 1) * a.o_stride + static_cast<int64_t>(a.Hq) * a.D;
#pragma unroll
                for (int n = 0; n < NO; ++n) {
                    if (n * 8 >= a.D || !store_ok(at + n * 8 + 1, o_len, a.err)) break;
                    const float x = o[n][2 * j] * inv, y = o[n][2 * j + 1] * inv;
                    if (a.ot == Q4_F32)
                        *reinterpret_cast<float2 *>(static_cast<float *>(a.o) + at + n * 8) = make_float2(x, y);
                    else
                        *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.o) + at + n * 8) = pack2<F16>(x, y);
                }
                if ((lane & 3) == 0) store_lse(a, trow[j], hrow[j], m[j] - LIFT<F16>, l[j]);
            }
        }
        __syncwarp();
    }
    cp_async_wait<0>();
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
    p.grid = std::min<int>(sm_count, MOST_CTAS);
    // One row tile streams the cache once; more tiles would read it again (us,
    // streaming / tensor cores: 8 rows, 2 x 32768 keys 55 / 63; 24 rows, 16
    // requests of 4000 keys 81 / 62; 32 rows 84 / 62; 64 rows 136 / 63).  The
    // whole call goes by its longest request: 40 decodes of 8000 keys take 206
    // alone, a chunk of 128 after 2000 takes 40, both in one call 236.
    p.tc = max_fresh > R / GQ;
    const size_t slot = (D > 64 ? Sizes<128>::SLOT : Sizes<64>::SLOT) * sizeof(float);
    const size_t part = p.tc ? attention_tc_part_bytes(D, p.grid) : 2 * static_cast<size_t>(p.grid) * NW * slot;
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
