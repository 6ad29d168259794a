// attention8.cu -- attention over the 8-bit blocked cache, few rows per KV
// head: the decode kernel.
//
// Rows.  The n new tokens of a request and the GQ query heads that share a KV
// head form n * GQ rows that read the same keys, in row tiles of 8, 16 or 32.  Bound:
// with one tile the codes are read once; HBM bounds the call as long as a
// byte's work, twice what a byte of a 16-bit cache brings, fits beside its load.
//
// Keys are the m of mma.sync m16n8k16 and rows its n: with 8 rows no part of
// the tile is empty, and codes are A fragments, widened to binary16 in registers
// on the way from shared memory (exactly: int8 by the bytes of 1024 + 128 + c,
// e4m3 by its conversion instruction).
//   scores   S^T[key][row] = K Q^T: the order of the dims in the sum is free, so a
//            lane takes 16 consecutive bytes of its two keys and the queries are
//            permuted alike;
//   outputs  O^T[dim][row] = V^T P^T: a lane takes 16 consecutive dims of four
//            keys and pairs the keys' bytes; it ends with 16 consecutive dims of
//            its two rows.  The weights turn by movmatrix in between.
// Queries in bf16 are scaled by a power of two per row, so that their largest
// lies in [2^14, 2^15), and go to binary16 without rounding as long as no other one
// lies more than 2^31 below it.  Otherwise (the large ones may meet zero codes) the
// piece is summed by the careful loop below, where queries stay in bf16 and codes
// are widened to that.
//
// Scales.  A unit is 16 keys, all of one block, so its two scales are uniform:
// 2^ek goes into the factor of the scores, 2^ev into the weights' exponent: with
// x_j = s_j + ev the second product sums 2^(x_j - ref) c_j and the row sum
// 2^(x_j - ref) 2^-ev, both under one running reference that follows x.  The
// reference lies 2^7 below the x that it was taken from and moves when that is
// passed by 2^8, so the weights in binary16 (which end at 2^16 and 2^-25) are at
// least 2^(7 - d) times their softmax weight (1 at most), where ev lies d below
// the largest so far.  At the first unit with d > 7 the piece goes on in a careful
// loop, where each unit has its own reference and its product is added in f32.  So
// a weight is off by 2^-12 of itself or 2^-25 of the largest, whatever the scales:
// what a dim holds beside zero codes of a large scale is kept.
//
// Work.  As in the 16-bit kernel (attention.cu): all units of the call form one
// sequence cut into an equal range per warp; a ring of units per warp filled by
// cp.async; split items meet in a tree, in sequence order.
//
// Measured (64 query / 8 KV heads of 128, bf16, graph): 48 requests of 1001..24576
// keys, int8, 200 us, 6.3 TB/s (0.93 of the measured copy bandwidth; over 16 bits
// 384 us); 32 of 101..8192 keys, e4m3, 57 us (0.70; 96 us over 16 bits); 32 of
// 8001 92 us int8, 90 e4m3, 62 with heads of 64; one of 65536 40 us; one of 777
// keys (32 heads) 14 us, which is latency.  DRAM reads are 1.004 of the codes;
// the arithmetic pipe of the bytes' permutations is 45% busy.
// Rows cost: 32 requests of 8000, int8, with 2 new tokens (16 rows) 116 us, with 4
// (32) 174: four row tiles leave room for 8 warps, which issue 0.46 instructions per
// cycle and scheduler (dependent ones), and mma.sync is at 29% of its rate.
#include <type_traits>

#include "attention.cuh"
#include "cache8.cuh"

namespace q4 {
namespace {

constexpr int TK = 16;       // keys per unit
// Warps: 12 with 8 rows (48 requests of 1001..24576 keys, 64/8 heads of 128: 205
// us; 8 warps 221, 16 204, but 32 of 101..8192 keys 57, 60 and 63), 8 with 16 (2
// new tokens after 8000, 32 requests: 115; 12 warps spill: 131, or with the queries
// in shared memory 119) and 32.
template <int NT>
constexpr int WARPS = NT == 1 ? 12 : 8;
static_assert(WARPS<2> == WARPS<4>, "workspace");
// (32 keys a unit at head sizes up to 64 gained nothing: 32 requests of 8000, 64/8
// heads of 64, 62.6 us either way.)
constexpr int PAD = 4, MIN_UNITS = 4;
constexpr float LIFT = 7.0f, SLACK = 8.0f;
constexpr int NEAR = 7;  // powers of two that scales under one reference lie below the largest
constexpr int MERGE = 8, LEVELS = 4, MOST_CTAS = 256;
static_assert(MERGE * MERGE * MERGE * MERGE >= WARPS<1> * MOST_CTAS, "levels");
static_assert(LEVELS * 2 * WARPS<1> * MOST_CTAS * sizeof(unsigned int) <= ATTN_COUNTER_BYTES, "counters");

template <int DP, int NT>
struct Sizes {
    static constexpr int STAGES = DP == 128 ? (NT == 1 ? 3 : NT == 2 ? 6 : 4) : 6;  // units in flight per warp
    static constexpr int TILE = TK * DP;               // bytes of a unit's keys
    static constexpr int RING = STAGES * 2 * TILE;
    static constexpr int QUERIES = NT == 4 ? NT * DP * 16 : 0;  // of a warp, where registers are too few
    static constexpr int SMEM = WARPS<NT> * (RING + QUERIES + STAGES * 2 * 4);
    static constexpr int SLOT = 128 * NT * (DP / 16 + 1);  // floats of a partial result
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t at)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t at)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at) : "memory");
    return v;
}

template <bool F16 = true>
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

__device__ __forceinline__ uint32_t transposed(uint32_t x)
{
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// Bytes 0, 1 (lo) and 2, 3 (hi) of a word of codes as pairs of binary16.
template <int CODE>
__device__ __forceinline__ void widen(uint32_t w, uint32_t &lo, uint32_t &hi)
{
    if (CODE == I8) {
        const uint32_t u = w ^ 0x80808080u;
        const __half2 off = __half2half2(__ushort_as_half(0xE480));  // -(1024 + 128)
        const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 x = __hadd2(*reinterpret_cast<const __half2 *>(&a), off), y = __hadd2(*reinterpret_cast<const __half2 *>(&b), off);
        lo = *reinterpret_cast<const uint32_t *>(&x);
        hi = *reinterpret_cast<const uint32_t *>(&y);
    } else {
        lo = e4m3_to_f16x2(w);
        hi = e4m3_to_f16x2(w >> 16);
    }
}

// Adds NT row tiles of n parts, the first at x and the others 2 * stride slots on
// each (a first piece of an item lies in the odd slot of its worker), to empty
// sums; the tiles' references and sums lie ml on.  AHEAD parts' loads are in flight.
template <int NT, int NO, int AHEAD>
__device__ __forceinline__ void add_parts(const float4 *x, int ml, int stride, int n, bool odd, int slot, float (&o)[NT][NO][4],
                                          float (&m)[NT][2], float (&l)[NT][2])
{
    const float4 *even = x - (odd ? slot / 4 : 0);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        m[t][0] = m[t][1] = -INFINITY;
        l[t][0] = l[t][1] = 0.0f;
#pragma unroll
        for (int k = 0; k < NO; ++k) o[t][k][0] = o[t][k][1] = o[t][k][2] = o[t][k][3] = 0.0f;
    }
#pragma unroll 1
    for (int i0 = 0; i0 < n; i0 += AHEAD) {
        float4 y[AHEAD][NT][NO], r[AHEAD][NT];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const bool in = i0 + i < n;
            const float4 *p = i0 + i == 0 ? x : even + static_cast<int64_t>(i0 + i) * stride * (slot / 2);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                r[i][t] = in ? __ldcg(p + ml + t * 32) : make_float4(-INFINITY, 0.0f, -INFINITY, 0.0f);
#pragma unroll
                for (int k = 0; k < NO; ++k) y[i][t][k] = in ? __ldcg(p + (t * NO + k) * 32) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            }
        }
#pragma unroll
        for (int i = 0; i < AHEAD; ++i)
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                float g0[2], g1[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float mi = j ? r[i][t].z : r[i][t].x, li = j ? r[i][t].w : r[i][t].y;
                    const float mn = fmaxf(m[t][j], mi), ref = mn == -INFINITY ? 0.0f : mn;
                    g0[j] = ex2(m[t][j] - ref);
                    g1[j] = ex2(mi - ref);
                    m[t][j] = mn;
                    l[t][j] = l[t][j] * g0[j] + li * g1[j];
                }
#pragma unroll
                for (int k = 0; k < NO; ++k) {
                    o[t][k][0] = o[t][k][0] * g0[0] + y[i][t][k].x * g1[0];
                    o[t][k][1] = o[t][k][1] * g0[1] + y[i][t][k].y * g1[1];
                    o[t][k][2] = o[t][k][2] * g0[0] + y[i][t][k].z * g1[0];
                    o[t][k][3] = o[t][k][3] * g0[1] + y[i][t][k].w * g1[1];
                }
            }
    }
}

template <int CODE, bool F16, int DP, int NT>
__global__ void __launch_bounds__(WARPS<NT> * 32, 1) k_attn8_stream(const AttnArgs a)
{
    using X = Exponents<CODE, F16>;
    using Z = Sizes<DP, NT>;
    constexpr int R = 8 * NT, STAGES = Z::STAGES, NW = WARPS<NT>;
    constexpr int CH = DP / 16, RPI = 32 / CH, LPT = TK / RPI;  // 16-byte pieces of a key; keys per load; loads
    constexpr int KH = DP / 64;                                 // pieces of a key that a lane takes
    constexpr int NO = DP / 16;                                 // output m tiles
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ LocateScratch ls;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, lg = lane >> 2, lt = lane & 3;

    grid_dep_wait();
    grid_dep_launch_dependents();
    sum_slabs<R, TK, NW, PAD>(a, ls);
    // neighbours in the sequence on different SMs: few units use many SMs
    const int me = warp * gridDim.x + blockIdx.x;
    const Range rng = find_share<R, TK, NW, MIN_UNITS, PAD>(a, ls, me, NW * gridDim.x);
    if (rng.u0 >= rng.u1) return;

    using Pieces = Walk<R, TK, PAD>;
    Pieces k(a, rng), ld = k;  // being summed; being loaded
    const uint32_t ring = smem_u32(smem) + warp * Z::RING;
    int *const scales = reinterpret_cast<int *>(smem + NW * (Z::RING + Z::QUERIES)) + warp * STAGES * 2;  // (ek, ev) per slot
    uint4 *const queries = reinterpret_cast<uint4 *>(smem + NW * Z::RING + warp * Z::QUERIES) + lane;  // [piece][tiles 2t, 2t + 1][lane]
    const uint8_t *const kb = reinterpret_cast<const uint8_t *>(a.k), *const vb = reinterpret_cast<const uint8_t *>(a.v);
    int ld_i = 0, ld_slot = 0;  // unit of ld, ring slot
    int exp_slot = -1;  // exponents on their way (lanes 0-15 keys', 16-31 values'):
    int exp = 0;        // kept a unit later, so that nothing waits for their loads
    auto block_of = [&]() {  // table entry of the unit to load
        const int key = (ld.kt0 + ld.kt + ld_i) * TK;
        return ld.more(rng) && key < ld.kv ? a.table[ld.it.b * a.table_stride + a.by_S.div(key)] : -1;
    };
    int blk = block_of();
    auto issue = [&]() {
        if (exp_slot >= 0 && (lane & 15) == 0) scales[exp_slot * 2 + (lane >> 4)] = X::of(exp);
        exp_slot = -1;
        if (ld.more(rng)) {
            const int key = (ld.kt0 + ld.kt + ld_i) * TK;
            const bool in = static_cast<unsigned>(blk) < static_cast<unsigned>(a.blocks);
            const uint32_t dst = ring + ld_slot * 2 * Z::TILE;
            // lane: 16-byte piece p of keys hi, hi + RPI, ..
            const int p = lane % CH, hi = lane / CH;
            int64_t at = in ? blk * a.block_stride + (key - a.by_S.div(key) * a.S + hi) * a.token_stride +
                                  ld.it.head * a.head_stride + p * 16
                            : 0;
            // (outside the cache the least one: zeros lift no reference over real values)
            exp = in ? (lane < 16 ? a.k_exp : a.v_exp)[static_cast<int64_t>(blk) * a.Hkv + ld.it.head] : 0;
            exp_slot = ld_slot;
            const int rows = in && p * 16 < a.D ? ld.kv - key : 0;  // keys that exist
            // and those that the window leaves to some row
            const int row0 = a.window > 0 && ld.kt + ld_i == 0 ? ld.first_key(a) - key : 0;
#pragma unroll
            for (int l = 0; l < LPT; ++l) {
                const int row = l * RPI + hi;
                const bool ok = row >= row0 && row < rows;
                // no two of the lanes that read together meet in a bank
                const int pk = DP == 128 ? p ^ ((row & 1) << 2) : p;
                const int pv = DP == 128 ? p ^ ((row >> 1 & 3) << 1) : p ^ (row >> 1 & 3);
                cp_async16(dst + row * DP + (pk << 4), kb + (ok ? at : 0), ok);
                cp_async16(dst + Z::TILE + row * DP + (pv << 4), vb + (ok ? at : 0), ok);
                at += RPI * a.token_stride;
            }
            ld_slot = ld_slot + 1 == STAGES ? 0 : ld_slot + 1;
            if (++ld_i == ld.nu) {
                ld.next(a, rng);
                ld_i = 0;
            }
            blk = block_of();
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) issue();

    int slot = 0;
    for (; k.more(rng); k.next(a, rng)) {
        // ---- queries as B fragments: row lg of a tile, the lane's pieces of it; in
        // binary16, or as they are (bf16 from 2^111 on by up to 2^-17: no sum of 128
        // products with 448 passes f32).  True if binary16 would lose some of them.
        uint32_t qf[NT][KH * 4][2];
        float cr[NT][2];  // scores' factor of rows 2 lt and 2 lt + 1
        auto load_queries = [&](auto as_they_are) {
            constexpr bool ALIKE = decltype(as_they_are)::value;
            bool lossy = false;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int r = k.row0 + 8 * t + lg;
                const bool in = r < k.row1;
                const int tok = in ? a.by_GQ.div(r) : 0;
                const uint16_t *q = a.q + (k.t0 + tok) * a.q_stride + static_cast<int64_t>(k.it.head * a.GQ + r - tok * a.GQ) * a.D;
                uint32_t peak = 0, least = ~0u;  // (less 1, so that zeros do not count)
#pragma unroll
                for (int h = 0; h < KH; ++h) {
                    const int d = (lt + 4 * h) * 16;
                    uint4 x = make_uint4(0, 0, 0, 0), y = x;
                    if (in && d < a.D) {
                        x = *reinterpret_cast<const uint4 *>(q + d);
                        y = *reinterpret_cast<const uint4 *>(q + d + 8);
                    }
                    const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        qf[t][h * 4 + i / 2][i & 1] = w[i];
                        const uint32_t lo = w[i] & 0x7FFFu, hi = w[i] >> 16 & 0x7FFFu;
                        if (!F16) peak = max(peak, max(lo, hi));
                        if (!F16 && !ALIKE) least = min(least, min(lo - 1, hi - 1));
                    }
                }
                int ex = 0;
                if (!F16) {
                    peak = max(peak, __shfl_xor_sync(0xffffffffu, peak, 1));
                    peak = max(peak, __shfl_xor_sync(0xffffffffu, peak, 2));
                    const int top = static_cast<int>(peak >> 7) - 127;
                    if (!ALIKE) lossy |= static_cast<int>(least + 1 >> 7) - 127 < top - 31 && least != ~0u;
                    ex = ALIKE ? max(top - 110, 0) : peak ? min(max(top - 14, -126), 126) : 0;
                    const float f = pow2(-ex);
                    if (peak >= 0x7F80u) ex = 0;  // scores of a row that is not finite are not either, whatever their factor
#pragma unroll
                    for (int i = 0; i < KH * 4; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint32_t w = qf[t][i][j];
                            qf[t][i][j] = pack2<!ALIKE>(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f);
                        }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) cr[t][j] = a.scale_log2 * pow2(__shfl_sync(0xffffffffu, ex, 4 * (2 * lt + j)));
                if (NT == 4) {  // (read by the same lane alone)
#pragma unroll
                    for (int i = 0; i < KH * 4; ++i)
                        *reinterpret_cast<uint2 *>(reinterpret_cast<uint32_t *>(queries + (i * NT / 2 + t / 2) * 32) + 2 * (t & 1)) =
                            make_uint2(qf[t][i][0], qf[t][i][1]);
                }
            }
            return __any_sync(0xffffffffu, lossy) != 0;
        };
        const bool lossy = load_queries(std::false_type{});
        const int lo_place = k.base + a.by_GQ.div(k.row0), hi_place = k.base + a.by_GQ.div(k.row1 - 1);

        float o[NT][NO][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            m[t][0] = m[t][1] = -INFINITY;
            l[t][0] = l[t][1] = 0.0f;
#pragma unroll
            for (int i = 0; i < NO; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.0f;
        }

        // Codes of the lane's two keys as A fragments, 4 dims of each half at a time.
        auto keys = [&](uint32_t ks, auto &&each) {
#pragma unroll
            for (int h = 0; h < KH; ++h) {
                const int p = DP == 128 ? (lt + 4 * h) ^ ((lg & 1) << 2) : lt;
                const uint4 x = lds16(ks + lg * DP + (p << 4)), y = lds16(ks + (lg + 8) * DP + (p << 4));
                const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t f[4];
                    widen<CODE>(xw[w], f[0], f[2]);
                    widen<CODE>(yw[w], f[1], f[3]);
                    each(h * 4 + w, f);
                }
            }
        };
        // The lane's dims of keys 2 lt, 2 lt + 1, and those + 8, two m tiles at a time:
        // dims 4w, 4w + 1 and 4w + 2, 4w + 3.
        auto values = [&](uint32_t vs, auto &&each) {
            uint32_t v[4][NO / 2];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = 2 * lt + (e & 1) + (e >> 1) * 8;
                if (DP == 128) {
                    const uint4 x = lds16(vs + key * DP + ((lg ^ ((key >> 1 & 3) << 1)) << 4));
                    v[e][0] = x.x;
                    v[e][1] = x.y;
                    v[e][NO / 2 - 2] = x.z;
                    v[e][NO / 2 - 1] = x.w;
                } else {
                    const uint2 x = lds8(vs + key * DP + (((lg >> 1) ^ (key >> 1 & 3)) << 4) + (lg & 1) * 8);
                    v[e][0] = x.x;
                    v[e][1] = x.y;
                }
            }
#pragma unroll
            for (int w = 0; w < NO / 2; ++w) {
                uint32_t f[2][4];
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    widen<CODE>(__byte_perm(v[2 * b][w], v[2 * b + 1][w], 0x5140), f[0][2 * b], f[0][2 * b + 1]);
                    widen<CODE>(__byte_perm(v[2 * b][w], v[2 * b + 1][w], 0x7362), f[1][2 * b], f[1][2 * b + 1]);
                }
                each(2 * w, f[0]);
                each(2 * w + 1, f[1]);
            }
        };
        // Of a unit from key0 on: whether some row does not see all of it; and the mask.
        auto in_part = [&](int key0) { return key0 + TK - 1 > lo_place || (a.window > 0 && key0 <= hi_place - a.window); };
        auto mask = [&](int key0, int t, float (&x)[4]) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = k.row0 + 8 * t + 2 * lt + j, at = r < k.row1 ? k.base + a.by_GQ.div(r) : -1;
#pragma unroll
                for (int e = j; e < 4; e += 2) {
                    const int key = key0 + lg + (e >> 1) * 8;
                    if (!(key <= at && (a.window == 0 || key > at - a.window))) x[e] = -INFINITY;
                }
            }
        };
        auto of_warp = [](float x) {  // the largest of a row's keys
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
            return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        };

        int i = 0, top = -128;  // the unit, the largest ev so far
        for (; !lossy && i < k.nu; ++i) {
            asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
            __syncwarp();  // the other lanes' copies too; and all lanes are done with the slot below
            issue();
            const uint32_t ks = ring + slot * 2 * Z::TILE, vs = ks + Z::TILE;
            const int ek = scales[slot * 2], ev = scales[slot * 2 + 1];
            slot = slot + 1 == STAGES ? 0 : slot + 1;
            float sc[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t) sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.0f;
            keys(ks, [&](int c, const uint32_t (&f)[4]) {
                if (NT == 4) {
#pragma unroll
                    for (int t = 0; t < NT; t += 2) {
                        const uint4 b = lds16(smem_u32(queries + (c * NT + t) / 2 * 32));
                        mma16816(sc[t], f, b.x, b.y);
                        mma16816(sc[(t + 1) % NT], f, b.z, b.w);
                    }
                } else {
#pragma unroll
                    for (int t = 0; t < NT; ++t) mma16816(sc[t], f, qf[t][c][0], qf[t][c][1]);
                }
            });
            // ---- mask and weights in units of log 2
            const int key0 = (k.kt0 + k.kt + i) * TK;
            const bool part = in_part(key0);
            const float fk = pow2(ek), fv = static_cast<float>(ev), undo = pow2(-ev);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[t][e] = fmaf(sc[t][e], cr[t][e & 1] * fk, fv);
            if (part) {  // (a branch: as selects the unmasked units took 4% longer, with 32 rows 20%)
#pragma unroll
                for (int t = 0; t < NT; ++t) mask(key0, t, sc[t]);
            }
            const bool far = ev < top - NEAR;
            top = max(top, ev);
            bool past = far;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e) past |= !(sc[t][e] <= m[t][e & 1] + SLACK);
            if (__any_sync(0xffffffffu, past)) {
                if (far) break;
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    float f[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        // NaN of a factor past f32 (2^113 of the queries times 2^48) and a score of 0
                        if (!F16 && isinf(cr[t][j] * fk)) {
                            if (isnan(sc[t][j])) sc[t][j] = fv;
                            if (isnan(sc[t][2 + j])) sc[t][2 + j] = fv;
                        }
                        const float mn = fmaxf(m[t][j], of_warp(fmaxf(sc[t][j], sc[t][2 + j]))), ref = mn == -INFINITY ? 0.0f : mn;
                        f[j] = ex2(m[t][j] - ref);
                        m[t][j] = mn;
                        l[t][j] *= f[j];
                    }
#pragma unroll
                    for (int n = 0; n < NO; ++n) {
                        o[t][n][0] *= f[0];
                        o[t][n][1] *= f[1];
                        o[t][n][2] *= f[0];
                        o[t][n][3] *= f[1];
                    }
                }
            }
            uint32_t p[NT][2];  // B fragments: keys are k, rows n
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float ref = m[t][j] == -INFINITY ? 0.0f : m[t][j];
                    sc[t][j] = ex2((sc[t][j] - ref) + LIFT);  // no rounding of a large ref
                    sc[t][2 + j] = ex2((sc[t][2 + j] - ref) + LIFT);
                    l[t][j] = fmaf(sc[t][j] + sc[t][2 + j], undo, l[t][j]);
                }
                p[t][0] = transposed(pack2<true>(sc[t][0], sc[t][1]));
                p[t][1] = transposed(pack2<true>(sc[t][2], sc[t][3]));
            }
            values(vs, [&](int n, const uint32_t (&f)[4]) {
#pragma unroll
                for (int t = 0; t < NT; ++t) mma16816(o[t][n], f, p[t][0], p[t][1]);
            });
        }
        // ---- the careful loop, a tile at a time.  (As a branch of the loop above it
        // cost that one 2 to 11%, with the sums set aside in local memory 2 to 12%,
        // this way 0 to 5%: 48 long decodes 197.7 -> 201.0 us, 32 requests with 2 new
        // tokens 112.2 -> 115.8, with 4 164.8 -> 173.4.  Where all pieces go through
        // here they take 1.2 (8 rows) to 3 times (32) as long.)
        if (!F16 && i < k.nu) load_queries(std::true_type{});
        for (bool landed = !lossy; i < k.nu; ++i, landed = false) {
            if (!landed) {
                asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
                __syncwarp();
                issue();
                slot = slot + 1 == STAGES ? 0 : slot + 1;
            }
            const int at = slot == 0 ? STAGES - 1 : slot - 1, key0 = (k.kt0 + k.kt + i) * TK;
            const uint32_t ks = ring + at * 2 * Z::TILE, vs = ks + Z::TILE;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const int ev = scales[at * 2 + 1];
                const float fk = pow2(scales[at * 2]), undo = pow2(-ev);
                float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                keys(ks, [&](int c, const uint32_t (&f)[4]) {
                    uint2 b = make_uint2(qf[t][c][0], qf[t][c][1]);
                    if (NT == 4) b = lds8(smem_u32(queries + (c * NT + t) / 2 * 32) + 8 * (t & 1));
                    if (F16) {
                        mma16816(x, f, b.x, b.y);
                    } else {
                        const uint32_t g[4] = {f16x2_upper(f[0]), f16x2_upper(f[1]), f16x2_upper(f[2]), f16x2_upper(f[3])};
                        mma16816<false>(x, g, b.x, b.y);
                    }
                });
                // (in this order a product of 0 stays 0, whatever the factors)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = fmaf(x[e] * cr[t][e & 1], fk, static_cast<float>(ev));
                if (in_part(key0)) mask(key0, t, x);
                float f[2], g[2];  // factors of what was summed and of the unit
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float mx = of_warp(fmaxf(x[j], x[2 + j])), own = mx == -INFINITY ? 0.0f : mx;
                    const float mn = fmaxf(m[t][j], mx), ref = mn == -INFINITY ? 0.0f : mn;
                    f[j] = ex2(m[t][j] - ref);
                    g[j] = ex2(mx - ref);
                    m[t][j] = mn;
                    x[j] = ex2((x[j] - own) + LIFT);
                    x[2 + j] = ex2((x[2 + j] - own) + LIFT);
                    l[t][j] = fmaf((x[j] + x[2 + j]) * undo, g[j], l[t][j] * f[j]);
                }
                const uint32_t p0 = transposed(pack2<true>(x[0], x[1])), p1 = transposed(pack2<true>(x[2], x[3]));
                values(vs, [&](int n, const uint32_t (&w)[4]) {
                    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    mma16816(y, w, p0, p1);
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[t][n][e] = fmaf(y[e], g[e & 1], o[t][n][e] * f[e & 1]);
                });
                __syncwarp();  // (keeps the tiles' code apart: without it 32 rows spill more, 169 -> 186 us)
            }
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                l[t][j] += __shfl_xor_sync(0xffffffffu, l[t][j], 4);
                l[t][j] += __shfl_xor_sync(0xffffffffu, l[t][j], 8);
                l[t][j] += __shfl_xor_sync(0xffffffffu, l[t][j], 16);
            }

        // a row tile's outputs
        auto store = [&](int t, const float (&o)[NO][4], const float (&m)[2], const float (&l)[2]) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = k.row0 + 8 * t + 2 * lt + j;
                if (r >= k.row1) continue;
                const int tok = a.by_GQ.div(r), h = k.it.head * a.GQ + r - tok * a.GQ;
                const float inv = inverse(l[j]);
                float y[2 * NO];
#pragma unroll
                for (int n = 0; n < NO; ++n) {
                    y[2 * n] = o[n][j] * inv;
                    y[2 * n + 1] = o[n][2 + j] * inv;
                }
                store_dims<F16, 2 * NO>(a, k.t0 + tok, h, lg * 2 * NO, y);
                if (lg == 0) store_lse(a, k.t0 + tok, h, m[j] - LIFT, l[j]);
            }
        };
        auto store_all = [&]() {
#pragma unroll
            for (int t = 0; t < NT; ++t) store(t, o[t], m[t], l[t]);
        };
        const bool split = !k.whole();
        bool whole = !split;  // the registers hold the item's sum
        if (NT == 4 && whole) store_all();
        if (split) {
            // as in the 16-bit kernel: the item's pieces are the leaves of a tree
            // of MERGE-fold nodes over the workers that hold them; whoever
            // completes a node adds its parts in order, leaves the sum in the
            // first part's place and goes on to the next level.  A node's counter
            // goes by its first worker, which may also hold the end of another item.
            int w0, w1;
            k.holders(rng, w0, w1);
            // [tile][m tile][lane][4], then [tile][lane](reference, sum) of two rows
            auto slot_of = [&](int w) {
                return reinterpret_cast<float4 *>(a.part + (2 * static_cast<int64_t>(w) + (w == w0)) * Z::SLOT) + lane;
            };
            auto keep = [&](float4 *ps, int t, const float (&o)[NO][4], const float (&m)[2], const float (&l)[2]) {
                if (!store_ok(reinterpret_cast<float *>(ps - lane) + Z::SLOT - 1 - a.part, a.part_len, a.err)) return;
#pragma unroll
                for (int n = 0; n < NO; ++n) ps[(t * NO + n) * 32] = make_float4(o[n][0], o[n][1], o[n][2], o[n][3]);
                ps[(NT * NO + t) * 32] = make_float4(m[0], l[0], m[1], l[1]);
            };
            int at = me;            // where this warp's sum goes
            int nodes = w1 - w0 + 1, idx = me - w0, stride = 1;  // of the level
            unsigned int *count = a.count;
            auto keep_all = [&]() {
                float4 *ps = slot_of(at);
#pragma unroll
                for (int t = 0; t < NT; ++t) keep(ps, t, o[t], m[t], l[t]);
            };
            if (NT == 4) keep_all();
            do {
                if (NT < 4) keep_all();
                __threadfence();
                __syncwarp();
                const int first = idx / MERGE * MERGE, n_parts = min(MERGE, nodes - first);
                at = w0 + first * stride;
                int last = 0;
                if (lane == 0) {
                    unsigned int *cnt = count + 2 * at + (first == 0);
                    last = store_ok(cnt - a.count, a.count_len, a.err) &&
                           atomic_add_acq_rel_gpu(cnt, 1u) == static_cast<unsigned>(n_parts - 1);
                    if (last) *cnt = 0u;
                }
                if (!__shfl_sync(0xffffffffu, last, 0)) break;
                __syncwarp();  // lane 0's acquire holds for the other lanes' reads too: a shuffle orders no memory
                idx = first / MERGE;
                nodes = (nodes + MERGE - 1) / MERGE;
                float4 *ps = slot_of(at);
                if constexpr (NT == 4) {
                    // a tile at a time, so that registers hold four parts' loads (all
                    // tiles of a part: 1 request of 30000 61.5 us, this way 55)
#pragma unroll 1
                    for (int t = 0; t < NT; ++t) {
                        float x[1][NO][4], mx[1][2], lx[1][2];
                        add_parts<1, NO, 4>(ps + t * NO * 32, (NT * NO + t - t * NO) * 32, stride, n_parts, w0 == at, Z::SLOT, x, mx, lx);
                        if (nodes == 1)
                            store(t, x[0], mx[0], lx[0]);
                        else
                            keep(ps, t, x[0], mx[0], lx[0]);
                    }
                } else {
                    add_parts<NT, NO, NT * NO <= 4 ? 2 : 1>(ps, NT * NO * 32, stride, n_parts, w0 == at, Z::SLOT, o, m, l);
                    whole = nodes == 1;
                }
                stride *= MERGE;
                count += 2 * NW * gridDim.x;
            } while (nodes > 1);
        }
        if (NT < 4 && whole) store_all();
        __syncwarp();
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

template <int CODE, bool F16, int DP, int NT>
cudaError_t launch(const AttnPlan &p, const AttnArgs &a, cudaStream_t s)
{
    static std::atomic<bool> done[64];
    auto kern = k_attn8_stream<CODE, F16, DP, NT>;
    const cudaError_t e = allow_smem(kern, Sizes<DP, NT>::SMEM, done);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3(p.grid), WARPS<NT> * 32, Sizes<DP, NT>::SMEM, s, a);
}

template <int CODE, bool F16>
cudaError_t launch_rows(const AttnPlan &p, const AttnArgs &a, cudaStream_t s)
{
    if (p.tiles == 4) return a.D > 64 ? launch<CODE, F16, 128, 4>(p, a, s) : launch<CODE, F16, 64, 4>(p, a, s);
    if (a.D > 64) return p.tiles == 1 ? launch<CODE, F16, 128, 1>(p, a, s) : launch<CODE, F16, 128, 2>(p, a, s);
    return p.tiles == 1 ? launch<CODE, F16, 64, 1>(p, a, s) : launch<CODE, F16, 64, 2>(p, a, s);
}

}  // namespace

// Up to 16 rows per KV head go to this kernel, more than 32 to the tensor cores'
// (attention8_tc.cu); between them it is this one if there are many requests and
// heads, as one with few splits each over many warps, whose 32 rows take long to
// join: 4 new tokens (32 rows) after 8000, int8, 8 KV heads, 4 requests 50 us here
// and 43 there, 8 requests 66 and 69, 32 requests 174 and 201; after 500, 8 requests
// 23 and 19, 64 requests 43 and 68.
static constexpr int64_t MANY = 64;

AttnPlan attention8_plan(int64_t max_fresh, int64_t GQ, int64_t D, int64_t items, int sm_count)
{
    AttnPlan p{};
    p.grid = std::min<int>(sm_count, MOST_CTAS);
    p.tc = max_fresh > 32 / GQ || (max_fresh > 16 / GQ && items < MANY);
    p.tiles = max_fresh > 16 / GQ ? 4 : max_fresh > 8 / GQ ? 2 : 1;
    // for any number of requests, and for steps of fewer new tokens too
    const size_t slot = (D > 64 ? Sizes<128, 1>::SLOT : Sizes<64, 1>::SLOT) * sizeof(float) * p.tiles;
    const size_t here = GQ > 32 ? 0 : 2 * static_cast<size_t>(p.grid) * (p.tiles == 1 ? WARPS<1> : WARPS<2>) * slot;
    const size_t there = p.tiles == 4 ? attention_tc_part_bytes(D, p.grid) : 0;
    p.workspace = ATTN_COUNTER_BYTES + std::max(here, there);
    return p;
}

cudaError_t attention8_launch(const AttnPlan &p, const AttnArgs &a, q4_code code, bool f16, cudaStream_t s)
{
    if (p.tc) return attention8_tc_launch(p.grid, a, code, f16, s);
    if (code == Q4_I8) return f16 ? launch_rows<I8, true>(p, a, s) : launch_rows<I8, false>(p, a, s);
    return f16 ? launch_rows<E4M3, true>(p, a, s) : launch_rows<E4M3, false>(p, a, s);
}

}  // namespace q4
