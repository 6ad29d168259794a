// attention_tc.cu -- attention over the blocked KV cache, many rows per KV
// head: the tensor-core kernel.
//
// Rows.  The n new tokens of a request and the GQ query heads that share a
// KV head form n * GQ rows (token-major), taken in tiles of 256: two subtiles
// of 128 rows, each an M = 128 operand of tcgen05.mma, that share every key
// and value tile.  A key tile is 128 keys.  Bound: with 256 rows per byte of
// cache the tensor cores, and next to them the exponentials: a subtile and
// tile cost 2 * 128 * 128 * head_dim multiply-adds and 128 * 128 exponentials.
//
// One persistent CTA per SM takes an equal share of all (item, key tile)
// units of the call (attention.cuh), 12 warps with fixed roles:
//   warps 0-3, 4-7  softmax of subtile 0 and 1, a thread per row: scores from
//                   tensor memory, mask, weights back to tensor memory over
//                   the scores (the A operand of the second product), row sums
//                   in registers; at the end of an item the row's output;
//   warps 8-10      producers of keys, values and queries into the 128-byte
//                   swizzled operand layouts: tensor copies, one per run of
//                   keys that lies in one block of the cache for certain (16
//                   keys at least) and 64 dims, each lane issuing one; two
//                   slots of 32 KB each for keys and values.  Only the value
//                   tiles that hold the request's end or the window's
//                   beginning go by cp.async, which puts zeros outside (0
//                   times a stale NaN would reach the sums; stale keys only
//                   make scores that are masked), and queries whose group of
//                   heads does not divide 128;
//   warp 11         allocates tensor memory; one thread issues the MMAs.
// Tensor memory (512 columns): the two subtiles' scores (128 columns each)
// and outputs (head_dim each).  While one subtile's softmax runs, the other's
// products do: the issue order is P0 V(j), Q0 K(j+1), P1 V(j), Q1 K(j+1), on
// through the ends of items.
// MMAs of one thread run in order, so a subtile's next scores may be issued
// right behind the product that reads the weights they overwrite, and scores
// being complete implies that every earlier product is.
//
// The weights' reference follows the running maximum, but only moves when it
// is passed by more than 2^8: the output is rarely rescaled and the final
// division removes the reference, so the result is the same formula.  In
// binary16, which ends at 2^16 and 2^-25, the reference lies 2^7 below the
// maximum, so that weights reach 2^15 and many small ones beside a large one
// do not vanish.
// Keys that a tile's rows all see need no mask; only tiles on the diagonal or
// a window's edge do.
//
// Items cut by a range boundary leave their unscaled outputs, references and
// sums in the workspace; the subtile's last CTA to arrive adds them in CTA
// order.  Every barrier wait is bounded; on expiry the CTA raises the device
// error word, every role stops, copies and MMAs in flight are waited for,
// tensor memory is freed and the kernel returns.
//
// Measured (bf16, 64 query / 8 KV heads of 128, inputs from HBM): 512 new
// tokens after 16384 in 188 us, 1.49 PFLOP/s (0.77 of the measured peak; 180 to
// 182 us with inputs in L2); a prompt of 4096 tokens, 32 heads, f16, in 118 us,
// 1.17 PFLOP/s; 12 requests with 1..160 new tokens after 50..4000 in 81 us;
// prompts of 2048 with head sizes of 64, 80, 96 and 128 in 62, 73, 74 and 75
// us (80 and 96 run as 128), with f32 output 103.  A unit of 256 rows took some
// 2800 cycles when traced; its operations are 2048 cycles of the tensor pipe
// (8192 per cycle and SM).  The rest is the MMA thread's waits and commits,
// which come one after the other with its MMAs, as those queue only a few deep.
// The CTA's range stays in shared memory: held in registers it made the softmax
// warps spill (188 us against 186).
#include <type_traits>

#include "attention.cuh"
#include "tcgen05.cuh"

namespace q4 {
namespace {

constexpr int R = 256;   // rows per item
constexpr int SR = 128;  // rows per subtile
constexpr int TK = 128;  // keys per unit
// Places of the sequence that each item takes beside its units: beginning and
// finishing an item costs about as much as two units.
constexpr int PAD = 2;
constexpr int MIN_UNITS = 4;  // per CTA: a piece that is joined costs about as much as two units
constexpr int W_K = 8, W_V = 9, W_Q = 10;  // producers
constexpr int W_M = 11;         // MMA issue
constexpr int NW = 12, THREADS = NW * 32;  // 168 registers per thread; a 13th warp would cost 40 of them
constexpr int MANY_PARTS = 3;  // more parts behind the first are added four at a time
// Registers move from the copying and issuing warpgroup to the softmax ones,
// which keep a row's 128 scores in registers.
constexpr int REG_HI = 208, REG_LO = 80;
static_assert(2 * REG_HI + REG_LO <= 3 * 168, "within the registers of the launch");

// Powers of two that a weight's reference lies below the maximum it follows,
// and that the maximum may pass it by before it moves.
template <bool F16>
constexpr float LIFT = F16 ? 7.0f : 0.0f;
constexpr float SLACK = 8.0f;
// f32 rounds a row's largest score, as the reference, by up to 2^-24 of it, and
// the fused multiply-adds of the weights bring that back as a factor on all of
// them, which would leave the range of the types.  So for their weights a row's
// scores are scaled to this size (2^24) at most: larger ones that still come
// close differ by a few of f32's own steps.  (Scores taken from the reference
// before they are scaled need no such bound; prompts took 2% longer.)
constexpr float LARGE = 16777216.0f;
// A tile's sum of weights below which none of them is past the slack.
template <bool F16>
constexpr float MOST_SUM = F16 ? 32768.0f : 256.0f;

template <int DP>
struct Sizes {
    static constexpr int CH = DP / 64;           // 64-element chunks of a row
    static constexpr int CHUNK = 128 * 128;      // bytes of 128 rows of a chunk
    static constexpr int TILE = CH * CHUNK;      // 128 rows: a subtile's queries, a key or value tile
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_R = 2 * TILE;
    static constexpr int OFF_O = OFF_R + 4 * TILE;  // output staging, 32 rows x 128 bytes per warp
    static constexpr int OFF_B = OFF_O + 8 * 4096;
    static constexpr int NBAR = 8 + 4 + 6 + 1;
    static constexpr int SMEM = OFF_B + NBAR * 8 + 64 + 1024;  // slack to align the base
    static constexpr int PART = SR * (DP + 2);  // floats of a subtile's partial result
    static constexpr uint32_t S_COL = 0, O_COL = 256;
    static_assert(O_COL + 2 * DP <= 512, "scores and outputs fit tensor memory");
    static_assert(SMEM <= 227 * 1024, "one CTA per SM");
};

using Pieces = Walk<R, TK, PAD>;

// Units [a, b) of a piece that subtile w sees, and the places of its first and
// last row.
struct Seen {
    int a, b, lo, hi;
};
__device__ __forceinline__ Seen seen(const AttnArgs &a, const Pieces &k, int w)
{
    Seen s = {0, 0, -1, -1};
    const int r0 = k.row0 + w * SR, r1 = min(k.row1, r0 + SR);
    if (r0 >= r1) return s;
    s.lo = k.base + a.by_GQ.div(r0);
    s.hi = k.base + a.by_GQ.div(r1 - 1);
    if (s.hi < 0) return s;
    const int u0 = window_start(a, s.lo) / TK - k.kt0 - k.kt;
    const int u1 = s.hi / TK + 1 - k.kt0 - k.kt;
    s.a = min(max(u0, 0), k.nu);
    s.b = max(s.a, min(u1, k.nu));
    return s;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}

// One probe that may wait for the hardware's own time: reacts sooner than
// one with a long time given, and takes no issue slots as polling does (whole
// tiles of 256 rows: 4% and 7% of the time).
__device__ __forceinline__ bool mbar_ready(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// This lane's arrival on bar after its copies so far have landed, in order
// with the tensor cores' reads.
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar)
{
    asm volatile("cp.async.wait_all;" ::: "memory");
    fence_proxy_async_smem();
    mbar_arrive(bar);
}

// a * b + c and a + b on pairs of f32
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z)
{
    uint64_t a, b, c, d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(x.x), "f"(x.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(y.x), "f"(y.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(c) : "f"(z.x), "f"(z.y));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
    return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y)
{
    uint64_t a, b, d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(x.x), "f"(x.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(b) : "f"(y.x), "f"(y.y));
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(d));
    return r;
}

// A value that all lanes hold (at least 0), by an instruction whose result the
// compiler knows to be the same in all lanes: what only depends on such values
// stays in uniform registers, where the MMA instructions take their operands
// from, instead of being moved there for each of them.
__device__ __forceinline__ int uniform(int x) { return static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<uint32_t>(x))); }

// The call's tensor maps and how the producers use them.
struct Maps {
    CUtensorMap k, v;  // (dim, token, head, block), boxes of 64 x kb x 1 x 1
    CUtensorMap q;     // (dim, query head, row), boxes of 64 x GQ x 128 / GQ
    CUtensorMap o;     // the same of a 16-bit output, boxes of 64 x GQ x 32 / GQ
    int kb;            // keys per box: the largest power of two up to 128 that divides block_size
    int q_boxes;       // GQ divides 128: queries by tensor copies
    int o_boxes;       // GQ divides 32: a warp's output rows, when all exist, by one tensor copy
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3,
                                            uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
        : "memory");
}

// A warp's output rows to global memory, by one lane.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, int c0, int c1, int c2, uint32_t src)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(c2), "r"(src)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

template <bool F16, int DP>
__global__ void __launch_bounds__(THREADS, 1) k_attn_tc(const __grid_constant__ Maps maps, const AttnArgs a)
{
    using Z = Sizes<DP>;
    constexpr int C8 = DP / 8;  // 16-byte pieces of a row
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    // kfull/kempty: slots, two for keys then two for values; qfull/qempty:
    // queries; sfull: scores ready; pfull: weights stored (and the output
    // rescaled); ofull: output complete.  Each lane of a producer arrives.
    uint64_t *kfull = reinterpret_cast<uint64_t *>(smem + Z::OFF_B), *kempty = kfull + 4;
    uint64_t *qfull = kempty + 4, *qempty = qfull + 2, *sfull = qempty + 2, *pfull = sfull + 2;
    uint64_t *ofull = pfull + 2, *drain = ofull + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile int *last_s = reinterpret_cast<volatile int *>(tmem_slot + 2);  // [2]
    // what the MMA warp needs of a piece, written by the query producer before
    // it arrives on qfull[0] (pieces in turn): units, each subtile's first and
    // last of them, whether another piece follows
    volatile int *note = reinterpret_cast<volatile int *>(tmem_slot + 4);  // [2][6]
    __shared__ LocateScratch ls;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&kfull[i], 32);
            mbar_init(&kempty[i], 1);
        }
        for (int w = 0; w < 2; ++w) {
            mbar_init(&qfull[w], 32);
            mbar_init(&qempty[w], 1);
            mbar_init(&sfull[w], 1);
            mbar_init(&pfull[w], 4);
            mbar_init(&ofull[w], 1);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == W_M) tmem_alloc(tmem_slot, 512);
    grid_dep_wait();
    grid_dep_launch_dependents();
    tc_fence_before();
    share<R, TK, NW, MIN_UNITS, PAD>(a, ls, blockIdx.x, gridDim.x);  // barriers inside
    const Range &rng = ls.r;  // read where it is: a piece's end is rare, registers are not
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (mbar_ready(bar, parity)) return true;
        const uint64_t t0 = globaltimer_ns();
        for (;;) {
            if (mbar_ready(bar, parity)) return true;
            if (*abort_flag) return false;
            if (globaltimer_ns() - t0 > a.wait_ns) {
                *abort_flag = 1;
                atomicOr(a.err, ERR_TIMEOUT);
                return false;
            }
        }
    };
    // by whole warps: the lanes get one answer, also when a wait runs out
    auto warp_wait = [&](uint64_t *bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
    };
    bool ok = true;

    if (warp == W_K || warp == W_V) {
        // --------------------------------------------- keys and values
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_LO));
        const bool vals = warp == W_V;
        const CUtensorMap *map = vals ? &maps.v : &maps.k;
        const uint16_t *vh = a.v;
        uint64_t *full = kfull + (vals ? 2 : 0), *empty = kempty + (vals ? 2 : 0);
        const uint32_t ring = smem_u32(smem + Z::OFF_R) + (vals ? 2 * Z::TILE : 0);
        // lane: one box of a tile, keys [bk, bk + kb), chunk ch
        const int bk = lane / Z::CH * maps.kb, ch = lane % Z::CH;
        const bool boxed = bk < TK;
        const uint32_t bd = ch * Z::CHUNK + bk * 128;
        Pieces k(a, rng);
        int g = 0;  // units loaded
        for (; ok && k.more(rng) && !a.debug_no_copy; k.next(a, rng)) {
            const int *trow = a.table + k.it.b * a.table_stride;
            auto block_of = [&](int key) { return key < k.kv ? trow[a.by_S.div(key)] : -1; };
            const int first = (k.kt0 + k.kt) * TK;
            const int lo = a.window > 0 ? k.first_key(a) : 0;
            int blk = boxed ? block_of(first + bk) : -1;
            for (int j = 0; j < k.nu; ++j, ++g) {
                const int s = g & 1, key0 = first + j * TK;
                if (g >= 2 && !(ok = warp_wait(&empty[s], ((g >> 1) - 1) & 1))) break;
                const uint32_t dst = ring + s * Z::TILE;
                if (!vals || (key0 + TK <= k.kv && key0 >= lo)) {
                    if (boxed) {
                        // a block outside the cache reads as zeros
                        mbar_arrive_expect_tx(&full[s], maps.kb * 128);
                        const int key = key0 + bk;
                        tma_load_4d(dst + bd, map, ch * 64, key - a.by_S.div(key) * a.S, k.it.head, blk, &full[s]);
                        blk = j + 1 < k.nu ? block_of(key + TK) : -1;
                    } else {
                        mbar_arrive(&full[s]);
                    }
                    __syncwarp();
                } else {
                    if (boxed) blk = j + 1 < k.nu ? block_of(key0 + TK + bk) : -1;
                    // groups of 16 keys, each within one block of the cache
                    constexpr int RPI = 32 / C8;
                    const int c = lane % C8, hi = lane / C8;
                    const uint32_t dc = dst + (c >> 3) * Z::CHUNK + hi * 128;
#pragma unroll 1
                    for (int r0 = 0; r0 < TK; r0 += 16) {
                        const int key = key0 + r0, b = block_of(key);
                        const bool in = static_cast<unsigned>(b) < static_cast<unsigned>(a.blocks);
                        const uint16_t *base = vh + k.it.head * a.head_stride + (in ? b * a.block_stride : 0) +
                                               (key - a.by_S.div(key) * a.S) * a.token_stride + c * 8;
#pragma unroll
                        for (int l = 0; l < 16 / RPI; ++l) {
                            const int row = l * RPI + hi;
                            const bool ok16 = in && key + row < k.kv && key + row >= lo && c * 8 < a.D;
                            cp_async16(dc + (r0 + l * RPI) * 128 + (((c & 7) ^ (row & 7)) << 4),
                                       ok16 ? base + row * a.token_stride : vh, ok16);
                        }
                    }
                    cp_async_arrive(&full[s]);
                }
            }
        }
        // every copy lands before the CTA may exit
        asm volatile("cp.async.wait_all;" ::: "memory");
        for (int i = max(0, g - 2); i < g; ++i)
            mbar_wait_bounded(&full[i & 1], (i >> 1) & 1, abort_flag, a.wait_ns, a.err, false);
        __syncwarp();
    } else if (warp == W_Q) {
        // ------------------------------------------------------ queries
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_LO));
        const uint32_t sq = smem_u32(smem + Z::OFF_Q);
        Pieces k(a, rng);
        Seen s0, s1;
        int pc = 0, loaded = 0;
        for (; ok && k.more(rng) && !a.debug_no_copy; ++pc, k.next(a, rng)) {
            for (int w = 0; w < 2; ++w) {
                if (w == 0 && !k.same) {
                    s0 = seen(a, k, 0);
                    s1 = seen(a, k, 1);
                }
                if (pc > 0 && !(ok = warp_wait(&qempty[w], (pc - 1) & 1))) break;
                ++loaded;
                if (w == 0) {
                    if (lane == 0) {
                        volatile int *x = note + (pc & 1) * 6;
                        x[0] = k.nu;
                        x[1] = s0.a;
                        x[2] = s0.b;
                        x[3] = s1.a;
                        x[4] = s1.b;
                        x[5] = k.follows(rng);
                    }
                    __syncwarp();
                }
                const uint32_t dst = sq + w * Z::TILE;
                if (maps.q_boxes) {
                    // lane: one chunk.  Rows past the request's are other
                    // requests' (or zeros past T): their results go nowhere
                    if (lane < Z::CH) {
                        mbar_arrive_expect_tx(&qfull[w], SR * 128);
                        tma_load_3d(dst + lane * Z::CHUNK, &maps.q, lane * 64, k.it.head * a.GQ,
                                    k.t0 + a.by_GQ.div(k.row0 + w * SR), &qfull[w]);
                    } else {
                        mbar_arrive(&qfull[w]);
                    }
                    __syncwarp();
                } else {
                    constexpr int RPI = 32 / C8;
                    const int c = lane % C8, hi = lane / C8;
                    const int dt = RPI / a.GQ, dg = RPI - dt * a.GQ;
                    const int r = k.row0 + w * SR + hi, t = a.by_GQ.div(r);
                    int g = r - t * a.GQ, left = k.row1 - r;  // rows from this one on
                    const uint16_t *src = a.q + (k.t0 + t) * a.q_stride +
                                          static_cast<int64_t>(k.it.head * a.GQ + g) * a.D + c * 8;
                    const int64_t step = dt * a.q_stride + static_cast<int64_t>(dg) * a.D;
                    const int64_t wrap = a.q_stride - static_cast<int64_t>(a.GQ) * a.D;
#pragma unroll 1
                    for (int r0 = 0; r0 < SR; r0 += 8) {
#pragma unroll
                        for (int l = 0; l < 8 / RPI; ++l) {
                            const int row = l * RPI + hi;  // within 8 rows
                            const bool in = left > 0 && c * 8 < a.D;
                            cp_async16(dst + (c >> 3) * Z::CHUNK + (r0 + row) * 128 + (((c & 7) ^ row) << 4),
                                       in ? src : a.q, in);
                            left -= RPI;
                            src += step;
                            g += dg;
                            if (g >= a.GQ) {
                                g -= a.GQ;
                                src += wrap;
                            }
                        }
                    }
                    cp_async_arrive(&qfull[w]);
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        for (int i = max(0, loaded - 2); i < loaded; ++i)
            mbar_wait_bounded(&qfull[i & 1], (i >> 1) & 1, abort_flag, a.wait_ns, a.err, false);
        __syncwarp();
    } else if (warp == W_M) {
        // ---------------------------------------------------- MMA issue
        // the warp stays whole (one lane is elected per instruction): operands
        // that differ by lane would have to be moved for every MMA
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_LO));
        constexpr uint32_t AB = F16 ? 0u : 1u;
        const uint32_t id_qk = idesc_f16(AB, TK), id_pv = idesc_f16(AB, DP) | IDESC_B_MN;
        const uint64_t dq = sw128_desc(smem_u32(smem + Z::OFF_Q));
        const uint64_t dk = sw128_desc(smem_u32(smem + Z::OFF_R));
        const uint64_t dv = sw128_desc(smem_u32(smem + Z::OFF_R), Z::CHUNK);
        const uint32_t tm = uniform(tmem);
        // scores of subtile w with the keys in slot s; output of subtile w
        // with the values in slot s
        auto qk = [&](auto w_, int s) {
            constexpr int w = decltype(w_)::value;
            mma_rows_ss<DP / 16>(tm + Z::S_COL + w * 128, dq + ((w * Z::TILE) >> 4), dk + ((s * Z::TILE) >> 4), id_qk,
                                 &sfull[w]);
        };
        auto pv = [&](auto w_, int s, bool acc, uint32_t parity) {
            constexpr int w = decltype(w_)::value;
            if (!warp_wait(&pfull[w], parity)) return false;
            tc_fence_after();
            mma_rows_ts(tm + Z::O_COL + w * DP, tm + Z::S_COL + w * 128, dv + (((2 + s) * Z::TILE) >> 4), id_pv, acc);
            return true;
        };
        int g = 0;                  // units so far
        uint32_t np0 = 0, np1 = 0;  // weights consumed per subtile
        using C0 = std::integral_constant<int, 0>;
        using C1 = std::integral_constant<int, 1>;
        // The subtiles' streams run over the pieces' ends: while one subtile's
        // rows finish an item, the other's, and its own next scores, go on.
        int nu = 0, a0 = 0, b0 = 0, a1 = 0, b1 = 0, follows = 0;  // the piece
        int j = 0, pc = 0;
        bool more = __any_sync(0xffffffffu, Pieces(a, rng).more(rng));  // there is a next unit
        auto read_note = [&]() {
            const volatile int *x = note + (pc & 1) * 6;
            nu = uniform(x[0]);
            a0 = uniform(x[1]);
            b0 = uniform(x[2]);
            a1 = uniform(x[3]);
            b1 = uniform(x[4]);
            follows = uniform(x[5]);
        };
        if (more) {
            ok = warp_wait(&qfull[0], 0) && warp_wait(&qfull[1], 0) && warp_wait(&kfull[0], 0);
            if (ok) {
                read_note();
                if (a0 == 0 && b0 > 0) qk(C0(), 0);
                if (nu == 1) mma_commit_elected(&qempty[0]);
                if (a1 == 0 && b1 > 0) qk(C1(), 0);
                if (nu == 1) mma_commit_elected(&qempty[1]);
                mma_commit_elected(&kempty[0]);
            }
        }
        while (ok && more) {
            // unit g: its values in slot v of theirs, the next unit's keys in
            // slot nk of theirs
            const int v = g & 1, nk = v ^ 1;
            // the unit after this one: of this piece or the first of the next
            const bool turn = j + 1 == nu;
            more = !turn || follows;
            // what the unit needs beside the weights has usually landed: asked
            // for while the products issued last still run
            if (!(ok = warp_wait(&kfull[2 + v], (g >> 1) & 1))) break;
            if (more && !(ok = warp_wait(&kfull[nk], ((g + 1) >> 1) & 1))) break;
            if (j >= a0 && j < b0) {
                if (!(ok = pv(C0(), v, j > a0, np0++ & 1))) break;
                if (j == b0 - 1) mma_commit_elected(&ofull[0]);
            }
            const bool on1 = j >= a1 && j < b1, acc1 = j > a1, end1 = j == b1 - 1;
            ++j;
            if (more) {
                if (turn) {
                    j = 0;
                    ++pc;
                    if (!(ok = warp_wait(&qfull[0], pc & 1))) break;
                    read_note();
                }
                if (j >= a0 && j < b0) qk(C0(), nk);
                if (j + 1 == nu) mma_commit_elected(&qempty[0]);
            }
            if (on1) {
                if (!(ok = pv(C1(), v, acc1, np1++ & 1))) break;
                if (end1) mma_commit_elected(&ofull[1]);
            }
            mma_commit_elected(&kempty[2 + v]);
            if (more) {
                if (turn && !(ok = warp_wait(&qfull[1], pc & 1))) break;
                if (j >= a1 && j < b1) qk(C1(), nk);
                if (j + 1 == nu) mma_commit_elected(&qempty[1]);
                mma_commit_elected(&kempty[nk]);
            }
            ++g;
        }
        // MMAs in flight end before tensor memory is freed
        mma_commit_elected(drain);
        mbar_wait_bounded(drain, 0, abort_flag, a.wait_ns, a.err, false);
        __syncwarp();
    } else {
        // ------------------------------------------------------ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_HI));
        const int w = warp >> 2, rr = tid & (SR - 1);
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // lane field: 32 * (warp % 4) << 16
        const uint32_t ts = tmem + lanes + Z::S_COL + w * 128, to = tmem + lanes + Z::O_COL + w * DP;
        const bool neg = a.scale_log2 <= 0.0f;
        const float sc = neg ? 1.0f : a.scale_log2;  // what is left to scale behind the maximum
        uint32_t ns = 0, no = 0;
        Seen p;
        int r, place;
        bool in;
        for (Pieces k(a, rng); k.more(rng); k.next(a, rng)) {
            if (!k.same) {
                p = seen(a, k, w);
                r = k.row0 + w * SR + rr;
                in = r < k.row1;
                place = in ? k.base + a.by_GQ.div(r) : -1;
            }
            float peak = -INFINITY, l = 0.0f;  // the score that the reference follows
            for (int j = p.a; ok && j < p.b; ++j, ++ns) {
                if (!(ok = warp_wait(&sfull[w], ns & 1))) break;
                tc_fence_after();
                const int key0 = (k.kt0 + k.kt + j) * TK;
                // columns [c0, c1] are the keys this row sees
                const bool part = key0 + TK - 1 > p.lo || (a.window > 0 && key0 <= p.hi - a.window) || p.lo < 0;
                const int c1 = place - key0;
                const int c0 = a.window > 0 && place - a.window + 1 > key0 ? place - a.window + 1 - key0 : 0;
                uint32_t pk[TK / 2];
                float2 s2[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
                // The reference seldom moves: weights are taken under the one
                // there is, and again when their sum shows that one of them may
                // be past the slack (the sum is needed anyway, their maximum is
                // not: 181 us against 186 for 512 tokens after 16384).  Masked
                // tiles and an item's first know beforehand.
                bool again = true;
                float slack = SLACK;
                if (!part && !neg && j > p.a) {
                    const float ref = peak * sc - LIFT<F16>;
                    const float2 sc2 = make_float2(sc, sc), rf2 = make_float2(-ref, -ref);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t v[2][32];
                        tmem_ld32x(ts + h * 64, v[0]);
                        tmem_ld32x(ts + h * 64 + 32, v[1]);
                        tmem_wait_ld_of(v[0]);
                        tmem_wait_ld_of(v[1]);
#pragma unroll
                        for (int i = 0; i < 64; i += 2) {
                            float2 x = make_float2(__uint_as_float(v[i / 32][i % 32]), __uint_as_float(v[i / 32][i % 32 + 1]));
                            x = fma2(x, sc2, rf2);
                            x.x = ex2(x.x);
                            x.y = ex2(x.y);
                            s2[(i / 2) & 1] = add2(s2[(i / 2) & 1], x);
                            pk[h * 32 + i / 2] = pack2<F16>(x.x, x.y);
                        }
                    }
                    const float sum = (s2[0].x + s2[0].y) + (s2[1].x + s2[1].y);
                    again = __any_sync(0xffffffffu, in && (!(sum <= MOST_SUM<F16>) || !(fabsf(ref) < LARGE)));
                    slack = 0.0f;  // many weights above 1 would bring it here each time
                }
                if (again) {
                    uint32_t v[4][32];
                    s2[0] = s2[1] = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_ld32x(ts + c * 32, v[c]);
#pragma unroll
                    for (int c = 0; c < 4; ++c) tmem_wait_ld_of(v[c]);
                    if (neg) {  // the maximum is taken of scaled scores (hidden ones are -inf, not -inf * 0)
#pragma unroll
                        for (int i = 0; i < TK; ++i)
                            v[i / 32][i % 32] = __float_as_uint(__uint_as_float(v[i / 32][i % 32]) * a.scale_log2);
                    }
                    if (part) {
                        constexpr uint32_t HIDDEN = 0xFF800000u;  // -inf
#pragma unroll
                        for (int i = 0; i < TK; ++i)
                            if (i > c1) v[i / 32][i % 32] = HIDDEN;
                        if (a.window > 0) {
#pragma unroll
                            for (int i = 0; i < TK; ++i)
                                if (i < c0) v[i / 32][i % 32] = HIDDEN;
                        }
                    }
                    float m4[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) m4[c] = __uint_as_float(v[c][0]);
#pragma unroll
                    for (int i = 1; i < 31; i += 2)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            m4[c] = fmaxf(m4[c], fmaxf(__uint_as_float(v[c][i]), __uint_as_float(v[c][i + 1])));
#pragma unroll
                    for (int c = 0; c < 4; ++c) m4[c] = fmaxf(m4[c], __uint_as_float(v[c][31]));
                    const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
                    float f = 1.0f;
                    if ((mx - peak) * sc > slack) {
                        f = peak == -INFINITY ? 1.0f : ex2((peak - mx) * sc);  // nothing is summed under -inf
                        peak = mx;
                        l *= f;
                    }
                    if (j > p.a && __any_sync(0xffffffffu, f != 1.0f)) {
#pragma unroll 1
                        for (int c = 0; c < DP; c += 16) {
                            uint32_t x[16];
                            tmem_ld16x(to + c, x);
                            tmem_wait_ld_of(x);
#pragma unroll
                            for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(__uint_as_float(x[i]) * f);
                            tmem_st16(to + c, x);
                        }
                    }
                    // (the quick quotient is 0 from 2^126 on)
                    const float sw = fabsf(peak * sc) > LARGE && peak != -INFINITY
                                         ? __fdividef(LARGE, fminf(fabsf(peak), 4.0e37f))
                                         : sc;
                    const float ref = peak == -INFINITY ? 0.0f : peak * sw - LIFT<F16>;
                    const float2 sc2 = make_float2(sw, sw), rf2 = make_float2(-ref, -ref);
#pragma unroll
                    for (int i = 0; i < TK; i += 2) {
                        float2 x = make_float2(__uint_as_float(v[i / 32][i % 32]), __uint_as_float(v[i / 32][i % 32 + 1]));
                        x = fma2(x, sc2, rf2);
                        x.x = ex2(x.x);
                        x.y = ex2(x.y);
                        s2[(i / 2) & 1] = add2(s2[(i / 2) & 1], x);
                        pk[i / 2] = pack2<F16>(x.x, x.y);
                    }
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t x[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = pk[c * 32 + i];
                    tmem_st32(ts + c * 32, x);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pfull[w]);
                s2[0] = add2(s2[0], s2[1]);
                l += s2[0].x + s2[0].y;
            }
            const float m = peak * sc - LIFT<F16>;  // the reference, in powers of two
            const bool any = p.b > p.a;
            if (ok && any) {
                ok = warp_wait(&ofull[w], no & 1);
                ++no;
                tc_fence_after();
            }
            // every warp of the subtile comes here; all go on or none
            if (named_barrier_or(1 + w, SR, !ok)) {
                ok = false;
                break;
            }
            const bool rows = k.row0 + w * SR < k.row1;
            const int64_t t_row = k.t0 + (in ? a.by_GQ.div(r) : 0);
            const int h_row = k.it.head * a.GQ + (in ? r - a.by_GQ.div(r) * a.GQ : 0);
            // 64 dims of the subtile from c on: they turn through shared memory,
            // so that 8 lanes store 128 bytes of one row
            auto put = [&](int c, const float (&o)[64]) {
                if (a.ot == Q4_F32) {
                    if (in) store_dims<F16, 64>(a, t_row, h_row, c, o);
                    return;
                }
                uint8_t *st = smem + Z::OFF_O + warp * 4096;
                const int q = lane & 7, first = k.row0 + w * SR + (warp & 3) * 32;
                const int64_t o_len = static_cast<int64_t>(a.T - 1) * a.o_stride + static_cast<int64_t>(a.Hq) * a.D;
                // the last tensor copy has read the staging
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 64; i += 8)
                    *reinterpret_cast<uint4 *>(st + lane * 128 + (((i / 8) ^ (lane & 7)) << 4)) =
                        make_uint4(pack2<F16>(o[i], o[i + 1]), pack2<F16>(o[i + 2], o[i + 3]),
                                   pack2<F16>(o[i + 4], o[i + 5]), pack2<F16>(o[i + 6], o[i + 7]));
                if (maps.o_boxes && first + 32 <= k.row1) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0)
                        tma_store_3d(&maps.o, c, k.it.head * a.GQ, k.t0 + a.by_GQ.div(first), smem_u32(st));
                    return;
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int x = i * 4 + lane / 8, gr = first + x;
                    const uint4 y = *reinterpret_cast<const uint4 *>(st + x * 128 + ((q ^ (x & 7)) << 4));
                    const int t = a.by_GQ.div(gr);
                    const int64_t at = (k.t0 + t) * a.o_stride +
                                       static_cast<int64_t>(k.it.head * a.GQ + gr - t * a.GQ) * a.D + c + q * 8;
                    if (gr < k.row1 && c + q * 8 < a.D && store_ok(at + 7, o_len, a.err))
                        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.o) + at) = y;
                }
            };
            // 64 dims of the output in tensor memory
            auto sums = [&](int c, float (&o)[64]) {
                uint32_t v[2][32] = {};
                __syncwarp();
                if (any) {
                    tmem_ld32x(to + c, v[0]);
                    tmem_ld32x(to + c + 32, v[1]);
                    tmem_wait_ld_of(v[0]);
                    tmem_wait_ld_of(v[1]);
                }
#pragma unroll
                for (int i = 0; i < 64; ++i) o[i] = __uint_as_float(v[i / 32][i % 32]);
            };
            if (k.whole()) {
                const float inv = any ? inverse(l) : 0.0f;
#pragma unroll 1
                for (int c = 0; c < DP; c += 64) {
                    float o[64];
                    sums(c, o);
#pragma unroll
                    for (int i = 0; i < 64; ++i) o[i] *= inv;
                    put(c, o);
                }
                if (in) store_lse(a, t_row, h_row, m, l);
                __syncwarp();
            } else if (rows) {
                // [dim / 4][row][4], so that a warp stores and loads whole lines,
                // 16 bytes a lane
                float *ps = a.part + ((2 * static_cast<int64_t>(blockIdx.x) + (k.kt == 0)) * 2 + w) * Z::PART;
                const bool fits = store_ok(ps + Z::PART - 1 - a.part, a.part_len, a.err);
#pragma unroll 1
                for (int c = 0; c < DP; c += 64) {
                    float o[64];
                    sums(c, o);
                    if (fits && in)
#pragma unroll
                        for (int i = 0; i < 64; i += 4)
                            *reinterpret_cast<float4 *>(ps + (c + i) * SR + rr * 4) =
                                make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
                }
                if (fits) {
                    ps[DP * SR + rr] = m;
                    ps[(DP + 1) * SR + rr] = l;
                }
                int f0, f1;
                k.holders(rng, f0, f1);
                named_barrier_sync(1 + w, SR);
                if (rr == 0) {
                    const int at = 2 * f0 + w;
                    const bool last = store_ok(at, a.count_len, a.err) &&
                                      atomic_add_acq_rel_gpu(a.count + at, 1u) == static_cast<unsigned>(f1 - f0);
                    if (last) a.count[at] = 0u;
                    last_s[w] = last;
                }
                named_barrier_sync(1 + w, SR);
                if (last_s[w]) {  // whole warps: they read tensor memory
                    auto slot = [&](int f) {
                        return a.part + ((2 * static_cast<int64_t>(f) + (f == f0)) * 2 + w) * Z::PART;
                    };
                    // The row's reference and sum over the parts; the first
                    // parts' references stay in registers.
                    float m4[4];
                    auto reference = [&](int f, int row) {
                        const int i = f - f0;
                        return i == 0   ? m4[0]
                               : i == 1 ? m4[1]
                               : i == 2 ? m4[2]
                               : i == 3 ? m4[3]
                                        : __ldcg(slot(f) + DP * SR + row);
                    };
                    auto total = [&](int row, float &top, float &sum) {
                        top = -INFINITY;
                        sum = 0.0f;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            m4[i] = f0 + i <= f1 ? __ldcg(slot(f0 + i) + DP * SR + row) : -INFINITY;
#pragma unroll 4
                        for (int f = f0; f <= f1; ++f) {
                            const float mf = reference(f, row), lf = __ldcg(slot(f) + (DP + 1) * SR + row);
                            const float mn = fmaxf(top, mf), ref = mn == -INFINITY ? 0.0f : mn;
                            sum = sum * ex2(top - ref) + lf * ex2(mf - ref);
                            top = mn;
                        }
                    };
                    float top, sum;
                    if (f1 - f0 >= MANY_PARTS) {
                        // Long chains of parts come with few rows: the threads
                        // share out a row's dims when there are at most 64 or
                        // 32 rows, and four parts' loads are in flight.
                        const int nr = min(SR, k.row1 - (k.row0 + w * SR));
                        const int rp = nr <= 32 ? 32 : nr <= 64 ? 64 : 128, row = rr & (rp - 1);
                        const int dims = DP * rp / SR, d0 = rr / rp * dims;  // at least 16
                        const int gr = k.row0 + w * SR + row, t = a.by_GQ.div(gr);
                        total(row, top, sum);
                        const float ref = top == -INFINITY ? 0.0f : top, inv = inverse(sum);
                        for (int d = d0; row < nr && d < d0 + dims; d += 16) {
                            float o[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] = 0.0f;
#pragma unroll 1
                            for (int f = f0; f <= f1; f += 4) {
                                alignas(16) float y[4][16];
                                float g[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float4 *x = reinterpret_cast<const float4 *>(slot(min(f + e, f1)) + d * SR) + row;
                                    g[e] = f + e <= f1 ? reference(f + e, row) : -INFINITY;
#pragma unroll
                                    for (int i = 0; i < 4; ++i) reinterpret_cast<float4 *>(y[e])[i] = __ldcg(x + i * SR);
                                }
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float ge = ex2(g[e] - ref);
#pragma unroll
                                    for (int i = 0; i < 16; ++i) o[i] = fmaf(ge, y[e][i], o[i]);
                                }
                            }
#pragma unroll
                            for (int i = 0; i < 16; ++i) o[i] *= inv;
                            store_dims<F16, 16>(a, k.t0 + t, k.it.head * a.GQ + gr - t * a.GQ, d, o);
                        }
                        if (row < nr && d0 == 0) store_lse(a, k.t0 + t, k.it.head * a.GQ + gr - t * a.GQ, top, sum);
                    } else {
                        total(rr, top, sum);
                        const float ref = top == -INFINITY ? 0.0f : top, inv = inverse(sum);
                        // the CTA's own part is still in tensor memory
                        const int mine = static_cast<int>(blockIdx.x);
#pragma unroll 1
                        for (int d = 0; d < DP; d += 64) {
                            float o[64];
#pragma unroll
                            for (int i = 0; i < 64; ++i) o[i] = 0.0f;
#pragma unroll 1
                            for (int f = f0; f <= f1; ++f) {
                                const float4 *x = reinterpret_cast<const float4 *>(slot(f) + d * SR) + rr;
                                alignas(16) float y[64];
                                if (f != mine) {
#pragma unroll
                                    for (int i = 0; i < 16; ++i) reinterpret_cast<float4 *>(y)[i] = __ldcg(x + i * SR);
                                } else {
                                    sums(d, y);
                                }
                                const float g = ex2(reference(f, rr) - ref);
#pragma unroll
                                for (int i = 0; i < 64; ++i) o[i] = fmaf(g, y[i], o[i]);
                            }
#pragma unroll
                            for (int i = 0; i < 64; ++i) o[i] *= inv;
                            put(d, o);
                        }
                        if (in) store_lse(a, t_row, h_row, top, sum);
                    }
                }
                __syncwarp();
            }
            tc_fence_before();  // this piece's tensor-memory reads end before the next one's products
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == W_M) tmem_dealloc(tmem, 512);
}

// Tensor map of n dimensions; a dimension of extent 1 has no stride of its own.
bool encode(CUtensorMap *map, const void *base, bool f16, int n, const uint64_t *extent, const int64_t *stride,
            const uint32_t *box)
{
    const auto fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[4], bytes[3];
    cuuint32_t b[4], one[4] = {1, 1, 1, 1};
    for (int i = 0; i < n; ++i) {
        dims[i] = extent[i];
        b[i] = box[i];
        if (i > 0) bytes[i - 1] = extent[i] > 1 ? static_cast<cuuint64_t>(stride[i]) * 2 : 16;
    }
    return fn(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, n,
              const_cast<void *>(base), dims, bytes, b, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool F16, int DP>
cudaError_t launch(int grid, const AttnArgs &a, cudaStream_t s)
{
    static std::atomic<bool> done[64];
    auto kern = k_attn_tc<F16, DP>;
    const cudaError_t e = allow_smem(kern, Sizes<DP>::SMEM, done);
    if (e != cudaSuccess) return e;
    Maps m = {};
    m.kb = std::min(a.S & -a.S, TK);
    m.q_boxes = SR % a.GQ == 0;
    const auto u = [](int x) { return static_cast<uint64_t>(x); };
    const uint64_t kv_ext[4] = {u(a.D), u(a.S), u(a.Hkv), u(a.blocks)};
    const int64_t kv_str[4] = {1, a.token_stride, a.head_stride, a.block_stride};
    const uint32_t kv_box[4] = {64, static_cast<uint32_t>(m.kb), 1, 1};
    bool ok = encode(&m.k, a.k, F16, 4, kv_ext, kv_str, kv_box) && encode(&m.v, a.v, F16, 4, kv_ext, kv_str, kv_box);
    if (ok && m.q_boxes) {
        const uint64_t ext[3] = {u(a.D), u(a.Hq), u(a.T)};
        const int64_t str[3] = {1, a.D, a.q_stride};
        const uint32_t box[3] = {64, static_cast<uint32_t>(a.GQ), static_cast<uint32_t>(SR / a.GQ)};
        ok = encode(&m.q, a.q, F16, 3, ext, str, box);
    }
    // debug builds check every store, which a tensor copy's cannot be
    m.o_boxes = !kDebugBounds && a.ot != Q4_F32 && 32 % a.GQ == 0;
    if (ok && m.o_boxes) {
        const uint64_t ext[3] = {u(a.D), u(a.Hq), u(a.T)};
        const int64_t str[3] = {1, a.D, a.o_stride};
        const uint32_t box[3] = {64, static_cast<uint32_t>(a.GQ), static_cast<uint32_t>(32 / a.GQ)};
        ok = encode(&m.o, a.o, F16, 3, ext, str, box);
    }
    if (!ok) return cudaErrorInvalidValue;
    return launch_dependent(kern, dim3(grid), THREADS, Sizes<DP>::SMEM, s, m, a);
}

}  // namespace

size_t attention_tc_part_bytes(int64_t D, int grid)
{
    return static_cast<size_t>(grid) * 4 * (D > 64 ? Sizes<128>::PART : Sizes<64>::PART) * sizeof(float);
}

cudaError_t attention_tc_launch(int grid, const AttnArgs &a, bool f16, cudaStream_t s)
{
    if (a.D > 64) return f16 ? launch<true, 128>(grid, a, s) : launch<false, 128>(grid, a, s);
    return f16 ? launch<true, 64>(grid, a, s) : launch<false, 64>(grid, a, s);
}

}  // namespace q4
