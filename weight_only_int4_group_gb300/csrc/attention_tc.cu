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
//   warps 8-10      producers: queries, keys and values by cp.async into the
//                   128-byte-swizzled operand layouts (blocks of the cache
//                   are 16 keys at least, anywhere: an address per row, zeros
//                   for what lies past the request's end), a ring of four
//                   32 KB slots holding K0 V0 K1 V1 ..;
//   warp 11         allocates tensor memory; one thread issues the MMAs.
// Tensor memory (512 columns): the two subtiles' scores (128 columns each)
// and outputs (head_dim each).  While one subtile's softmax runs, the other's
// products do: the issue order is P0 V(j), Q0 K(j+1), P1 V(j), Q1 K(j+1).
// MMAs of one thread run in order, so a subtile's next scores may be issued
// right behind the product that reads the weights they overwrite, and scores
// being complete implies that every earlier product is.
//
// The running maximum is a reference that only moves when a row's maximum
// passes it by more than 2^8 (weights then stay below 256, well inside
// binary16): the output is rarely rescaled and the final division removes the
// reference, so the result is the same formula.  Keys that a tile's rows all
// see need no mask; only tiles on the diagonal or a window's edge do.
//
// Items cut by a range boundary leave their unscaled outputs, references and
// sums in the workspace; the subtile's last CTA to arrive adds them in CTA
// order.  Every barrier wait is bounded; on expiry the CTA raises the device
// error word, every role stops, copies and MMAs in flight are waited for,
// tensor memory is freed and the kernel returns.
#include "attention.cuh"
#include "tcgen05.cuh"

namespace q4 {
namespace {

constexpr int R = 256;   // rows per item
constexpr int SR = 128;  // rows per subtile
constexpr int TK = 128;  // keys per unit
constexpr int SLOTS = 4;
constexpr int W_P = 8, NP = 3;  // producers: warps 8..10
constexpr int W_M = 11;         // MMA issue
constexpr int NW = 12, THREADS = NW * 32;  // 168 registers per thread; a 13th warp would cost 40 of them
constexpr int KG = 16;          // keys that lie in one block of the cache for certain
constexpr int GPW = (TK / KG + NP - 1) / NP;  // groups of them per producer warp and tile

template <int DP>
struct Sizes {
    static constexpr int CH = DP / 64;           // 64-element chunks of a row
    static constexpr int CHUNK = 128 * 128;      // bytes of 128 rows of a chunk
    static constexpr int TILE = CH * CHUNK;      // 128 rows: a subtile's queries, a key or value tile
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_R = 2 * TILE;
    static constexpr int OFF_B = OFF_R + SLOTS * TILE;
    static constexpr int NBAR = 2 * SLOTS + 2 + 6 + 1;
    static constexpr int SMEM = OFF_B + NBAR * 8 + 32 + 1024;  // slack to align the base
    static constexpr int PART = SR * (DP + 2);  // floats of a subtile's partial result
    static constexpr uint32_t S_COL = 0, O_COL = 256;
    static_assert(O_COL + 2 * DP <= 512, "scores and outputs fit tensor memory");
    static_assert(SMEM <= 227 * 1024, "one CTA per SM");
};

// A CTA's pieces of items, walked alike by every role.
struct Piece {
    int kt, nu;        // units [kt, kt + nu) of the item
    bool whole;        // the item's only piece
    int a[2], b[2];    // units [a, b) of the piece that subtile w sees
    int lo[2], hi[2];  // places of its first and last row
};
__device__ __forceinline__ Piece piece_of(const AttnArgs &a, const Span<R, TK> &sp, int kt, int64_t left)
{
    Piece p;
    p.kt = kt;
    p.nu = static_cast<int>(min(static_cast<int64_t>(sp.units - kt), left));
    p.whole = kt == 0 && p.nu == sp.units;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        const int r0 = sp.row0 + w * SR, r1 = min(sp.row1, r0 + SR);
        p.a[w] = p.b[w] = 0;
        p.lo[w] = p.hi[w] = -1;
        if (r0 >= r1) continue;
        p.lo[w] = sp.base + r0 / a.GQ;
        p.hi[w] = sp.base + (r1 - 1) / a.GQ;
        if (p.hi[w] < 0) continue;
        const int64_t first = static_cast<int64_t>(p.lo[w]) - a.window + 1;
        const int u0 = (a.window > 0 && first > 0 ? static_cast<int>(first) : 0) / TK - sp.kt0 - kt;
        const int u1 = p.hi[w] / TK + 1 - sp.kt0 - kt;
        p.a[w] = min(max(u0, 0), p.nu);
        p.b[w] = max(p.a[w], min(u1, p.nu));
    }
    return p;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(valid ? 16 : 0)
                 : "memory");
}

template <bool F16, int DP>
__global__ void __launch_bounds__(THREADS, 1) k_attn_tc(const AttnArgs a)
{
    using Z = Sizes<DP>;
    constexpr int C8 = DP / 8;  // 16-byte pieces of a row
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    // kfull/kempty: ring slots; qfull/qempty: queries; sfull: scores ready;
    // pfull: weights stored (and the output rescaled); ofull: output complete
    uint64_t *kfull = reinterpret_cast<uint64_t *>(smem + Z::OFF_B), *kempty = kfull + SLOTS;
    uint64_t *qfull = kempty + SLOTS, *qempty = qfull + 1, *sfull = qempty + 1, *pfull = sfull + 2;
    uint64_t *ofull = pfull + 2, *drain = ofull + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    volatile int *last_s = reinterpret_cast<volatile int *>(tmem_slot + 2);  // [2]
    __shared__ LocateScratch ls;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(&kfull[i], NP * 32);
            mbar_init(&kempty[i], 1);
        }
        mbar_init(qfull, NP * 32);
        mbar_init(qempty, 1);
        for (int w = 0; w < 2; ++w) {
            mbar_init(&sfull[w], 1);
            mbar_init(&pfull[w], 4);
            mbar_init(&ofull[w], 1);
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == W_M) tmem_alloc(tmem_slot, 512);
    grid_dep_launch_dependents();
    grid_dep_wait();
    tc_fence_before();
    const Range rng = cta_range<R, TK, NW>(a, ls);  // barriers inside
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
        return mbar_wait_bounded(bar, parity, abort_flag, a.wait_ns, a.err);
    };
    // by whole warps: the lanes get one answer, also when a wait runs out
    auto warp_wait = [&](uint64_t *bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait(bar, parity)) != 0;
    };
    bool ok = true;

    if (warp >= W_P && warp < W_P + NP) {
        // ----------------------------------------------------- producers
        const int pw = warp - W_P;
        const uint32_t sq = smem_u32(smem + Z::OFF_Q), sr = smem_u32(smem + Z::OFF_R);
        // a barrier takes each lane's arrival when the lane's copies so far
        // have landed; the MMA thread fences the proxies after its wait
        auto issued = [&](uint64_t *bar) {
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
        };
        Item it = rng.first;
        int64_t u = rng.u0;
        int kt = rng.kt, n = 0;  // n: ring position
        for (int pc = 0; ok && u < rng.u1 && !a.debug_no_copy; ++pc) {
            const Span<R, TK> sp(a, it.b, it.rt);
            const Piece p = piece_of(a, sp, kt, rng.u1 - u);
            // queries: rows dealt over the warps' half-warps (16-byte pieces)
            if (pc > 0 && !warp_wait(qempty, (pc - 1) & 1)) {
                ok = false;
                break;
            }
#pragma unroll 4
            for (int e = pw * 32 + lane; e < R * C8; e += NP * 32) {
                const int row = e / C8, c = e % C8, r = sp.row0 + row;
                const bool in = r < sp.row1 && c * 8 < a.D;
                const int t = in ? r / a.GQ : 0, g = in ? r - t * a.GQ : 0;
                const uint16_t *src = in ? a.q + (sp.t0 + t) * a.q_stride +
                                               static_cast<int64_t>(it.head * a.GQ + g) * a.D + c * 8
                                         : a.q;
                const int rr = row & (SR - 1);
                cp_async16(sq + (row / SR) * Z::TILE + (c >> 3) * Z::CHUNK + rr * 128 +
                               (((c & 7) ^ (rr & 7)) << 4),
                           src, in);
            }
            issued(qfull);
            // keys and values: groups of 16 keys, each within one block of
            // the cache, dealt over the warps
            const uint16_t *kb = a.k + it.head * a.head_stride, *vb = a.v + it.head * a.head_stride;
            const int *trow = a.table + it.b * a.table_stride;
            auto block_of = [&](int j, int i) {
                const int key = (sp.kt0 + kt + j) * TK + (pw + i * NP) * KG;
                return j < p.nu && pw + i * NP < TK / KG && key < sp.kv ? __ldg(trow + key / a.S) : -1;
            };
            int blk[GPW];
#pragma unroll
            for (int i = 0; i < GPW; ++i) blk[i] = block_of(0, i);
            for (int j = 0; ok && j < p.nu; ++j) {
                const int key0 = (sp.kt0 + kt + j) * TK;
                int64_t off[GPW];  // element offset of the group's first key; -1: zeros
#pragma unroll
                for (int i = 0; i < GPW; ++i) {
                    const bool in = static_cast<unsigned>(blk[i]) < static_cast<unsigned>(a.blocks);
                    off[i] = in ? blk[i] * a.block_stride + ((key0 + (pw + i * NP) * KG) % a.S) * a.token_stride : -1;
                    blk[i] = block_of(j + 1, i);
                }
#pragma unroll 1
                for (int kv = 0; kv < 2; ++kv, ++n) {
                    const int s = n % SLOTS;
                    if (n >= SLOTS && !warp_wait(&kempty[s], (n / SLOTS - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    const uint16_t *base = kv ? vb : kb;
                    const uint32_t dst = sr + s * Z::TILE;
#pragma unroll
                    for (int i = 0; i < GPW; ++i) {
                        if (pw + i * NP >= TK / KG) break;
                        const int r0 = (pw + i * NP) * KG;
#pragma unroll
                        for (int l = 0; l < KG * C8 / 32; ++l) {
                            const int e = l * 32 + lane, row = r0 + e / C8, c = e % C8;
                            const bool v = off[i] >= 0 && key0 + row < sp.kv && c * 8 < a.D;
                            const uint16_t *src = v ? base + off[i] + (e / C8) * a.token_stride + c * 8 : base;
                            cp_async16(dst + (c >> 3) * Z::CHUNK + row * 128 + (((c & 7) ^ (row & 7)) << 4), src, v);
                        }
                    }
                    issued(&kfull[s]);
                }
            }
            u += p.nu;
            kt = 0;
            it.next(a, R);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp == W_M) {
        // ---------------------------------------------------- MMA issue
        if (lane == 0) {
            constexpr uint32_t AB = F16 ? 0u : 1u;
            const uint32_t id_qk = idesc_f16(AB, TK), id_pv = idesc_f16(AB, DP) | IDESC_B_MN;
            const uint64_t dq = sw128_desc(smem_u32(smem + Z::OFF_Q));
            const uint64_t dk = sw128_desc(smem_u32(smem + Z::OFF_R));
            const uint64_t dv = sw128_desc(smem_u32(smem + Z::OFF_R), Z::CHUNK);
            auto qk = [&](int w, int s) {
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    const int o = (k / 4) * Z::CHUNK + (k % 4) * 32;
                    mma_ss(tmem + Z::S_COL + w * 128, dq + ((w * Z::TILE + o) >> 4),
                           dk + ((s * Z::TILE + o) >> 4), id_qk, k > 0);
                }
            };
            auto pv = [&](int w, int s, bool acc) {
#pragma unroll
                for (int k = 0; k < TK / 16; ++k)
                    mma_ts(tmem + Z::O_COL + w * DP, tmem + Z::S_COL + w * 128 + k * 8,
                           dv + ((s * Z::TILE + k * 16 * 128) >> 4), id_pv, acc || k > 0);
            };
            Item it = rng.first;
            int64_t u = rng.u0;
            int kt = rng.kt, n = 0;
            uint32_t np[2] = {0, 0};  // weights consumed per subtile
            for (int pc = 0; ok && u < rng.u1; ++pc) {
                const Span<R, TK> sp(a, it.b, it.rt);
                const Piece p = piece_of(a, sp, kt, rng.u1 - u);
                if (!(ok = wait(qfull, pc & 1))) break;
                if (!(ok = wait(&kfull[n % SLOTS], (n / SLOTS) & 1))) break;
                fence_proxy_async_smem();
#pragma unroll
                for (int w = 0; w < 2; ++w)
                    if (p.a[w] == 0 && p.b[w] > 0) {
                        qk(w, n % SLOTS);
                        mma_commit(&sfull[w]);
                    }
                mma_commit(&kempty[n % SLOTS]);
                if (p.nu == 1) mma_commit(qempty);
                ++n;
                for (int j = 0; ok && j < p.nu; ++j) {
                    const int sv = n % SLOTS, sk = (n + 1) % SLOTS;
                    const bool more = j + 1 < p.nu;
                    if (!(ok = wait(&kfull[sv], (n / SLOTS) & 1))) break;
                    fence_proxy_async_smem();
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        if (j >= p.a[w] && j < p.b[w]) {
                            if (!(ok = wait(&pfull[w], np[w] & 1))) break;
                            ++np[w];
                            tc_fence_after();
                            pv(w, sv, j > p.a[w]);
                            if (j == p.b[w] - 1) mma_commit(&ofull[w]);
                        }
                        if (more) {
                            if (w == 0) {
                                if (!(ok = wait(&kfull[sk], ((n + 1) / SLOTS) & 1))) break;
                                fence_proxy_async_smem();
                            }
                            if (j + 1 >= p.a[w] && j + 1 < p.b[w]) {
                                qk(w, sk);
                                mma_commit(&sfull[w]);
                            }
                        }
                    }
                    if (!ok) break;
                    mma_commit(&kempty[sv]);
                    if (more) {
                        mma_commit(&kempty[sk]);
                        if (j + 2 == p.nu) mma_commit(qempty);
                    }
                    n += more ? 2 : 1;
                }
                u += p.nu;
                kt = 0;
                it.next(a, R);
            }
            // MMAs in flight end before tensor memory is freed
            mma_commit(drain);
            mbar_wait_bounded(drain, 0, abort_flag, a.wait_ns, a.err, false);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------ softmax
        const int w = warp >> 2, rr = tid & (SR - 1);
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // lane field: 32 * (warp % 4) << 16
        const uint32_t ts = tmem + lanes + Z::S_COL + w * 128, to = tmem + lanes + Z::O_COL + w * DP;
        const bool neg = a.scale_log2 < 0.0f;
        Item it = rng.first;
        int64_t u = rng.u0;
        int kt = rng.kt;
        uint32_t ns = 0, no = 0;
        while (u < rng.u1) {
            const Span<R, TK> sp(a, it.b, it.rt);
            const Piece p = piece_of(a, sp, kt, rng.u1 - u);
            const int r = sp.row0 + w * SR + rr;
            const bool in = r < sp.row1;
            const int place = in ? sp.base + r / a.GQ : -1;
            float m = -INFINITY, l = 0.0f;
            for (int j = p.a[w]; ok && j < p.b[w]; ++j, ++ns) {
                if (!(ok = warp_wait(&sfull[w], ns & 1))) break;
                tc_fence_after();
                const int key0 = (sp.kt0 + kt + j) * TK;
                // columns [c0, c1] are the keys this row sees
                const bool part = key0 + TK - 1 > p.lo[w] ||
                                  (a.window > 0 && key0 <= p.hi[w] - a.window) || p.lo[w] < 0;
                const int c1 = place - key0;
                const int c0 = a.window > 0 && place - a.window + 1 > key0 ? place - a.window + 1 - key0 : 0;
                float mx = -INFINITY;
                uint32_t v[32];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    tmem_ld32x(ts + c * 32, v);
                    tmem_wait_ld();
                    if (part || neg) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float x = __uint_as_float(v[i]) * a.scale_log2;
                            if (c * 32 + i >= c0 && c * 32 + i <= c1) mx = fmaxf(mx, x);
                        }
                    } else {
                        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int i = 0; i < 32; ++i) m4[i & 3] = fmaxf(m4[i & 3], __uint_as_float(v[i]));
                        mx = fmaxf(mx, fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])));
                    }
                }
                if (!(part || neg)) mx *= a.scale_log2;
                bool move = false;
                float f = 1.0f;
                if (m == -INFINITY) {
                    m = mx;
                } else if (mx > m + 8.0f) {
                    f = ex2(m - mx);
                    m = mx;
                    l *= f;
                    move = true;
                }
                if (__any_sync(0xffffffffu, move) && j > p.a[w]) {
#pragma unroll
                    for (int c = 0; c < DP / 32; ++c) {
                        tmem_ld32x(to + c * 32, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
                        tmem_st32(to + c * 32, v);
                    }
                }
                const float ref = m == -INFINITY ? 0.0f : m;
                float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    tmem_ld32x(ts + c * 32, v);
                    tmem_wait_ld();
                    uint32_t pk[16];
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float x = fmaf(__uint_as_float(v[i]), a.scale_log2, -ref);
                        float y = fmaf(__uint_as_float(v[i + 1]), a.scale_log2, -ref);
                        if (part) {
                            if (c * 32 + i < c0 || c * 32 + i > c1) x = -INFINITY;
                            if (c * 32 + i + 1 < c0 || c * 32 + i + 1 > c1) y = -INFINITY;
                        }
                        x = ex2(x);
                        y = ex2(y);
                        s4[i & 2] += x;
                        s4[(i & 2) + 1] += y;
                        pk[i / 2] = pack2<F16>(x, y);
                    }
                    tmem_st16(ts + c * 16, pk);
                }
                l += (s4[0] + s4[1]) + (s4[2] + s4[3]);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&pfull[w]);
            }
            const bool any = p.b[w] > p.a[w];
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
            const bool rows = sp.row0 + w * SR < sp.row1;
            const int64_t t_row = sp.t0 + (in ? r / a.GQ : 0);
            const int h_row = it.head * a.GQ + (in ? r % a.GQ : 0);
            if (p.whole) {
                uint32_t v[32];
                const float inv = inverse(l);
#pragma unroll
                for (int c = 0; c < DP / 32; ++c) {
                    __syncwarp();
                    if (any) {
                        tmem_ld32x(to + c * 32, v);
                        tmem_wait_ld();
                    }
                    if (in) {
                        float o[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = any ? __uint_as_float(v[i]) * inv : 0.0f;
                        store_dims<F16, 32>(a, t_row, h_row, c * 32, o);
                    }
                }
                if (in) store_lse(a, t_row, h_row, m, l);
                __syncwarp();
            } else if (rows) {
                // [dim][row], so that a warp's stores and loads are whole lines
                float *ps = a.part + ((2 * static_cast<int64_t>(blockIdx.x) + (kt == 0)) * 2 + w) * Z::PART;
                const bool fits = store_ok(ps + Z::PART - 1 - a.part, a.part_len, a.err);
                uint32_t v[32];
#pragma unroll
                for (int c = 0; c < DP / 32; ++c) {
                    if (any) {
                        tmem_ld32x(to + c * 32, v);
                        tmem_wait_ld();
                    }
                    if (fits)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            ps[(c * 32 + i) * SR + rr] = any ? __uint_as_float(v[i]) : 0.0f;
                }
                if (fits) {
                    ps[DP * SR + rr] = m;
                    ps[(DP + 1) * SR + rr] = l;
                }
                const int64_t i0 = u - kt, i1 = i0 + sp.units;
                const int f0 = owner_of(i0, rng.total, rng.G), f1 = owner_of(i1 - 1, rng.total, rng.G);
                named_barrier_sync(1 + w, SR);
                if (rr == 0) {
                    const int at = 2 * f0 + w;
                    const bool last = store_ok(at, a.count_len, a.err) &&
                                      atomic_add_acq_rel_gpu(a.count + at, 1u) == static_cast<unsigned>(f1 - f0);
                    if (last) a.count[at] = 0u;
                    last_s[w] = last;
                }
                named_barrier_sync(1 + w, SR);
                if (last_s[w] && in) {
                    auto slot = [&](int f) {
                        return a.part + ((2 * static_cast<int64_t>(f) + (f == f0)) * 2 + w) * Z::PART + rr;
                    };
                    float top = -INFINITY, sum = 0.0f;
                    for (int f = f0; f <= f1; ++f) top = fmaxf(top, __ldcg(slot(f) + DP * SR));
                    const float ref = top == -INFINITY ? 0.0f : top;
#pragma unroll 1
                    for (int d = 0; d < DP; d += 32) {
                        float o[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = 0.0f;
                        sum = 0.0f;
#pragma unroll 1
                        for (int f = f0; f <= f1; ++f) {
                            const float *x = slot(f);
                            float y[32];
#pragma unroll
                            for (int i = 0; i < 32; ++i) y[i] = __ldcg(x + (d + i) * SR);
                            const float g = ex2(__ldcg(x + DP * SR) - ref);
                            sum += g * __ldcg(x + (DP + 1) * SR);
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] += g * y[i];
                        }
                        const float inv = inverse(sum);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] *= inv;
                        store_dims<F16, 32>(a, t_row, h_row, d, o);
                    }
                    store_lse(a, t_row, h_row, top, sum);
                }
                __syncwarp();
            }
            tc_fence_before();  // this piece's tensor-memory reads end before the next one's products
            u += p.nu;
            kt = 0;
            it.next(a, R);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == W_M) tmem_dealloc(tmem, 512);
}

template <bool F16, int DP>
cudaError_t launch(int grid, const AttnArgs &a, cudaStream_t s)
{
    static std::atomic<bool> done[64];
    auto kern = k_attn_tc<F16, DP>;
    const cudaError_t e = allow_smem(kern, Sizes<DP>::SMEM, done);
    if (e != cudaSuccess) return e;
    return launch_dependent(kern, dim3(grid), THREADS, Sizes<DP>::SMEM, s, a);
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
