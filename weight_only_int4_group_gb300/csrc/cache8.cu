// cache8.cu -- the KV cache in 8 bits: the rotary append that quantises as it
// writes, and reading tokens back.
#include "cache8.cuh"

namespace q4 {

// ------------------------------------------------ rotary append, quantising
// Memory-bound: qkv is read once, the queries are written in 16 bits and the
// keys and values in 8.  What couples tokens is the scale of a block: the run
// of new tokens in one block is looked at twice, for its largest magnitude and
// to be quantised; the second look finds it in the first-level cache.
//
// A CTA takes a chunk of `rows` token rows and some heads of one kind: queries
// (rotated and stored), keys, or values.  For keys and values it owns the runs
// that begin in its chunk, to their ends (a run is at most a block), so that no
// two CTAs meet in a block.  A thread holds 8 elements of a row; their
// angles serve all its heads.  Fractions of a turn are 64-bit integers
// (position * frequency mod 1 in units of 2^-64): this card's f64 units would
// take longer than the copy.
namespace {

constexpr int MOST_ROWS = 64;    // of a chunk
constexpr int MOST_HEADS = 16;   // of a CTA
constexpr int AHEAD = 2;         // heads whose loads are in flight in a thread

// The pair partner's factors: y = x * c + partner * s.
struct Turn {
    float c[8], s[8];
};

template <bool INTER>
__device__ __forceinline__ void angles(const Append8Args &a, const uint64_t *freq, int row, int d0, Turn &t)
{
    const int half = a.rot / 2;
    const uint64_t pos = static_cast<uint64_t>(static_cast<int64_t>(d0 < a.rot ? a.position[row] : 0));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int d = d0 + i;
        if (INTER && (i & 1)) {
            t.c[i] = t.c[i - 1];
            t.s[i] = -t.s[i - 1];
            continue;
        }
        if (d >= a.rot) {
            t.c[i] = 1.0f;
            t.s[i] = 0.0f;
            continue;
        }
        const bool first = INTER || d < half;
        const uint64_t x = pos * freq[INTER ? d / 2 : first ? d : d - half];
        float sn, cs;
        // +-1/2 turn in units of 2^-32
        sincospif(static_cast<float>(static_cast<int32_t>(x >> 32)) * 4.656612873077393e-10f, &sn, &cs);
        t.c[i] = cs * a.factor;
        t.s[i] = (first ? -sn : sn) * a.factor;
    }
}

__device__ __forceinline__ uint32_t half_of(const uint4 &v, int i)
{
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return (w >> (16 * (i & 1))) & 0xFFFFu;
}

// Elements d0 .. d0 + 7 of a head at x and their pair partners, and what the
// rotation makes of them.  `vec`: the partners are 8 aligned elements too.
struct Raw {
    uint4 v, p;
};

template <bool INTER>
__device__ __forceinline__ Raw load_raw(const uint16_t *x, int d0, int rot, bool vec)
{
    Raw r;
    r.v = *reinterpret_cast<const uint4 *>(x + d0);
    r.p = make_uint4(0, 0, 0, 0);
    if (INTER || d0 >= rot) return r;
    const int half = rot / 2;
    if (vec) {
        r.p = *reinterpret_cast<const uint4 *>(x + (d0 < half ? d0 + half : d0 - half));
        return r;
    }
    uint32_t w[4] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int d = d0 + i;
        if (d < rot) w[i / 2] |= static_cast<uint32_t>(x[d < half ? d + half : d - half]) << (16 * (i & 1));
    }
    r.p = make_uint4(w[0], w[1], w[2], w[3]);
    return r;
}

template <bool F16, bool INTER>
__device__ __forceinline__ void rotate(const Raw &r, int d0, int rot, const Turn &t, float (&y)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x = bits_to_f32<F16>(half_of(r.v, i)), p = bits_to_f32<F16>(half_of(INTER ? r.v : r.p, INTER ? i ^ 1 : i));
        y[i] = d0 + i < rot ? x * t.c[i] + p * t.s[i] : x;
    }
}

template <bool F16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi)
{
    if (F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Whether token row t begins a run: it has no predecessor in its block.  Rows
// without a slot in the cache stand alone.
__device__ __forceinline__ bool begins(const int64_t *slot, int64_t slots, int S, int t)
{
    const int64_t s = slot[t];
    if (t == 0 || s < 0 || s >= slots || slot[t - 1] != s - 1) return true;
    return s % S == 0;
}

struct AppendGrid {
    int rows, lanes_log;  // token rows of a chunk; threads of a row, log 2
    int gk, nk, gq;       // heads per CTA and CTAs for keys (and for values); heads per CTA for queries
};

template <int CODE, bool F16, bool INTER>
__global__ void __launch_bounds__(1024) k_append8(const Append8Args a, const AppendGrid g)
{
    using X = Exponents<CODE, F16>;
    __shared__ uint64_t freq[64];
    __shared__ unsigned starts[2];                   // rows of the chunk that begin a run
    __shared__ int end_row;                          // behind the last run
    __shared__ uint32_t peak[MOST_HEADS][MOST_ROWS]; // of the run that begins at a row
    __shared__ int8_t scale[MOST_HEADS][MOST_ROWS], growth[MOST_HEADS][MOST_ROWS];
    const int tid = threadIdx.x, S = a.c.S, D = a.c.D;
    const int d0 = (tid & ((1 << g.lanes_log) - 1)) * 8, i = tid >> g.lanes_log;
    const int c0 = blockIdx.x * g.rows, rows = min(g.rows, a.T - c0);
    const int part = blockIdx.y;
    const bool keys = part < g.nk, queries = part >= 2 * g.nk;
    const bool vec = a.rot / 2 % 8 == 0;
    const int rot = keys || queries ? a.rot : 0;

    grid_dep_wait();
    grid_dep_launch_dependents();
    if (tid < rot / 2) {
        const double turns = a.freq[tid] * 0.15915494309189535;
        freq[tid] = __double2ull_rz((turns - floor(turns)) * 18446744073709551616.0);
    }
    if (queries) {
        __syncthreads();
        if (i >= rows || d0 >= D) return;
        const int row = c0 + i, h0 = (part - 2 * g.nk) * g.gq, h1 = min(h0 + g.gq, a.Hq);
        Turn t;
        angles<INTER>(a, freq, row, d0, t);
        const uint16_t *x = a.qkv + row * a.qkv_stride;
        const int64_t at = row * a.q_stride + d0, len = (a.T - 1) * a.q_stride + static_cast<int64_t>(a.Hq) * D;
        for (int h = h0; h < h1; h += AHEAD) {
            Raw raw[AHEAD];
#pragma unroll
            for (int n = 0; n < AHEAD; ++n)
                if (h + n < h1) raw[n] = load_raw<INTER>(x + (h + n) * D, d0, rot, vec);
            __syncwarp();  // q_out may be qkv: a head's lanes have read it before one writes
#pragma unroll
            for (int n = 0; n < AHEAD; ++n) {
                float y[8];
                rotate<F16, INTER>(raw[n], d0, rot, t, y);
                if (h + n < h1 && store_ok(at + (h + n) * D + 7, len, a.err))
                    *reinterpret_cast<uint4 *>(a.q_out + at + (h + n) * D) =
                        make_uint4(pack16<F16>(y[0], y[1]), pack16<F16>(y[2], y[3]), pack16<F16>(y[4], y[5]),
                                   pack16<F16>(y[6], y[7]));
            }
        }
        return;
    }

    // ---- keys or values: the runs
    const int h0 = (keys ? part : part - g.nk) * g.gk, nh = min(g.gk, a.c.heads - h0);
    uint8_t *codes = keys ? a.c.k : a.c.v, *exps = keys ? a.c.k_exp : a.c.v_exp;
    const int64_t slots = static_cast<int64_t>(a.c.blocks) * S;
    const int64_t codes_len = (a.c.blocks - 1) * a.c.block_stride + (a.c.heads - 1) * a.c.head_stride +
                              (S - 1) * a.c.token_stride + D;
    const uint16_t *qkv = a.qkv + static_cast<int64_t>(a.Hq + (keys ? 0 : a.c.heads) + h0) * D;
    if (tid == 0) end_row = min(c0 + rows + S, a.T);
    if (tid < 64) {
        const unsigned m = __ballot_sync(0xffffffffu, tid < rows && begins(a.slot, slots, S, c0 + tid));
        if ((tid & 31) == 0) starts[tid >> 5] = m;
    }
    for (int n = tid; n < nh * MOST_ROWS; n += blockDim.x) peak[n / MOST_ROWS][n % MOST_ROWS] = 0u;
    __syncthreads();
    const uint64_t mask = starts[0] | static_cast<uint64_t>(starts[1]) << 32;
    if (!mask) return;
    for (int t = c0 + rows + tid; t < min(c0 + rows + S, a.T); t += blockDim.x)
        if (begins(a.slot, slots, S, t)) atomicMin(&end_row, t);
    __syncthreads();
    const int end = end_row;
    // of a row: the chunk's row that its run begins at (-1: another chunk's), and its place
    struct Row {
        int lead;
        int64_t slot;
    };
    auto row_of = [&](int row) {
        Row r = {-1, -1};
        if (row >= end) return r;
        const uint64_t upto = row - c0 >= 63 ? mask : mask & ((2ull << (row - c0)) - 1);
        if (!upto) return r;
        r.slot = a.slot[row];
        if (r.slot < 0 || r.slot >= slots) return r;
        r.lead = 63 - __clzll(static_cast<long long>(upto));
        return r;
    };
    // ---- largest magnitudes
    for (int r0 = c0; r0 < end; r0 += g.rows) {
        const Row r = row_of(r0 + i);
        const bool on = r.lead >= 0 && d0 < D;
        Turn t;
        if (on) angles<INTER>(a, freq, r0 + i, keys ? d0 : 128, t);
        for (int h = 0; h < nh; h += AHEAD) {
            Raw raw[AHEAD];
#pragma unroll
            for (int n = 0; n < AHEAD; ++n)
                if (on && h + n < nh) raw[n] = load_raw<INTER>(qkv + (r0 + i) * a.qkv_stride + (h + n) * D, d0, rot, vec);
#pragma unroll
            for (int n = 0; n < AHEAD; ++n) {
                if (h + n >= nh) break;
                float m = 0.0f;
                if (on) {
                    float y[8];
                    rotate<F16, INTER>(raw[n], d0, rot, t, y);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float v = fabsf(y[e]);
                        m = v <= 3.4028234664e38f ? fmaxf(m, v) : m;  // infinities and NaN do not count
                    }
                }
                for (int d = 1 << g.lanes_log >> 1; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                if (r.lead >= 0 && d0 == 0) atomicMax(&peak[h + n][r.lead], __float_as_uint(m));
            }
        }
    }
    __syncthreads();
    // ---- the runs' scales
    for (int n = tid; n < nh * g.rows; n += blockDim.x) {
        const int h = n / g.rows, lead = n - h * g.rows;
        if (!(mask >> lead & 1)) continue;
        growth[h][lead] = 0;
        const int64_t slot = a.slot[c0 + lead];
        if (slot < 0 || slot >= slots) continue;
        const int64_t blk = slot / S;
        uint8_t *at = exps + blk * a.c.heads + h0 + h;
        int e = needed<CODE, F16>(peak[h][lead]);
        if (slot != blk * S) {
            const int old = X::of(*at);
            if (e > old)
                growth[h][lead] = static_cast<int8_t>(min(e - old, 127));
            else
                e = old;
        }
        scale[h][lead] = static_cast<int8_t>(e);
        if (store_ok(at - exps, static_cast<int64_t>(a.c.blocks) * a.c.heads, a.err)) *at = static_cast<uint8_t>(e + 127);
    }
    __syncthreads();
    // ---- the new codes
    for (int r0 = c0; r0 < end; r0 += g.rows) {
        const Row r = row_of(r0 + i);
        if (r.lead < 0 || d0 >= D) continue;
        Turn t;
        angles<INTER>(a, freq, r0 + i, keys ? d0 : 128, t);
        const int64_t blk = r.slot / S;
        const int64_t at = blk * a.c.block_stride + (r.slot - blk * S) * a.c.token_stride + h0 * a.c.head_stride + d0;
        for (int h = 0; h < nh; h += AHEAD) {
            Raw raw[AHEAD];
#pragma unroll
            for (int n = 0; n < AHEAD; ++n)
                if (h + n < nh) raw[n] = load_raw<INTER>(qkv + (r0 + i) * a.qkv_stride + (h + n) * D, d0, rot, vec);
#pragma unroll
            for (int n = 0; n < AHEAD; ++n) {
                if (h + n >= nh) break;
                float y[8];
                rotate<F16, INTER>(raw[n], d0, rot, t, y);
                const float inv = pow2(-scale[h + n][r.lead]);
                const float lo[4] = {y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv};
                const float hi[4] = {y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv};
                const int64_t to = at + (h + n) * a.c.head_stride;
                if (store_ok(to + 7, codes_len, a.err))
                    *reinterpret_cast<uint2 *>(codes + to) = make_uint2(f32_to_codes<CODE>(lo), f32_to_codes<CODE>(hi));
            }
        }
    }
    // ---- codes held already, where the scale grew: a warp per run and head
    const int warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5, pieces = D / 16;
    for (int n = warp; n < nh * g.rows; n += warps) {
        const int h = n / g.rows, lead = n - h * g.rows;
        if (!(mask >> lead & 1) || growth[h][lead] == 0) continue;
        const int64_t slot = a.slot[c0 + lead], blk = slot / S;
        const float f = pow2(-min(static_cast<int>(growth[h][lead]), 126));
        const int64_t base = blk * a.c.block_stride + (h0 + h) * a.c.head_stride;
        for (int u = lane; u < static_cast<int>(slot - blk * S) * pieces; u += 32) {
            const int64_t at = base + u / pieces * a.c.token_stride + u % pieces * 16;
            uint4 v = *reinterpret_cast<const uint4 *>(codes + at);
            uint32_t *w = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float x[4];
                codes_to_f32<CODE>(w[e], x);
#pragma unroll
                for (int b = 0; b < 4; ++b) x[b] *= f;
                w[e] = f32_to_codes<CODE>(x);
            }
            if (store_ok(at + 15, codes_len, a.err)) *reinterpret_cast<uint4 *>(codes + at) = v;
        }
    }
}

template <int CODE, bool F16>
cudaError_t append_launch(const Append8Args &a, bool interleaved, int sm_count, cudaStream_t s)
{
    AppendGrid g{};
    g.lanes_log = a.c.D > 64 ? 4 : 3;
    g.rows = a.c.S >= 64 ? 64 : a.c.S >= 32 ? 32 : 16;
    const int chunks = ctas_for(a.T, g.rows);
    // heads per CTA: fewer where there are few chunks
    g.gk = std::min({std::max(1, static_cast<int>(static_cast<int64_t>(chunks) * 2 * a.c.heads / (4 * sm_count))), a.c.heads, 8});
    g.nk = ctas_for(a.c.heads, g.gk);
    g.gq = std::min({std::max(1, static_cast<int>(static_cast<int64_t>(chunks) * a.Hq / (4 * sm_count))), a.Hq, 16});
    const dim3 grid(chunks, 2 * g.nk + ctas_for(a.Hq, g.gq));
    const int threads = g.rows << g.lanes_log;
    return interleaved ? launch_dependent(k_append8<CODE, F16, true>, grid, threads, 0, s, a, g)
                       : launch_dependent(k_append8<CODE, F16, false>, grid, threads, 0, s, a, g);
}

// -------------------------------------------------------------- reading back
// Memory-bound: a byte in, two (or four) out.  A CTA takes 32 token rows, finds
// their requests (one warp), and each thread widens 16 codes at a time.
constexpr int READ_ROWS = 32, READ_THREADS = 256;

template <int CODE, bool F16, bool F32>
__global__ void __launch_bounds__(READ_THREADS) k_read8(const Read8Args a)
{
    __shared__ int64_t place[READ_ROWS];  // of a row's token in the codes; -1: zeros, -2: no request
    __shared__ int block[READ_ROWS];
    const int tid = threadIdx.x, t0 = blockIdx.x * READ_ROWS, rows = min(READ_ROWS, a.T - t0);
    grid_dep_wait();
    grid_dep_launch_dependents();
    if (tid < 32) {
        const int b0 = request_of(a.q_start, a.B, t0);
        const int t = min(t0 + tid, a.T - 1), next = a.q_start[min(b0 + 1 + tid, a.B)];
        // starts at or before the row; past the last request's the rows are nobody's
        int b = b0;
#pragma unroll
        for (int n = 0; n < 32; ++n) b += b0 + 1 + n <= a.B && __shfl_sync(0xffffffffu, next, n) <= t;
        if (b == b0 + 32)
            while (b < a.B && a.q_start[b + 1] <= t) ++b;
        int64_t at = -2;
        int blk = 0;
        if (b < a.B) {
            const int first = max(a.q_start[b], 0), last = min(max(a.q_start[b + 1], 0), a.T);
            if (t >= first && t < last) {
                const int kv = static_cast<int>(min(static_cast<int64_t>(max(a.kv_len[b], 0)), static_cast<int64_t>(a.width) * a.c.S));
                const int p = kv - (last - t);
                at = -1;
                if (p >= 0) {
                    const int j = a.c.by_S.div(p);
                    blk = a.table[b * a.table_stride + j];
                    if (static_cast<unsigned>(blk) < static_cast<unsigned>(a.c.blocks))
                        at = blk * a.c.block_stride + (p - j * a.c.S) * a.c.token_stride;
                    else
                        blk = 0;
                }
            }
        }
        place[tid] = at;
        block[tid] = blk;
    }
    __syncthreads();
    const int pieces = a.c.D / 16, per = a.c.heads * pieces;  // 16-code pieces of a row's keys
    for (int n = tid; n < rows * 2 * per; n += READ_THREADS) {
        const int r = n / (2 * per), u = n - r * 2 * per;
        const int64_t at = place[r];
        if (at == -2) continue;
        const bool vals = u >= per;
        const int w = vals ? u - per : u, h = w / pieces, c = w - h * pieces;
        uint4 v = make_uint4(0, 0, 0, 0);
        float f = 1.0f;
        if (at >= 0) {
            v = __ldcs(reinterpret_cast<const uint4 *>((vals ? a.c.v : a.c.k) + at + h * a.c.head_stride + c * 16));
            f = pow2(Exponents<CODE, F16>::of((vals ? a.c.v_exp : a.c.k_exp)[static_cast<int64_t>(block[r]) * a.c.heads + h]));
        }
        const int64_t stride = vals ? a.v_stride : a.k_stride, to = (t0 + r) * stride + w * 16;
        if (!store_ok(to + 15, (a.T - 1) * stride + static_cast<int64_t>(a.c.heads) * a.c.D, a.err)) continue;
        void *out = vals ? a.v_out : a.k_out;
        const uint32_t words[4] = {v.x, v.y, v.z, v.w};
        float x[4][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            codes_to_f32<CODE>(words[e], x[e]);
#pragma unroll
            for (int b = 0; b < 4; ++b) x[e][b] *= f;
        }
        if (F32) {
            float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(out) + to);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = make_float4(x[e][0], x[e][1], x[e][2], x[e][3]);
        } else {
            uint4 *o = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + to);
#pragma unroll
            for (int e = 0; e < 2; ++e)
                o[e] = make_uint4(pack16<F16>(x[2 * e][0], x[2 * e][1]), pack16<F16>(x[2 * e][2], x[2 * e][3]),
                                  pack16<F16>(x[2 * e + 1][0], x[2 * e + 1][1]), pack16<F16>(x[2 * e + 1][2], x[2 * e + 1][3]));
        }
    }
}

template <int CODE, bool F16>
cudaError_t read_launch(const Read8Args &a, bool f32_out, cudaStream_t s)
{
    const dim3 grid(ctas_for(a.T, READ_ROWS));
    return f32_out ? launch_dependent(k_read8<CODE, F16, true>, grid, READ_THREADS, 0, s, a)
                   : launch_dependent(k_read8<CODE, F16, false>, grid, READ_THREADS, 0, s, a);
}

}  // namespace

cudaError_t append8_launch(const Append8Args &a, q4_code code, bool f16, bool interleaved, int sm_count, cudaStream_t s)
{
    if (code == Q4_I8) return f16 ? append_launch<I8, true>(a, interleaved, sm_count, s) : append_launch<I8, false>(a, interleaved, sm_count, s);
    return f16 ? append_launch<E4M3, true>(a, interleaved, sm_count, s) : append_launch<E4M3, false>(a, interleaved, sm_count, s);
}

cudaError_t read8_launch(const Read8Args &a, q4_code code, bool f16, bool f32_out, cudaStream_t s)
{
    if (code == Q4_I8) return f16 ? read_launch<I8, true>(a, f32_out, s) : read_launch<I8, false>(a, f32_out, s);
    return f16 ? read_launch<E4M3, true>(a, f32_out, s) : read_launch<E4M3, false>(a, f32_out, s);
}

}  // namespace q4
