// cache8.cu -- the KV cache in 8 bits: the rotary append that quantises as it
// writes, and reading tokens back.
#include "cache8.cuh"

namespace q4 {

// ------------------------------------------------ rotary append, quantising
// Memory-bound: qkv is read once, the queries are written in 16 bits and the
// keys and values in 8.  What couples tokens is the scale of a block: the run
// of new tokens in one block is looked at twice, for its largest magnitude and
// to be quantised; the second look finds it in a cache, or, where one head is all
// that a CTA has of a run within its chunk, in registers.
//
// A CTA takes a chunk of 32 token rows and some heads of one kind: queries
// (rotated and stored), keys, or values.  For keys and values it owns the runs
// that begin in its chunk, to their ends (a run is at most a block), so that no
// two CTAs meet in a block.  A thread holds 16 elements of a row: two
// 8-element loads that the rotation pairs (or that lie side by side), whose
// angles serve all its heads.  Fractions of a turn are 64-bit integers
// (position * frequency mod 1 in units of 2^-64): this card's f64 units would
// take longer than the copy.
//
// Measured (graph): 8192 rows of 64 + 2 * 8 heads of 128 in 68 us, 4.7 TB/s (0.69 of
// the measured copy bandwidth: the CTAs' beginnings and the second look are waits
// that four CTAs per SM do not hide; three with twice the loads in flight took 74);
// 1001 rows of 32 + 2 * 32 heads 20 us; 512 decoding requests 7 us, 4 of them 4.9,
// which is latency.  A loop of two looks per head, which reads each row once,
// waits at two barriers per head: 91 and 46 us.
namespace {

constexpr int ROWS = 32;         // of a chunk
constexpr int MOST_HEADS = 8;    // of a CTA, keys or values
constexpr int AHEAD = 1;         // heads whose loads are in flight in a thread

// How a thread's elements are paired: its two vectors with each other; within
// each, neighbours; or each with one somewhere (rot not a multiple of 16).
enum Pairs { HALF, NEXT, ANY };

// freq / (2 pi) mod 1 in units of 2^-64: the 53-bit mantissa times 2^64 / (2 pi),
// shifted by the exponent (0 for what is not finite).
__device__ __forceinline__ uint64_t turns_of(double freq)
{
    const uint64_t b = static_cast<uint64_t>(__double_as_longlong(freq));
    const int field = static_cast<int>(b >> 52) & 0x7FF;
    if (field == 0x7FF) return 0;
    const uint64_t m = (b & ((1ull << 52) - 1)) | (field ? 1ull << 52 : 0);
    constexpr uint64_t per = 2935890503282001226ull;
    const uint64_t hi = __umul64hi(m, per), lo = m * per;
    const int s = 52 + 1023 - max(field, 1);  // m * per >> s
    uint64_t f = 0;
    if (s <= 0)
        f = s > -64 ? lo << -s : 0;
    else if (s < 64)
        f = lo >> s | hi << (64 - s);
    else if (s < 128)
        f = hi >> (s - 64);
    return b >> 63 ? ~f + 1 : f;
}

// Cosine and sine, times the factor, of pair p's angle.
__device__ __forceinline__ float2 turn_of(const Append8Args &a, const uint64_t *freq, int64_t pos, int p)
{
    // The turn's quarter by rounding, what is left as +-1/8 turn in units of 2^-32,
    // pi / 4 at most: there the Taylor polynomials end within 2e-9 (sine, to the
    // 9th power) and 2e-10 (cosine, to the 10th).
    const uint32_t x = static_cast<uint32_t>(static_cast<uint64_t>(pos) * freq[p] >> 32);
    const uint32_t quarter = (x + 0x20000000u) >> 30;
    const float r = static_cast<float>(static_cast<int32_t>(x - (quarter << 30))) * 1.4629180792671596e-9f;  // 2 pi 2^-32
    const float q = r * r;
    const float sn = fmaf(r * q, fmaf(q, fmaf(q, fmaf(q, 1.0f / 362880, -1.0f / 5040), 1.0f / 120), -1.0f / 6), r);
    const float cs = fmaf(q, fmaf(q, fmaf(q, fmaf(q, fmaf(q, -1.0f / 3628800, 1.0f / 40320), -1.0f / 720), 1.0f / 24), -0.5f), 1.0f);
    const float c = quarter & 1 ? sn : cs, s = quarter & 1 ? cs : sn;
    return make_float2((quarter + 1) & 2 ? -c * a.factor : c * a.factor, quarter & 2 ? -s * a.factor : s * a.factor);
}

__device__ __forceinline__ uint32_t half_of(const uint4 &v, int i)
{
    const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
    return (w >> (16 * (i & 1))) & 0xFFFFu;
}

// A thread's 16 elements: 8 from e[0] on and 8 from e[1] on, which are rotated
// (`turns`) or not.
struct Place {
    int e[2];
    bool in, turns;
};
template <Pairs P>
__device__ __forceinline__ Place place_of(int u, int D, int rot)
{
    Place p;
    p.in = u * 16 < D;
    const int pairs = rot / 16;
    p.turns = P == HALF ? u < pairs : u * 16 < rot;
    p.e[0] = P == HALF && p.turns ? u * 8 : u * 16;
    p.e[1] = P == HALF && p.turns ? rot / 2 + u * 8 : u * 16 + 8;
    return p;
}

struct Raw {
    uint4 v[2];
};
__device__ __forceinline__ Raw load_raw(const uint16_t *x, const Place &p)
{
    Raw r;
    r.v[0] = *reinterpret_cast<const uint4 *>(x + p.e[0]);
    r.v[1] = *reinterpret_cast<const uint4 *>(x + p.e[1]);
    return r;
}

// The elements of a head at x, rotated: t holds the angles of 8 pairs (ANY: they
// are made here, and partners come from memory: `part` is the head as it was).
template <Pairs P, bool F16>
__device__ __forceinline__ void rotate(const Append8Args &a, const uint64_t *freq, int64_t pos, const uint16_t *part, const Raw &r,
                                       const Place &p, int rot, const float2 (&t)[8], float (&y)[2][8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float x0 = bits_to_f32<F16>(half_of(r.v[0], i)), x1 = bits_to_f32<F16>(half_of(r.v[1], i));
        y[0][i] = x0;
        y[1][i] = x1;
        if (P == HALF && p.turns) {
            y[0][i] = x0 * t[i].x - x1 * t[i].y;
            y[1][i] = x0 * t[i].y + x1 * t[i].x;
        }
    }
    if (P == NEXT) {
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
            if (p.e[0] + i >= rot) break;
            float &lo = y[i / 8][i % 8], &hi = y[i / 8][i % 8 + 1];
            const float x = lo, z = hi;
            lo = x * t[i / 2].x - z * t[i / 2].y;
            hi = x * t[i / 2].y + z * t[i / 2].x;
        }
    }
    if (P == ANY) {
        const int half = rot / 2;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int d = p.e[0] + i;
            if (d >= rot) break;
            const bool first = d < half;
            const float z = bits_to_f32<F16>(part[first ? d + half : d - half]);
            const float2 c = turn_of(a, freq, pos, first ? d : d - half);
            float &o = y[i / 8][i % 8];
            o = o * c.x + z * (first ? -c.y : c.y);
        }
    }
}

template <Pairs P>
__device__ __forceinline__ void angles(const Append8Args &a, const uint64_t *freq, int64_t pos, const Place &p, int rot, float2 (&t)[8])
{
    if (P == ANY || !p.turns) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int pair = P == HALF ? p.e[0] + i : p.e[0] / 2 + i;
        t[i] = pair < rot / 2 ? turn_of(a, freq, pos, pair) : make_float2(1.0f, 0.0f);
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
    int lanes_log;   // threads of a row, log 2
    int gk, nk, gq;  // heads per CTA and CTAs for keys (and for values); heads per CTA for queries
};

template <int CODE, bool F16, Pairs P>
__global__ void __launch_bounds__(ROWS * 8, 4) k_append8(const Append8Args a, const AppendGrid g)
{
    using X = Exponents<CODE, F16>;
    __shared__ uint64_t freq[64];
    __shared__ unsigned starts[8];              // rows that begin a run: the chunk's, and those behind it
    __shared__ int end_row;                     // behind the last run
    __shared__ uint32_t peak[MOST_HEADS][ROWS]; // of the run that begins at a row
    __shared__ int8_t scale[MOST_HEADS][ROWS], growth[MOST_HEADS][ROWS];
    __shared__ int odd;  // some element is not finite, or past the codes at the range's end
    const int tid = threadIdx.x, S = a.c.S, D = a.c.D;
    const int i = tid >> g.lanes_log, u = tid & ((1 << g.lanes_log) - 1);
    const int c0 = blockIdx.x * ROWS, rows = min(ROWS, a.T - c0);
    const int kind = blockIdx.y;
    const bool keys = kind < g.nk, queries = kind >= 2 * g.nk;
    const int rot = keys || queries ? a.rot : 0;
    const Place p = place_of<P>(u, D, rot);
    const int h0 = queries ? (kind - 2 * g.nk) * g.gq : (keys ? kind : kind - g.nk) * g.gk;
    const int nh = queries ? min(g.gq, a.Hq - h0) : min(g.gk, a.c.heads - h0);
    // the CTA's first head in a row of qkv
    const uint16_t *qkv = a.qkv + static_cast<int64_t>((queries ? 0 : a.Hq + (keys ? 0 : a.c.heads)) + h0) * D;

    grid_dep_wait();
    grid_dep_launch_dependents();
    Raw raw[AHEAD];
    auto head = [&](int row, int h) { return qkv + row * a.qkv_stride + h * D; };
    auto load = [&](int row, int h) {  // heads h .. of the CTA
#pragma unroll
        for (int n = 0; n < AHEAD; ++n)
            if (h + n < nh) raw[n] = load_raw(head(row, h + n), p);
    };
    if (i < rows && p.in) load(c0 + i, 0);
    if (tid < rot / 2) freq[tid] = turns_of(a.freq[tid]);
    float2 t[8];
    if (queries) {
        __syncthreads();
        if (i >= rows) return;  // (whole heads)
        const int row = c0 + i;
        const int64_t pos = rot ? a.position[row] : 0;
        if (p.in) angles<P>(a, freq, pos, p, rot, t);
        const int64_t at = row * a.q_stride + h0 * D, len = (a.T - 1) * a.q_stride + static_cast<int64_t>(a.Hq) * D;
        for (int h = 0; h < nh; h += AHEAD) {
            if (h > 0 && p.in) load(row, h);
            float y[AHEAD][2][8];
#pragma unroll
            for (int n = 0; n < AHEAD; ++n)
                if (h + n < nh && p.in) rotate<P, F16>(a, freq, pos, head(row, h + n), raw[n], p, rot, t, y[n]);
            __syncwarp();  // q_out may be qkv: a head's lanes have read it before one writes
#pragma unroll
            for (int n = 0; n < AHEAD; ++n) {
                if (h + n >= nh || !p.in) break;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int64_t to = at + (h + n) * D + p.e[e];
                    const float (&z)[8] = y[n][e];
                    if (store_ok(to + 7, len, a.err))
                        *reinterpret_cast<uint4 *>(a.q_out + to) = make_uint4(pack16<F16>(z[0], z[1]), pack16<F16>(z[2], z[3]),
                                                                              pack16<F16>(z[4], z[5]), pack16<F16>(z[6], z[7]));
                }
            }
        }
        return;
    }

    // ---- keys or values: the runs
    uint8_t *codes = keys ? a.c.k : a.c.v, *exps = keys ? a.c.k_exp : a.c.v_exp;
    const int64_t slots = static_cast<int64_t>(a.c.blocks) * S;
    const int64_t codes_len = (a.c.blocks - 1) * a.c.block_stride + (a.c.heads - 1) * a.c.head_stride +
                              (S - 1) * a.c.token_stride + D;
    {
        const unsigned m = __ballot_sync(0xffffffffu, c0 + tid < a.T && begins(a.slot, slots, S, c0 + tid));
        if ((tid & 31) == 0) starts[tid >> 5] = m;
        if (tid < 32)
            for (int h = 0; h < nh; ++h) peak[h][tid] = 0u;
        if (tid == 0) {
            end_row = min(c0 + ROWS + S, a.T);
            odd = 0;
        }
    }
    __syncthreads();
    const unsigned mask = starts[0];
    if (!mask) return;
    int end = end_row;
    for (int w = 1; w < static_cast<int>(blockDim.x >> 5); ++w)
        if (starts[w]) {
            end = min(end, c0 + w * 32 + __ffs(starts[w]) - 1);
            break;
        }
    if (end > c0 + static_cast<int>(blockDim.x)) {  // blocks larger than the look
        __syncthreads();
        for (int x = c0 + blockDim.x + tid; x < min(c0 + ROWS + S, a.T); x += blockDim.x)
            if (begins(a.slot, slots, S, x)) atomicMin(&end_row, x);
        __syncthreads();
        end = end_row;
    }
    // the exponents of continued blocks, asked for now
    int old[2];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int n = tid + x * blockDim.x, lead = n % ROWS;
        old[x] = 0;
        if (n >= nh * ROWS || !(mask >> lead & 1)) continue;
        const int64_t slot = a.slot[c0 + lead];
        if (slot >= 0 && slot < slots) old[x] = exps[slot / S * a.c.heads + h0 + n / ROWS];
    }
    // of a row: the chunk's row that its run begins at (-1: none of the chunk's), and its slot
    struct Row {
        int lead;
        int64_t slot;
    };
    auto row_of = [&](int row) {
        Row r = {-1, -1};
        if (row >= end) return r;
        const unsigned upto = row - c0 >= ROWS - 1 ? mask : mask & ((2u << (row - c0)) - 1);
        if (!upto) return r;
        r.slot = a.slot[row];
        if (r.slot >= 0 && r.slot < slots) r.lead = 31 - __clz(upto);
        return r;
    };
    const bool once = end <= c0 + ROWS && nh <= AHEAD;  // one look: the elements stay in registers
    static_assert(MOST_HEADS * ROWS <= 2 * ROWS * 4, "two of the runs' scales per thread");
    Row r;
    int64_t pos = 0;
    // ---- largest magnitudes
    for (int r0 = c0; r0 < end; r0 += ROWS) {
        if (r0 > c0 && p.in && r0 + i < a.T) load(r0 + i, 0);
        r = row_of(r0 + i);
        const bool on = r.lead >= 0 && p.in;
        if (on && rot) pos = a.position[r0 + i];
        if (on) angles<P>(a, freq, pos, p, rot, t);
        for (int h = 0; h < nh; h += AHEAD) {
            if (on && h > 0) load(r0 + i, h);
#pragma unroll
            for (int n = 0; n < AHEAD; ++n) {
                if (h + n >= nh) break;
                float m = 0.0f;
                if (on) {
                    float y[2][8];
                    rotate<P, F16>(a, freq, pos, head(r0 + i, h + n), raw[n], p, rot, t, y);
#pragma unroll
                    for (int e = 0; e < 16; ++e) m = max_nan(m, fabsf(y[e / 8][e % 8]));
                    if (!(m <= 3.4028234664e38f)) {  // infinities and NaN do not count
                        m = 0.0f;
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float v = fabsf(y[e / 8][e % 8]);
                            m = v <= 3.4028234664e38f ? fmaxf(m, v) : m;
                        }
                        odd = 1;
                    }
                }
                for (int d = 1 << g.lanes_log >> 1; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                if (r.lead >= 0 && u == 0) atomicMax(&peak[h + n][r.lead], __float_as_uint(m));
            }
        }
    }
    __syncthreads();
    // ---- the runs' scales
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        const int n = tid + x * blockDim.x, h = n / ROWS, lead = n % ROWS;
        if (n >= nh * ROWS || !(mask >> lead & 1)) continue;
        growth[h][lead] = 0;
        const int64_t slot = a.slot[c0 + lead];
        if (slot < 0 || slot >= slots) continue;
        const int64_t blk = slot / S;
        uint8_t *at = exps + blk * a.c.heads + h0 + h;
        int e = needed<CODE, F16>(peak[h][lead]);
        if (e == X::HI) odd = 1;
        if (slot != blk * S) {
            const int held = X::of(old[x]);
            if (e > held)
                growth[h][lead] = static_cast<int8_t>(e - held);
            else
                e = held;
        }
        scale[h][lead] = static_cast<int8_t>(e);
        if (store_ok(at - exps, static_cast<int64_t>(a.c.blocks) * a.c.heads, a.err)) *at = static_cast<uint8_t>(e + 127);
    }
    __syncthreads();
    // ---- the new codes
    const bool special = odd;
    for (int r0 = c0; r0 < end; r0 += ROWS) {
        if (!once && p.in && r0 + i < a.T) load(r0 + i, 0);
        if (!once) r = row_of(r0 + i);
        if (r.lead < 0 || !p.in) continue;
        if (!once && rot) pos = a.position[r0 + i];
        if (!once) angles<P>(a, freq, pos, p, rot, t);
        const int64_t blk = r.slot / S;
        const int64_t at = blk * a.c.block_stride + (r.slot - blk * S) * a.c.token_stride + h0 * a.c.head_stride;
        for (int h = 0; h < nh; h += AHEAD) {
            if (h > 0) load(r0 + i, h);
#pragma unroll
            for (int n = 0; n < AHEAD; ++n) {
                if (h + n >= nh) break;
                float y[2][8];
                rotate<P, F16>(a, freq, pos, head(r0 + i, h + n), raw[n], p, rot, t, y);
                const float inv = pow2(-scale[h + n][r.lead]);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    uint32_t w[2];
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        const float z[4] = {y[e][4 * b], y[e][4 * b + 1], y[e][4 * b + 2], y[e][4 * b + 3]};
                        if (special) {
                            const float x[4] = {z[0] * inv, z[1] * inv, z[2] * inv, z[3] * inv};
                            w[b] = f32_to_codes<CODE>(x);
                        } else {
                            w[b] = finite_to_codes<CODE>(z, inv);
                        }
                    }
                    const int64_t to = at + (h + n) * a.c.head_stride + p.e[e];
                    if (store_ok(to + 7, codes_len, a.err)) *reinterpret_cast<uint2 *>(codes + to) = make_uint2(w[0], w[1]);
                }
            }
        }
    }
    // ---- codes held already, where the scale grew: a warp per run and head
    const int warp = tid >> 5, lane = tid & 31, warps = blockDim.x >> 5, pieces = D / 16;
    for (int n = warp; n < nh * ROWS; n += warps) {
        const int h = n / ROWS, lead = n % ROWS;
        if (!(mask >> lead & 1) || growth[h][lead] == 0) continue;
        const int64_t slot = a.slot[c0 + lead], blk = slot / S;
        const float f = pow2(-growth[h][lead]);
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
    g.lanes_log = a.c.D > 64 ? 3 : 2;
    const int chunks = ctas_for(a.T, ROWS);
    // Heads per CTA: as many as leave about three CTAs of a kind per SM (8192 rows,
    // 64/8 heads: 68.5 us; six 67.2, but 1001 rows of 32/32 heads 20.4 and 22, 2048
    // of 64/8 19.6 and 23; twelve 73, 31 and 25).
    const auto heads_for = [&](int64_t heads, int most) {
        return static_cast<int>(std::min<int64_t>({std::max<int64_t>(1 + heads / 8192, chunks * heads / (3 * sm_count)), heads, most}));
    };
    g.gk = heads_for(2 * a.c.heads, std::min(a.c.heads, MOST_HEADS));
    g.nk = ctas_for(a.c.heads, g.gk);
    g.gq = heads_for(a.Hq, 16);
    const dim3 grid(chunks, 2 * g.nk + ctas_for(a.Hq, g.gq));
    const int threads = ROWS << g.lanes_log;
    if (interleaved) return launch_dependent(k_append8<CODE, F16, NEXT>, grid, threads, 0, s, a, g);
    if (a.rot % 16) return launch_dependent(k_append8<CODE, F16, ANY>, grid, threads, 0, s, a, g);
    return launch_dependent(k_append8<CODE, F16, HALF>, grid, threads, 0, s, a, g);
}

// -------------------------------------------------------------- reading back
// Memory-bound: a byte in, two (or four) out.  A CTA takes up to 32 token rows,
// finds their requests (one warp), and each thread widens 16 codes at a time,
// four such pieces in flight.  Measured: 24 requests of 900..8100 tokens, 8 heads
// of 128, in 110 us, 0.89 of the measured copy bandwidth; 777 tokens of 32 heads
// in 8.9 us.
constexpr int READ_ROWS = 32, READ_THREADS = 256, READ_AHEAD = 4;

struct ReadGrid {
    int rows;               // of a CTA
    FastDiv by_row, by_head;  // pieces of a row's keys and values; of a head
};

template <int CODE, bool F16, bool F32>
__global__ void __launch_bounds__(READ_THREADS) k_read8(const Read8Args a, const ReadGrid g)
{
    __shared__ int64_t place[READ_ROWS];  // of a row's token in the codes; -1: zeros, -2: no request
    __shared__ int block[READ_ROWS];
    const int tid = threadIdx.x, t0 = blockIdx.x * g.rows, rows = min(g.rows, a.T - t0);
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
    const int per = a.c.heads * (a.c.D / 16);  // pieces of a row's keys
    const int total = rows * 2 * per;
    for (int n0 = tid; n0 < total; n0 += READ_AHEAD * READ_THREADS) {
        uint4 v[READ_AHEAD];
        int e[READ_AHEAD];
        int64_t to[READ_AHEAD];  // -1: nothing
        bool vals[READ_AHEAD];
#pragma unroll
        for (int x = 0; x < READ_AHEAD; ++x) {
            const int n = n0 + x * READ_THREADS, r = g.by_row.div(min(n, total - 1)), u = n - r * 2 * per;
            const int64_t at = place[r];
            vals[x] = u >= per;
            const int w = vals[x] ? u - per : u, h = g.by_head.div(max(w, 0)), c = w - h * (a.c.D / 16);
            v[x] = make_uint4(0, 0, 0, 0);
            e[x] = 127;
            to[x] = n < total && at != -2 ? (t0 + r) * (vals[x] ? a.v_stride : a.k_stride) + w * 16 : -1;
            if (n < total && at >= 0) {
                v[x] = __ldcs(reinterpret_cast<const uint4 *>((vals[x] ? a.c.v : a.c.k) + at + h * a.c.head_stride + c * 16));
                e[x] = (vals[x] ? a.c.v_exp : a.c.k_exp)[static_cast<int64_t>(block[r]) * a.c.heads + h];
            }
        }
#pragma unroll
        for (int x = 0; x < READ_AHEAD; ++x) {
            if (to[x] < 0) continue;
            if (!store_ok(to[x] + 15, (a.T - 1) * (vals[x] ? a.v_stride : a.k_stride) + static_cast<int64_t>(a.c.heads) * a.c.D, a.err))
                continue;
            void *out = vals[x] ? a.v_out : a.k_out;
            const float f = pow2(Exponents<CODE, F16>::of(e[x]));
            const uint32_t words[4] = {v[x].x, v[x].y, v[x].z, v[x].w};
            float y[16];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float z[4];
                codes_to_f32<CODE>(words[q], z);
#pragma unroll
                for (int b = 0; b < 4; ++b) y[4 * q + b] = z[b] * f;
            }
            if (F32) {
                float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(out) + to[x]);
#pragma unroll
                for (int q = 0; q < 4; ++q) __stcs(o + q, make_float4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]));
            } else {
                uint4 *o = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + to[x]);
#pragma unroll
                for (int q = 0; q < 2; ++q)
                    __stcs(o + q, make_uint4(pack16<F16>(y[8 * q], y[8 * q + 1]), pack16<F16>(y[8 * q + 2], y[8 * q + 3]),
                                             pack16<F16>(y[8 * q + 4], y[8 * q + 5]), pack16<F16>(y[8 * q + 6], y[8 * q + 7])));
            }
        }
    }
}

template <int CODE, bool F16>
cudaError_t read_launch(const Read8Args &a, bool f32_out, int sm_count, cudaStream_t s)
{
    ReadGrid g{};
    const int per = 2 * a.c.heads * (a.c.D / 16);
    g.by_row.set(per);
    g.by_head.set(a.c.D / 16);
    // 16 pieces a thread, fewer where that leaves SMs without a CTA
    g.rows = std::max(1, std::min({READ_ROWS, 16 * READ_THREADS / per, ctas_for(a.T, 4 * sm_count)}));
    const dim3 grid(ctas_for(a.T, g.rows));
    return f32_out ? launch_dependent(k_read8<CODE, F16, true>, grid, READ_THREADS, 0, s, a, g)
                   : launch_dependent(k_read8<CODE, F16, false>, grid, READ_THREADS, 0, s, a, g);
}

}  // namespace

cudaError_t append8_launch(const Append8Args &a, q4_code code, bool f16, bool interleaved, int sm_count, cudaStream_t s)
{
    if (code == Q4_I8) return f16 ? append_launch<I8, true>(a, interleaved, sm_count, s) : append_launch<I8, false>(a, interleaved, sm_count, s);
    return f16 ? append_launch<E4M3, true>(a, interleaved, sm_count, s) : append_launch<E4M3, false>(a, interleaved, sm_count, s);
}

cudaError_t read8_launch(const Read8Args &a, q4_code code, bool f16, bool f32_out, int sm_count, cudaStream_t s)
{
    if (code == Q4_I8) return f16 ? read_launch<I8, true>(a, f32_out, sm_count, s) : read_launch<I8, false>(a, f32_out, sm_count, s);
    return f16 ? read_launch<E4M3, true>(a, f32_out, sm_count, s) : read_launch<E4M3, false>(a, f32_out, sm_count, s);
}

}  // namespace q4
