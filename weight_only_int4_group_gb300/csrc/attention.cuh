// attention.cuh -- what the two attention kernels share: the sequence of work
// units, how a worker (a CTA or a warp) finds and walks its range of it, and
// the final store.
#pragma once

#include "serve.cuh"

namespace q4 {

// A request's new tokens and length as the kernels use them: cut to the token
// rows and to the table's width, so that no index leaves its buffer whatever
// the device arrays hold.  Plain loads, here and of the table: this kernel is
// resident while the one that wrote them may still run, and the non-coherent
// path asks for data that nothing writes as long as a kernel lives.
__device__ __forceinline__ void request(const AttnArgs &a, int b, int &t0, int &n, int &kv)
{
    t0 = min(max(a.q_start[b], 0), a.T);
    n = max(0, min(max(a.q_start[b + 1], 0), a.T) - t0);
    kv = static_cast<int>(min(static_cast<int64_t>(max(a.kv_len[b], 0)),
                              static_cast<int64_t>(a.width) * a.S));
}

__device__ __forceinline__ int row_tiles(int n, int GQ, int R)
{
    return static_cast<int>((static_cast<int64_t>(n) * GQ + R - 1) / R);
}

// The first key that the window leaves to the row in place p (and with it to
// the rows behind it).
__device__ __forceinline__ int window_start(const AttnArgs &a, int p)
{
    const int64_t first = static_cast<int64_t>(p) - a.window + 1;
    return a.window > 0 && first > 0 ? static_cast<int>(first) : 0;
}

// Rows [row0, row1) of a request's n * GQ rows and the units of TK keys they
// see: units [kt0, kt0 + units) of the request's keys; one (all masked) when
// they see none, so that their empty results are written.
template <int R, int TK>
struct Span {
    int t0, kv, base, row0, row1, kt0, units;
    __device__ __forceinline__ Span(const AttnArgs &a, int b, int rt)
    {
        int n;
        request(a, b, t0, n, kv);
        init(a, n, rt);
    }
    __device__ __forceinline__ Span(const AttnArgs &a, int n, int kv_, int rt) : t0(0), kv(kv_)
    {
        init(a, n, rt);
    }

private:
    __device__ __forceinline__ void init(const AttnArgs &a, int n, int rt)
    {
        base = kv - n;
        row0 = rt * R;
        row1 = static_cast<int>(min(static_cast<int64_t>(n) * a.GQ, static_cast<int64_t>(row0) + R));
        const int lo_t = a.by_GQ.div(row0), hi_t = a.by_GQ.div(row1 - 1);
        const int hi = base + hi_t + 1;
        const int lo = window_start(a, base + lo_t);
        kt0 = lo / TK;
        units = hi > lo ? (hi - 1) / TK - kt0 + 1 : 1;
    }
};

struct Item {
    int b, rt, head;
    __device__ __forceinline__ void next(const AttnArgs &a, int R)
    {
        if (++head < a.Hkv) return;
        next_rows(a, R);
    }
    __device__ __forceinline__ void next_rows(const AttnArgs &a, int R)
    {
        head = 0;
        int t0, n, kv;
        request(a, b, t0, n, kv);
        if (++rt < row_tiles(n, a.GQ, R)) return;
        rt = 0;
        for (++b; b < a.B; ++b) {
            request(a, b, t0, n, kv);
            if (n > 0) return;
        }
    }
};

struct Range {
    int64_t u0, u1, total;  // the worker's places and all places of the call's sequence
    int G;                  // workers that share them
    Item first;             // item of place u0
    int kt;                 // u0 within that item
};

struct LocateScratch {
    int64_t slab[32];
    Range r;
};

// Worker holding place i of T cut into G equal ranges [c * T / G, (c + 1) * T / G).
__device__ __forceinline__ int owner_of(int64_t i, int64_t T, int64_t G)
{
    return static_cast<int>(((i + 1) * G - 1) / T);
}

// Places of all row tiles of request b for one KV head: their units and PAD
// more each.  Lanes hold one
// request each; requests of many row tiles are summed by the whole warp.
template <int R, int TK, int PAD>
__device__ __forceinline__ int64_t request_units(const AttnArgs &a, int b, bool in)
{
    int t0, n = 0, kv = 0;
    if (in) request(a, b, t0, n, kv);
    const int nt = row_tiles(n, a.GQ, R);
    int64_t sum = 0;
    if (nt <= 2)
        for (int rt = 0; rt < nt; ++rt) sum += Span<R, TK>(a, n, kv, rt).units + PAD;
    unsigned big = __ballot_sync(0xffffffffu, nt > 2);
    const int lane = threadIdx.x & 31;
    while (big) {
        const int src = __ffs(big) - 1;
        big &= big - 1;
        const int n2 = __shfl_sync(0xffffffffu, n, src), kv2 = __shfl_sync(0xffffffffu, kv, src),
                  nt2 = __shfl_sync(0xffffffffu, nt, src);
        int64_t part = 0;
        for (int rt = lane; rt < nt2; rt += 32) part += Span<R, TK>(a, n2, kv2, rt).units + PAD;
#pragma unroll
        for (int d = 16; d; d >>= 1) part += __shfl_xor_sync(0xffffffffu, part, d);
        if (lane == src) sum = part;
    }
    return sum;
}

// Sums of slabs of requests, one per warp; a barrier.  Nothing for up to 32
// requests, which one warp sees at once.
template <int R, int TK, int NW, int PAD>
__device__ __forceinline__ void sum_slabs(const AttnArgs &a, LocateScratch &ls)
{
    if (a.B <= 32) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int b0 = static_cast<int>(static_cast<int64_t>(a.B) * warp / NW),
              b1 = static_cast<int>(static_cast<int64_t>(a.B) * (warp + 1) / NW);
    int64_t slab = 0;
    for (int b = b0; b < b1; b += 32) slab += request_units<R, TK, PAD>(a, b + lane, b + lane < b1);
#pragma unroll
    for (int d = 16; d; d >>= 1) slab += __shfl_xor_sync(0xffffffffu, slab, d);
    if (lane == 0) ls.slab[warp] = slab;
    __syncthreads();
}

__device__ __forceinline__ int64_t inclusive_sum(int64_t v)
{
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t p = __shfl_up_sync(0xffffffffu, v, d);
        if (static_cast<int>(threadIdx.x & 31) >= d) v += p;
    }
    return v;
}

// Equal share `worker` of the sequence among as many of `workers` as get
// MIN_UNITS places each (none between two others is left without one: the
// pieces of an item are counted by their workers), and the item it begins in.
// Called by a whole warp after sum_slabs.
template <int R, int TK, int NW, int MIN_UNITS, int PAD>
__device__ Range find_share(const AttnArgs &a, const LocateScratch &ls, int worker, int workers)
{
    const int lane = threadIdx.x & 31;
    const bool few = a.B <= 32;
    int64_t all = 0, mine = 0, incl = 0;
    if (few) {
        mine = request_units<R, TK, PAD>(a, lane, lane < a.B) * a.Hkv;
        incl = inclusive_sum(mine);
        all = __shfl_sync(0xffffffffu, incl, 31);
    } else {
#pragma unroll
        for (int w = 0; w < NW; ++w) all += ls.slab[w] * a.Hkv;
    }
    Range r = {};
    r.total = all;
    r.G = static_cast<int>(min(static_cast<int64_t>(workers), (r.total + MIN_UNITS - 1) / MIN_UNITS));
    if (worker >= r.G) return r;
    r.u0 = worker * r.total / r.G;
    r.u1 = (worker + 1) * r.total / r.G;
    if (r.u0 >= r.u1) return r;
    // the slab, then the request, then the row tile that holds place u0
    int64_t left = r.u0;
    int b0 = 0, b1 = a.B;
    if (!few) {
        int slab = 0;
        while (left >= ls.slab[slab] * a.Hkv) left -= ls.slab[slab++] * a.Hkv;
        b0 = static_cast<int>(static_cast<int64_t>(a.B) * slab / NW);
        b1 = static_cast<int>(static_cast<int64_t>(a.B) * (slab + 1) / NW);
    }
    for (int b = b0; b < b1; b += 32) {
        if (!few) {
            mine = request_units<R, TK, PAD>(a, b + lane, b + lane < b1) * a.Hkv;
            incl = inclusive_sum(mine);
        }
        const unsigned past = __ballot_sync(0xffffffffu, incl > left);
        if (!past) {
            left -= __shfl_sync(0xffffffffu, incl, 31);
            continue;
        }
        const int src = __ffs(past) - 1;
        left -= __shfl_sync(0xffffffffu, incl - mine, src);
        int t0, n, kv;
        request(a, b + src, t0, n, kv);
        const int nt = row_tiles(n, a.GQ, R);
        for (int rt = 0; rt < nt; rt += 32) {
            const int per = rt + lane < nt ? Span<R, TK>(a, n, kv, rt + lane).units + PAD : 0;
            const int64_t m2 = static_cast<int64_t>(per) * a.Hkv, in2 = inclusive_sum(m2);
            const unsigned past2 = __ballot_sync(0xffffffffu, in2 > left);
            if (!past2) {
                left -= __shfl_sync(0xffffffffu, in2, 31);
                continue;
            }
            const int s2 = __ffs(past2) - 1;
            left -= __shfl_sync(0xffffffffu, in2 - m2, s2);
            const int pl = __shfl_sync(0xffffffffu, per, s2);
            r.first.b = b + src;
            r.first.rt = rt + s2;
            r.first.head = static_cast<int>(left / pl);
            r.kt = static_cast<int>(left % pl);
            break;
        }
        break;
    }
    return r;
}

// The share of one worker per CTA, by one warp for all, in ls.r; barriers.
template <int R, int TK, int NW, int MIN_UNITS, int PAD>
__device__ void share(const AttnArgs &a, LocateScratch &ls, int worker, int workers)
{
    sum_slabs<R, TK, NW, PAD>(a, ls);
    if (threadIdx.x < 32) {
        const Range r = find_share<R, TK, NW, MIN_UNITS, PAD>(a, ls, worker, workers);
        if (threadIdx.x == 0) ls.r = r;
    }
    __syncthreads();
}

// A worker's pieces of items.
template <int R, int TK, int PAD>
struct Walk {
    Item it;
    int64_t v0, vu;    // the item's and the piece's place in the call's sequence
    int vn;            // and its length there
    int kt, nu;        // units [kt, kt + nu) of the item
    int units, kt0;    // the item's units, the first one's index among the request's keys
    int row0, row1, t0, base, kv;
    bool same;         // all but the head as in the piece before
    __device__ __forceinline__ Walk(const AttnArgs &a, const Range &r) : it(r.first), same(false)
    {
        vu = r.u0;
        if (vu >= r.u1) return;
        load(a, r);
        cut(r, r.kt);
        while (nu <= 0 && vu < r.u1) step(a, r);
    }
    __device__ __forceinline__ bool more(const Range &r) const { return vu < r.u1; }
    // Another piece follows (one that would be padding alone does not count).
    __device__ __forceinline__ bool follows(const Range &r) const { return r.u1 - (vu + vn) > PAD; }
    // The next piece that holds a unit.
    __device__ __forceinline__ void next(const AttnArgs &a, const Range &r)
    {
        do step(a, r);
        while (nu <= 0 && vu < r.u1);
    }
    __device__ __forceinline__ bool whole() const { return kt == 0 && nu == units; }

private:
    __device__ __forceinline__ void load(const AttnArgs &a, const Range &r)
    {
        const Span<R, TK> sp(a, it.b, it.rt);
        units = sp.units;
        kt0 = sp.kt0;
        row0 = sp.row0;
        row1 = sp.row1;
        t0 = sp.t0;
        base = sp.base;
        kv = sp.kv;
    }
    // The piece of the item from its place v on: the first PAD places of an
    // item hold no unit.
    __device__ __forceinline__ void cut(const Range &r, int v)
    {
        v0 = vu - v;
        vn = static_cast<int>(min(static_cast<int64_t>(units + PAD - v), r.u1 - vu));
        kt = max(v - PAD, 0);
        nu = max(v + vn - PAD, 0) - kt;
    }
    __device__ __forceinline__ void step(const AttnArgs &a, const Range &r)
    {
        const bool was_whole = whole();
        vu += vn;
        same = false;
        if (vu >= r.u1) return;
        if (++it.head < a.Hkv) {  // the same rows and keys of the next head
            cut(r, 0);
            same = was_whole && nu == units;
            return;
        }
        it.next_rows(a, R);
        load(a, r);
        cut(r, 0);
    }

public:
    // The first key that any of the piece's rows sees; only the item's first
    // unit can hold keys before it.
    __device__ __forceinline__ int first_key(const AttnArgs &a) const
    {
        return window_start(a, base + a.by_GQ.div(row0));
    }
    // First and last worker that hold units of the item.
    __device__ __forceinline__ void holders(const Range &r, int &first, int &last) const
    {
        first = owner_of(v0 + PAD, r.total, r.G);
        last = owner_of(v0 + PAD + units - 1, r.total, r.G);
    }
};

// 2^x to about 2 ulp; 0 below the normal range.
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <bool F16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if (F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 1 / a row's sum of weights: 0 for a row that saw nothing, NaN kept.
__device__ __forceinline__ float inverse(float sum) { return sum == 0.0f ? 0.0f : 1.0f / sum; }

// Dims d..d + N - 1 (those below head_dim) of query head h of token row t,
// rounded once.
template <bool F16, int N>
__device__ __forceinline__ void store_dims(const AttnArgs &a, int64_t t, int h, int d, const float (&v)[N])
{
    constexpr int V = N < 8 ? N : 8;  // head_dim is a multiple of 8
    const int64_t at = t * a.o_stride + static_cast<int64_t>(h) * a.D + d;
#pragma unroll
    for (int i = 0; i < N; i += V) {
        if (d + i >= a.D) return;
        if (!store_ok(at + i + V - 1, static_cast<int64_t>(a.T - 1) * a.o_stride + static_cast<int64_t>(a.Hq) * a.D,
                      a.err))
            return;
        if (a.ot == Q4_F32) {
            float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.o) + at + i);
#pragma unroll
            for (int k = 0; k < V; k += 4) o[k / 4] = make_float4(v[i + k], v[i + k + 1], v[i + k + 2], v[i + k + 3]);
        } else {
            uint32_t w[V / 2];
#pragma unroll
            for (int k = 0; k < V; k += 2) w[k / 2] = pack2<F16>(v[i + k], v[i + k + 1]);
            uint16_t *o = static_cast<uint16_t *>(a.o) + at + i;
            if constexpr (V == 8)
                *reinterpret_cast<uint4 *>(o) = make_uint4(w[0], w[1], w[2], w[3]);
            else
                *reinterpret_cast<uint2 *>(o) = make_uint2(w[0], w[1]);
        }
    }
}

// The row's log-sum-exp; top is in units of log 2.
__device__ __forceinline__ void store_lse(const AttnArgs &a, int64_t t, int h, float top, float sum)
{
    const int64_t l = t * a.Hq + h;
    if (a.lse && store_ok(l, static_cast<int64_t>(a.T) * a.Hq, a.err))
        a.lse[l] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
}

}  // namespace q4
