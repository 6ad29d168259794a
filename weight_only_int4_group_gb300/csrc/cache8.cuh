// cache8.cuh -- what the kernels of the 8-bit cache share: the codes, their
// exponents, and how a token row finds its request.
#pragma once

#include "serve.cuh"

namespace q4 {

constexpr int I8 = Q4_I8, E4M3 = Q4_E4M3;

// Exponents that keep every c * 2^e a number of the 16-bit type.  binary16:
// 2^-24 is its smallest step (an e4m3 code is a multiple of 2^-9), 127 * 2^9 and
// 448 * 2^7 lie below 65504.  bf16 has the room of f32; 2^+-48 leaves weights
// and sums in f32 in units of any of these scales room too.
template <int CODE, bool F16>
struct Exponents {
    static constexpr int LO = F16 ? (CODE == I8 ? -24 : -15) : -48;
    static constexpr int HI = F16 ? (CODE == I8 ? 9 : 7) : 48;
    static __device__ __forceinline__ int of(int byte) { return min(max(byte - 127, LO), HI); }
};

// 2^e, -126 <= e <= 127
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// Two e4m3 codes (the low 16 bits) as a pair of binary16, exactly.
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t codes)
{
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(r) : "r"(codes));
    return r;
}

// The upper halves of two binary16 numbers' f32: of codes, as bf16.
__device__ __forceinline__ uint32_t f16x2_upper(uint32_t x)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&x));
    return __byte_perm(__float_as_uint(f.x), __float_as_uint(f.y), 0x7632);
}

// Four codes of a word as f32.
template <int CODE>
__device__ __forceinline__ void codes_to_f32(uint32_t w, float (&x)[4])
{
    if (CODE == I8) {
        // 2^23 + (c + 128) as f32, less 2^23 + 128
        const uint32_t u = w ^ 0x80808080u;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440 + i)) - 8388736.0f;
    } else {
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            const uint32_t h = e4m3_to_f16x2(w >> (8 * i));
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            x[i] = f.x;
            x[i + 1] = f.y;
        }
    }
}

// Four numbers in units of the scale to the nearest codes, ties to even; NaN to 0.
template <int CODE>
__device__ __forceinline__ uint32_t f32_to_codes(const float (&y)[4])
{
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = y[i] == y[i] ? y[i] : 0.0f;
    if (CODE == I8) {
        uint32_t r = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // 1.5 * 2^23 + x rounds x to an integer in the low bits
            const float f = fminf(fmaxf(x[i], -127.0f), 127.0f) + 12582912.0f;
            r |= (__float_as_uint(f) & 0xFFu) << (8 * i);
        }
        return r;
    }
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]));
    return r;
}

// The same of finite numbers that lie within the codes once they are scaled.
template <int CODE>
__device__ __forceinline__ uint32_t finite_to_codes(const float (&y)[4], float inv)
{
    if (CODE == I8) {
        uint32_t f[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __float_as_uint(fmaf(y[i], inv, 12582912.0f));  // (scaling by a power of two is exact)
        return __byte_perm(__byte_perm(f[0], f[1], 0x0040), __byte_perm(f[2], f[3], 0x0040), 0x5410);
    }
    uint32_t r;
    asm("{\n\t.reg .b16 lo, hi;\n\tcvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\tcvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(r)
        : "f"(y[0] * inv), "f"(y[1] * inv), "f"(y[2] * inv), "f"(y[3] * inv));
    return r;
}

// The larger one, NaN if one is.
__device__ __forceinline__ float max_nan(float x, float y)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

// The least exponent of the range under which a largest magnitude fits the
// codes: 127 = 1.984375 * 2^6, 448 = 1.75 * 2^8, and a mantissa above theirs
// carries into the exponent.
template <int CODE, bool F16>
__device__ __forceinline__ int needed(uint32_t peak_bits)
{
    using X = Exponents<CODE, F16>;
    const int e = CODE == I8 ? static_cast<int>((peak_bits + 0x1FFFFu) >> 23) - 127 - 6
                             : static_cast<int>((peak_bits + 0x1FFFFFu) >> 23) - 127 - 8;
    return min(max(e, X::LO), X::HI);
}

template <bool F16>
__device__ __forceinline__ float bits_to_f32(uint32_t b)
{
    if (!F16) return __uint_as_float(b << 16);
    __half_raw h;
    h.x = static_cast<unsigned short>(b);
    return __half2float(__half(h));
}

// The last request whose first row is at most t, by a whole warp (t the same in
// all lanes): 32 of the starts in a look.
__device__ __forceinline__ int request_of(const int *q_start, int B, int t)
{
    int lo = 0, n = B;
    while (n > 1) {
        const int lane = threadIdx.x & 31, step = (n + 31) / 32;
        const int64_t at = static_cast<int64_t>(lane) * step;
        const unsigned le = __ballot_sync(0xffffffffu, at < n && q_start[lo + min(at, static_cast<int64_t>(n - 1))] <= t);
        const int k = max(__popc(le) - 1, 0) * step;
        lo += k;
        n = min(step, n - k);
    }
    return lo;
}

}  // namespace q4
