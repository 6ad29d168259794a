// attention_tc.cu -- the tensor-core attention kernel over a 16-bit cache.
#include "attention_tc.cuh"

namespace q4 {

size_t attention_tc_part_bytes(int64_t D, int grid)
{
    return static_cast<size_t>(grid) * 4 * (D > 64 ? Sizes<128>::PART : Sizes<64>::PART) * sizeof(float);
}

cudaError_t attention_tc_launch(int grid, const AttnArgs &a, bool f16, cudaStream_t s)
{
    if (a.D > 64) return f16 ? launch<WIDE, true, 128>(grid, a, s) : launch<WIDE, false, 128>(grid, a, s);
    return f16 ? launch<WIDE, true, 64>(grid, a, s) : launch<WIDE, false, 64>(grid, a, s);
}

}  // namespace q4
