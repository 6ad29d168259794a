// attention8_tc.cu -- the tensor-core attention kernel over an 8-bit cache
// (attention_tc.cuh), for more than 32 rows per KV head, and for 17 to 32 with few
// requests (attention8.cu): its tiles of 256 rows read the codes once where the
// streaming kernel's of 32 would read them again for each (16 requests of 4000
// keys, 8 new tokens, 64/8 heads: 71 us, there 94 to 110).
#include "attention_tc.cuh"

namespace q4 {

template <int CODE>
static cudaError_t launch_code(int grid, const AttnArgs &a, bool f16, cudaStream_t s)
{
    if (a.D > 64) return f16 ? launch<CODE, true, 128>(grid, a, s) : launch<CODE, false, 128>(grid, a, s);
    return f16 ? launch<CODE, true, 64>(grid, a, s) : launch<CODE, false, 64>(grid, a, s);
}

cudaError_t attention8_tc_launch(int grid, const AttnArgs &a, q4_code code, bool f16, cudaStream_t s)
{
    return code == Q4_I8 ? launch_code<I8>(grid, a, f16, s) : launch_code<E4M3>(grid, a, f16, s);
}

}  // namespace q4
