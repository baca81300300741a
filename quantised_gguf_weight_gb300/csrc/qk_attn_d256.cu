// qk_attn_d256.cu -- the few-row form of attention over the 4-bit cache, heads of 256 channels.
#include "qk_attn_rows.cuh"

namespace qk {
namespace attn {

cudaError_t rows_launch_256(const AttnArgs &a, int pieces, int sets, int64_t grid, cudaStream_t st)
{
    return launch_rows_of<8>(a, pieces, sets, grid, st);
}

}  // namespace attn
}  // namespace qk
