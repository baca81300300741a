// qk_moe_tile_q4k.cu -- the many-token form of the experts' products, Q4K weights.
#include "qk_moe_tile.cuh"

namespace qk {
namespace moe {
cudaError_t tile_launch_q4k(const TileOperands &t, const TileArgs &a, bool paired, int sms, cudaStream_t st)
{
    return tile_launch<kFmtQ4K>(t, a, paired, sms, st);
}
}  // namespace moe
}  // namespace qk
