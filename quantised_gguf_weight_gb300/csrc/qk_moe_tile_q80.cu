// qk_moe_tile_q80.cu -- the many-token form of the experts' products, Q80 weights.
#include "qk_moe_tile.cuh"

namespace qk {
namespace moe {
cudaError_t tile_launch_q80(const TileOperands &t, const TileArgs &a, bool paired, int sms, cudaStream_t st)
{
    return tile_launch<kFmtQ80>(t, a, paired, sms, st);
}
}  // namespace moe
}  // namespace qk
