// qk_moe_tile_q6k.cu -- the many-token form of the experts' products, Q6K weights.
#include "qk_moe_tile.cuh"

namespace qk {
namespace moe {
cudaError_t tile_launch_q6k(const TileOperands &t, const TileArgs &a, bool paired, int sms, cudaStream_t st)
{
    return tile_launch<kFmtQ6K>(t, a, paired, sms, st);
}
}  // namespace moe
}  // namespace qk
