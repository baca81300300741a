// qk_moe_tile_q4k.cu -- the many-token form of the experts' products, Q4K weights.
#include "qk_moe_tile.cuh"

namespace qk {
namespace moe {
cudaError_t tile_launch_q4k(const CUtensorMap &hi, const CUtensorMap &lo, const TileArgs &a, bool paired, int sms, cudaStream_t st)
{
    return tile_launch<kFmtQ4K>(hi, lo, a, paired, sms, st);
}
}  // namespace moe
}  // namespace qk
