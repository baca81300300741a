// qk_moe_q80.cu -- the few-token form of the experts' products, Q80 weights.
#include "qk_moe_rows.cuh"

namespace qk {
namespace moe {
cudaError_t rows_launch_q80(const RowsArgs &a, bool paired, int sms, cudaStream_t st) { return rows_launch<kFmtQ80>(a, paired, sms, st); }
}  // namespace moe
}  // namespace qk
