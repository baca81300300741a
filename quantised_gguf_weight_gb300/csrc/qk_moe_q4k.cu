// qk_moe_q4k.cu -- the few-token form of the experts' products, Q4K weights.
#include "qk_moe_rows.cuh"

namespace qk {
namespace moe {
cudaError_t rows_launch_q4k(const RowsArgs &a, bool paired, int sms, cudaStream_t st) { return rows_launch<kFmtQ4K>(a, paired, sms, st); }
}  // namespace moe
}  // namespace qk
