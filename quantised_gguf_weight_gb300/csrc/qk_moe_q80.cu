// qk_moe_q80.cu -- the experts' products for few tokens an expert, and for few assignments, Q80 weights.
#include "qk_moe_few.cuh"
#include "qk_moe_rows.cuh"

namespace qk {
namespace moe {
cudaError_t rows_launch_q80(const RowsArgs &a, bool paired, int sms, cudaStream_t st) { return rows_launch<kFmtQ80>(a, paired, sms, st); }
cudaError_t few_gate_q80(const FewArgs &a, int64_t A, int down, bool chained, cudaStream_t st) { return few_gate<kFmtQ80>(a, A, down, chained, st); }
cudaError_t few_down_q80(const FewArgs &a, int64_t T, cudaStream_t st) { return few_down<kFmtQ80>(a, T, st); }
}  // namespace moe
}  // namespace qk
