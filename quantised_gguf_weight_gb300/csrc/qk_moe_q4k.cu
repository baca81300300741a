// qk_moe_q4k.cu -- the experts' products for few tokens an expert, and for few assignments, Q4K weights.
#include "qk_moe_few.cuh"
#include "qk_moe_rows.cuh"

namespace qk {
namespace moe {
cudaError_t rows_launch_q4k(const RowsArgs &a, bool paired, int sms, cudaStream_t st) { return rows_launch<kFmtQ4K>(a, paired, sms, st); }
cudaError_t few_gate_q4k(const FewArgs &a, int64_t A, int down, bool chained, cudaStream_t st) { return few_gate<kFmtQ4K>(a, A, down, chained, st); }
cudaError_t few_down_q4k(const FewArgs &a, int64_t T, cudaStream_t st) { return few_down<kFmtQ4K>(a, T, st); }
}  // namespace moe
}  // namespace qk
