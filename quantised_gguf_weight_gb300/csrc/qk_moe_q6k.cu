// qk_moe_q6k.cu -- the experts' products for few tokens an expert, and for few assignments, Q6K weights.
#include "qk_moe_few.cuh"
#include "qk_moe_rows.cuh"

namespace qk {
namespace moe {
cudaError_t rows_launch_q6k(const RowsArgs &a, bool paired, int sms, cudaStream_t st) { return rows_launch<kFmtQ6K>(a, paired, sms, st); }
cudaError_t few_gate_q6k(const FewArgs &a, int64_t A, int down, bool chained, cudaStream_t st) { return few_gate<kFmtQ6K>(a, A, down, chained, st); }
cudaError_t few_down_q6k(const FewArgs &a, int64_t T, cudaStream_t st) { return few_down<kFmtQ6K>(a, T, st); }
}  // namespace moe
}  // namespace qk
