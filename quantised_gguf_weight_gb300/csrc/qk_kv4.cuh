// qk_kv4.cuh -- the 4-bit key/value cache block (16 tokens of one head) and
// the element types of the attention operators, shared by the kernels that
// write, read back and attend over it.
//
// The order inside a block is that of the tensor cores' m16n8k16 B operand:
// lane (r = lane/4, c = lane%4) of a warp finds the words of its fragments at
// lane * Gp words, so a warp's loads are contiguous and free of bank
// conflicts, and four masks of a word give four fp16 pairs.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/qk.h"

namespace qk {

constexpr int kBlockTokens = 16;

__host__ __device__ constexpr int kv4_gp(int G) { return G % 4 == 0 ? 4 : G; }

// Byte offsets inside a block of head size D.
struct Kv4Place {
    int byte, nibble;   // the 32-bit word's first byte, and the nibble in it
};
__host__ __device__ inline Kv4Place kv4_key_place(int D, int t, int ch)
{
    const int Gp = kv4_gp(D / 32), g = ch >> 5;
    const int row = ((t >> 1) & 1) * 8 + (t >> 2) * 2 + (t & 1);
    const int w = (((g / Gp) * 16 + row) * 4 + ((ch & 31) >> 3)) * Gp + g % Gp;
    return {4 * w, ch & 7};
}
__host__ __device__ inline Kv4Place kv4_value_place(int D, int t, int ch)
{
    const int Gp = kv4_gp(D / 32), g = ch >> 5;
    const int w = (((g / Gp * 2 + ((t >> 1) & 1)) * 8 + ((ch & 31) >> 2)) * 4 + (t >> 2)) * Gp + g % Gp;
    return {8 * D + 4 * w, (t & 1) * 4 + (ch & 3)};
}
__host__ __device__ constexpr int kv4_key_scale(int D, int t, int g) { return 16 * D + 2 * (t * (D / 32) + g); }
__host__ __device__ constexpr int kv4_value_scale(int D, int t, int g) { return 17 * D + 2 * (t * (D / 32) + g); }

// Element access by type (QK_F32, QK_F16, QK_BF16), one rounding to nearest on store.
__device__ __forceinline__ float load_as_float(const void *p, int64_t i, int type)
{
    if (type == QK_F32) return static_cast<const float *>(p)[i];
    if (type == QK_F16) return __half2float(static_cast<const __half *>(p)[i]);
    return __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[i]);
}
__device__ __forceinline__ void store_float_as(void *p, int64_t i, int type, float v)
{
    if (type == QK_F32) static_cast<float *>(p)[i] = v;
    else if (type == QK_F16) static_cast<__half *>(p)[i] = __float2half_rn(v);
    else static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
}

}  // namespace qk
