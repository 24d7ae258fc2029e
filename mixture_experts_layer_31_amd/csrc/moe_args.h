// Argument checks and small device helpers shared by the operators around the
// layer (moe_balance.hip, moe_block.hip, moe_clip.hip).
#pragma once

#include "moe_common.h"

namespace moe {

inline bool aligned_to(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
inline int launched() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_EHIP; }
inline size_t type_bytes(int32_t t) { return t == MOE_TYPE_F32 ? 4 : t == MOE_TYPE_BF16 ? 2 : 1; }
inline long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }

}  // namespace moe
