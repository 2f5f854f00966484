// qmm_types.h -- host-side helpers of the entry points that take QMM_TYPE_* tensors.  No device code.
#pragma once

#include "qmm_host.h"

namespace qmm {

inline bool valid_type(int t) { return t == QMM_TYPE_F32 || t == QMM_TYPE_F16 || t == QMM_TYPE_BF16; }
inline uintptr_t type_bytes(int t) { return t == QMM_TYPE_F32 ? 4 : 2; }

}  // namespace qmm
