// op_ids.h -- ids, for the optional event timing, of the kernels that are not the codec's
// own: they follow the codec's (launch.h).
#pragma once
#include "launch.h"

namespace zipnn {

enum OpKernelId { kIdMxAmax = kNumKernelIds, kIdMxQuantize, kIdMxDequantize, kIdMxMatmul, kIdPagesPlan, kIdPagesMove, kNumAllIds };

}  // namespace zipnn
