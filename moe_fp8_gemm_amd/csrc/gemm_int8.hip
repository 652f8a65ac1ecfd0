// int8 GEMM instances: the tiles and variants of the FP8 GEMM on int8 operands with
// fp32 scales per token (row of A) and channel (row of B); see Int8Cfg.
#include "gemm_core.h"

namespace dgfp8 {

hipError_t launch_gemm_int8(GemmInstance inst, Variant v, const GemmParams& p, int grid, hipStream_t stream) {
  switch (inst) {
    case kInstHuge: return launch_variant<Int8Cfg<CfgHuge>, (1 << kDense) | (1 << kMasked) | (1 << kContiguous)>(v, p, grid, stream);
    case kInstSkinny128: return launch_variant<Int8Cfg<CfgSkinny128>, kDenseAndSplit>(v, p, grid, stream);
    case kInstSkinny64: return launch_variant<Int8Cfg<CfgSkinny64>, kDenseAndSplit | (1 << kMasked)>(v, p, grid, stream);
    case kInstLarge: return launch_variant<Int8Cfg<CfgLarge>, kAll>(v, p, grid, stream);
    case kInstMid: return launch_variant<Int8Cfg<CfgMid>, kAll>(v, p, grid, stream);
    case kInstDecode: return launch_variant<Int8Cfg<CfgDecode>, (1 << kMasked)>(v, p, grid, stream);
    case kInstTall: return launch_variant<Int8Cfg<CfgTall>, (1 << kDense)>(v, p, grid, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace dgfp8
