// FP8 (E4M3) GEMM instances: block scales in fp32 or as packed UE8M0 exponents.
#include "gemm_core.h"

namespace dgfp8 {
namespace {

template <class C, int Mask>
hipError_t launch_cfg(Variant v, const GemmParams& p, int grid, hipStream_t stream) {
  return p.sf_packed ? launch_variant<SfCfg<C, true>, Mask>(v, p, grid, stream)
                     : launch_variant<C, Mask>(v, p, grid, stream);
}

}  // namespace

InstanceInfo instance_info(GemmInstance inst) {
  switch (inst) {
    case kInstHuge: return {CfgHuge::BM, CfgHuge::BN, CfgHuge::kOcc};
    case kInstSkinny128: return {CfgSkinny128::BM, CfgSkinny128::BN, CfgSkinny128::kOcc};
    case kInstSkinny64: return {CfgSkinny64::BM, CfgSkinny64::BN, CfgSkinny64::kOcc};
    case kInstLarge: return {CfgLarge::BM, CfgLarge::BN, CfgLarge::kOcc};
    case kInstMid: return {CfgMid::BM, CfgMid::BN, CfgMid::kOcc};
    case kInstDecode: return {CfgDecode::BM, CfgDecode::BN, CfgDecode::kOcc};
    case kInstTall: return {CfgTall::BM, CfgTall::BN, CfgTall::kOcc};
    default: return {0, 0, 0};
  }
}

hipError_t launch_gemm(GemmInstance inst, Variant v, const GemmParams& p, int grid, hipStream_t stream) {
  switch (inst) {
    case kInstHuge: return launch_cfg<CfgHuge, (1 << kDense) | (1 << kMasked) | (1 << kContiguous)>(v, p, grid, stream);
    case kInstSkinny128: return launch_cfg<CfgSkinny128, kDenseAndSplit>(v, p, grid, stream);
    case kInstSkinny64: return launch_cfg<CfgSkinny64, kDenseAndSplit>(v, p, grid, stream);
    case kInstLarge: return launch_cfg<CfgLarge, kAll>(v, p, grid, stream);
    case kInstMid: return launch_cfg<CfgMid, kAll>(v, p, grid, stream);
    case kInstDecode: return launch_cfg<CfgDecode, (1 << kMasked)>(v, p, grid, stream);
    case kInstTall: return launch_cfg<CfgTall, (1 << kDense)>(v, p, grid, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace dgfp8
