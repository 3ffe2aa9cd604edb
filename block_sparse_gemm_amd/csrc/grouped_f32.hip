// The ragged grouped products of fp32 operands (grouped.hpp).
#include "grouped.hpp"

namespace bsg {

template <bool BK>
static hipError_t go(const GroupedParams& p, int epi, hipStream_t s) {
    switch (epi) {
    case kEpiNone: return grouped_go<kF32, BK, kEpiNone, kF32>(p, s);
    case kEpiGelu:
        return p.aux_out ? grouped_go<kF32, BK, kEpiGeluSave, kF32>(p, s)
                         : grouped_go<kF32, BK, kEpiGelu, kF32>(p, s);
    case kEpiSiluMul:
        return p.aux_out ? grouped_go<kF32, BK, kEpiSiluMulSave, kF32>(p, s)
                         : grouped_go<kF32, BK, kEpiSiluMul, kF32>(p, s);
    case kEpiGeluBwd: return grouped_go<kF32, BK, kEpiGeluBwd, kF32>(p, s);
    case kEpiSiluMulBwd: return grouped_go<kF32, BK, kEpiSiluMulBwd, kF32>(p, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_grouped_f32(const GroupedParams& p, int trans_b, int epi, hipStream_t s) {
    return trans_b ? go<true>(p, epi, s) : go<false>(p, epi, s);
}

}  // namespace bsg
