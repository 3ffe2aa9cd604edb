// The ragged grouped products of bf16 operands (grouped.hpp).
#include "grouped.hpp"

namespace bsg {

template <bool BK>
static hipError_t go(const GroupedParams& p, int epi, int c_dtype, hipStream_t s) {
    switch (epi) {
    case kEpiNone:
        return c_dtype == kF32 ? grouped_go<kBf16, BK, kEpiNone, kF32>(p, s)
                               : grouped_go<kBf16, BK, kEpiNone, kBf16>(p, s);
    case kEpiGelu:
        return p.aux_out ? grouped_go<kBf16, BK, kEpiGeluSave, kBf16>(p, s)
                         : grouped_go<kBf16, BK, kEpiGelu, kBf16>(p, s);
    case kEpiSiluMul:
        return p.aux_out ? grouped_go<kBf16, BK, kEpiSiluMulSave, kBf16>(p, s)
                         : grouped_go<kBf16, BK, kEpiSiluMul, kBf16>(p, s);
    case kEpiGeluBwd: return grouped_go<kBf16, BK, kEpiGeluBwd, kBf16>(p, s);
    case kEpiSiluMulBwd: return grouped_go<kBf16, BK, kEpiSiluMulBwd, kBf16>(p, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_grouped_bf16(const GroupedParams& p, int trans_b, int epi, int c_dtype,
                               hipStream_t s) {
    return trans_b ? go<true>(p, epi, c_dtype, s) : go<false>(p, epi, c_dtype, s);
}

}  // namespace bsg
