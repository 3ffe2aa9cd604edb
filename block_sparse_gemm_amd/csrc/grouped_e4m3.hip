// The ragged grouped products of e4m3 operands with row and column scales
// (grouped.hpp); weights K-contiguous.
#include "grouped.hpp"

namespace bsg {

hipError_t launch_grouped_e4m3(const GroupedParams& p, int epi, hipStream_t s) {
    switch (epi) {
    case kEpiNone: return grouped_go<kE4m3, true, kEpiNone, kBf16>(p, s);
    case kEpiGelu: return grouped_go<kE4m3, true, kEpiGelu, kBf16>(p, s);
    case kEpiSiluMul: return grouped_go<kE4m3, true, kEpiSiluMul, kBf16>(p, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace bsg
