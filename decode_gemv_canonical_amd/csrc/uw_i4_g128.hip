// The 4-bit product's kernels for groups of 128 columns.
#include "uw_i4_gemm.h"

namespace uw {

int i4_gemm_g128(const I4Args& a, int shape, hipStream_t s) { return run_form<128>(a, shape, s); }

}  // namespace uw
