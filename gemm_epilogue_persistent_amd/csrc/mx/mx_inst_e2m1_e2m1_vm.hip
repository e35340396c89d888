// MX product kernels: A E2M1, B E2M1, rows grouped by expert.
#include "mx_gemm.hpp"
namespace gep {
GEP_MX_LAUNCH(MX_E2M1, MX_E2M1, true)
}  // namespace gep
