// MX product kernels: A E4M3, B E2M1, rows grouped by expert.
#include "mx_gemm.hpp"
namespace gep {
GEP_MX_LAUNCH(MX_E4M3, MX_E2M1, true)
}  // namespace gep
