// MX product kernels: A E2M1, B E2M1, dense.
#include "mx_gemm.hpp"
namespace gep {
GEP_MX_LAUNCH(MX_E2M1, MX_E2M1, false)
}  // namespace gep
