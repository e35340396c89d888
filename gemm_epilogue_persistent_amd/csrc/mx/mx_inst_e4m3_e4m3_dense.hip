// MX product kernels: A E4M3, B E4M3, dense.
#include "mx_gemm.hpp"
namespace gep {
GEP_MX_LAUNCH(MX_E4M3, MX_E4M3, false)
}  // namespace gep
