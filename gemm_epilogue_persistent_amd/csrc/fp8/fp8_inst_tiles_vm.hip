#include "fp8_gemm.hpp"
namespace gep {
GEP_FP8_LAUNCH(false, true)
}
