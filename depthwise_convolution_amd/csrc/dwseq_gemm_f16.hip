// dwseq_gemm_f16.hip -- the tiled matrix product for binary16 elements.
#define DWSEQ_GEMM_KERNELS
#include "dwseq_gemm.h"

namespace dwseq {
template int launch_gemm<f16>(const Product &p, hipStream_t st);
}  // namespace dwseq
