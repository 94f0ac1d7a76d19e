// dwseq_gemm_bf16.hip -- the tiled matrix product for bfloat16 elements.
#define DWSEQ_GEMM_KERNELS
#include "dwseq_gemm.h"

namespace dwseq {
template int launch_gemm<bf16>(const Product &p, hipStream_t st);
}  // namespace dwseq
