// dwseq_gemm_i8.hip -- the tiled matrix product for 8-bit integers.
#define DWSEQ_GEMM_KERNELS
#include "dwseq_gemm.h"

namespace dwseq {
template int launch_gemm<I8<float>>(const Product &p, hipStream_t st);
template int launch_gemm<I8<f16>>(const Product &p, hipStream_t st);
template int launch_gemm<I8<bf16>>(const Product &p, hipStream_t st);
}  // namespace dwseq
