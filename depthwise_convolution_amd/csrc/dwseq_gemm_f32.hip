// dwseq_gemm_f32.hip -- the tiled matrix product for float32 elements.
#define DWSEQ_GEMM_KERNELS
#include "dwseq_gemm.h"

namespace dwseq {
template int launch_gemm<float>(const Product &p, hipStream_t st);
}  // namespace dwseq
