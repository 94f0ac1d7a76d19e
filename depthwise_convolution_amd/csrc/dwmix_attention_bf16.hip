// dwmix_attention_bf16.hip -- the walk of linear attention for bfloat16 elements.
#define DWMIX_ATTENTION_KERNELS
#include "dwmix_attention.h"

namespace dwmix {
template int launch_walk<dwseq::bf16>(const Walk &w, hipStream_t st);
}  // namespace dwmix
