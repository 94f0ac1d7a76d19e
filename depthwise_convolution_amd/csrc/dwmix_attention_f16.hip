// dwmix_attention_f16.hip -- the walk of linear attention for float16 elements.
#define DWMIX_ATTENTION_KERNELS
#include "dwmix_attention.h"

namespace dwmix {
template int launch_walk<dwseq::f16>(const Walk &w, hipStream_t st);
}  // namespace dwmix
