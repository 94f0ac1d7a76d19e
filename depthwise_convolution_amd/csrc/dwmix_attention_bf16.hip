// dwmix_attention_bf16.hip -- the walk of linear attention for bfloat16 elements.
#define DWMIX_ATTENTION_KERNELS
#include "dwmix_attention.h"

namespace dwmix {
template int launch_walks<dwseq::bf16>(const Walk *w, int count, hipStream_t st);
}  // namespace dwmix
