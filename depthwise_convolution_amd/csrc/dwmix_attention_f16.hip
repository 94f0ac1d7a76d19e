// dwmix_attention_f16.hip -- the walk of linear attention for float16 elements.
#define DWMIX_ATTENTION_KERNELS
#include "dwmix_attention.h"

namespace dwmix {
template int launch_walks<dwseq::f16>(const Walk *w, int count, hipStream_t st);
}  // namespace dwmix
