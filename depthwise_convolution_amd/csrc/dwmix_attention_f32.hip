// dwmix_attention_f32.hip -- the walk of linear attention for float32 elements.
#define DWMIX_ATTENTION_KERNELS
#include "dwmix_attention.h"

namespace dwmix {
template int launch_walks<float>(const Walk *w, int count, hipStream_t st);
}  // namespace dwmix
