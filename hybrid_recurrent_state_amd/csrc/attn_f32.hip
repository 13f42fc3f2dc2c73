// attn_verify_span for one span and cache type (attn_kernel.h).
#include "attn_kernel.h"

namespace hrs {
template AttnShape attn_shape<kF32>(int, int);
template void attn_launch<kF32>(const AttnTree&, const AttnLens&, int, int, hipStream_t);
}  // namespace hrs
