// attn_verify_span for one span and cache type (attn_kernel.h).
#include "attn_launch.h"

namespace hrs {
template AttnShape attn_shape<kB16>(int, int);
template void attn_launch<kB16>(const AttnTree&, const AttnLens&, int, int, hipStream_t);
}  // namespace hrs
