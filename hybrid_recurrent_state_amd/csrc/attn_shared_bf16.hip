// attn_verify_shared for one span and cache type (attn_kernel.h).
#include "attn_prefix.h"
#include "attn_shared_launch.h"

namespace hrs {
template void attn_own_launch<kB16>(const AttnSharedTree&, const AttnLens&, int, int, hipStream_t);
template void attn_prefix_launch<kB16>(const AttnShared&, const AttnLens&, int, int, hipStream_t);
template void attn_prefix_wide<kB16>(const AttnShared&, const AttnLens&, int, int, hipStream_t);
}  // namespace hrs
