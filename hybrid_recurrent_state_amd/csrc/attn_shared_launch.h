// Launches of attn_verify_shared's kernels for one span and cache type
// (attn_kernel.h), by head size and class of row counts.
#pragma once

#include "attn_kernel.h"

namespace hrs {
namespace {

template <int KIND, int D, int CLS, int MODE, typename Args>
__global__ __launch_bounds__((AttnCfg<KIND, D, CLS>::NT), (AttnCfg<KIND, D, CLS>::NT * AttnCfg<KIND, D, CLS>::PER_CU + 255) / 256)
void attn_shared_kernel(const AttnLens lens, const Args args) {
  attn_blocks<KIND, D, CLS, MODE>(lens, args);
}

template <int KIND, int D, int CLS, int MODE, typename Args>
void launch_shared(const Args& args, const AttnLens& l, hipStream_t s) {
  using C = AttnCfg<KIND, D, CLS>;
  hipLaunchKernelGGL((attn_shared_kernel<KIND, D, CLS, MODE, Args>), dim3(1 << l.log_blocks), dim3(C::NT), C::LDS, s, l, args);
}
struct OwnLaunch {
  template <int KIND, int D, int CLS> static void go(const AttnSharedTree& args, const AttnLens& l, hipStream_t s) {
    if (args.tree) launch_shared<KIND, D, CLS, kOwn>(args, l, s);
    else launch_shared<KIND, D, CLS, kOwn>(static_cast<const AttnShared&>(args), l, s);
  }
};
struct PrefixLaunch {
  template <int KIND, int D, int CLS> static void go(const AttnShared& args, const AttnLens& l, hipStream_t s) {
    launch_shared<KIND, D, CLS, kPrefix>(args, l, s);
  }
};
template <typename L, int KIND, int D, typename Args>
void launch_class(const Args& args, const AttnLens& l, int cls, hipStream_t s) {
  switch (cls) {
    case 0: return L::template go<KIND, D, 0>(args, l, s);
    case 1: return L::template go<KIND, D, 1>(args, l, s);
    case 2: return L::template go<KIND, D, 2>(args, l, s);
    case 3: return L::template go<KIND, D, 3>(args, l, s);
  }
  if constexpr (KIND == kF8 && D <= 128) L::template go<KIND, D, 4>(args, l, s);
}
template <typename L, int KIND, typename Args>
void launch_size(const Args& args, const AttnLens& l, int d, int cls, hipStream_t s) {
  if (d == 64) launch_class<L, KIND, 64>(args, l, cls, s);
  else if (d == 128) launch_class<L, KIND, 128>(args, l, cls, s);
  else launch_class<L, KIND, 256>(args, l, cls, s);
}

}  // namespace

template <int KIND> void attn_own_launch(const AttnSharedTree& args, const AttnLens& lens, int d, int cls, hipStream_t s) {
  launch_size<OwnLaunch, KIND>(args, lens, d, cls, s);
}
template <int KIND> void attn_prefix_launch(const AttnShared& args, const AttnLens& lens, int d, int cls, hipStream_t s) {
  launch_size<PrefixLaunch, KIND>(args, lens, d, cls, s);
}

}  // namespace hrs
