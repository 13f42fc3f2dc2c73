// Launches of attn_verify_span's kernel for one span and cache type
// (attn_kernel.h), by head size and class of row counts.
#pragma once

#include "attn_kernel.h"

namespace hrs {
namespace {

template <int KIND, int D, int CLS, typename Args>
void launch_as(const Args& args, const AttnLens& l, hipStream_t s) {
  using C = AttnCfg<KIND, D, CLS>;
  hipLaunchKernelGGL((attn_kernel<KIND, D, CLS, Args>), dim3(1 << l.log_blocks), dim3(C::NT), C::LDS, s, l.len, l.n, l.heads,
                     l.most, l.window, l.n_pos, l.log_blocks, args);
}
template <int KIND, int D, int CLS> void launch_one(const AttnTree& args, const AttnLens& l, hipStream_t s) {
  if (args.tree) launch_as<KIND, D, CLS>(args, l, s);
  else launch_as<KIND, D, CLS>(static_cast<const AttnBase&>(args), l, s);
}
template <int KIND, int D, int CLS> AttnShape shape_one() {
  using C = AttnCfg<KIND, D, CLS>;
  return {C::ROWS, C::TS, kAttnCus * C::PER_CU};
}

}  // namespace

template <int KIND> AttnShape attn_shape(int d, int cls) {
  switch (d * 8 + cls) {
    case 64 * 8 + 0: return shape_one<KIND, 64, 0>();
    case 64 * 8 + 1: return shape_one<KIND, 64, 1>();
    case 64 * 8 + 2: return shape_one<KIND, 64, 2>();
    case 64 * 8 + 3: return shape_one<KIND, 64, 3>();
    case 128 * 8 + 0: return shape_one<KIND, 128, 0>();
    case 128 * 8 + 1: return shape_one<KIND, 128, 1>();
    case 128 * 8 + 2: return shape_one<KIND, 128, 2>();
    case 128 * 8 + 3: return shape_one<KIND, 128, 3>();
    case 256 * 8 + 0: return shape_one<KIND, 256, 0>();
    case 256 * 8 + 1: return shape_one<KIND, 256, 1>();
    case 256 * 8 + 2: return shape_one<KIND, 256, 2>();
    case 256 * 8 + 3: return shape_one<KIND, 256, 3>();
  }
  if constexpr (KIND == kF8) {
    if (cls == 4) return d == 64 ? shape_one<KIND, 64, 4>() : shape_one<KIND, 128, 4>();
  }
  return {0, 0, 0};
}

template <int KIND> void attn_launch(const AttnTree& args, const AttnLens& lens, int d, int cls, hipStream_t s) {
  switch (d * 8 + cls) {
    case 64 * 8 + 0: return launch_one<KIND, 64, 0>(args, lens, s);
    case 64 * 8 + 1: return launch_one<KIND, 64, 1>(args, lens, s);
    case 64 * 8 + 2: return launch_one<KIND, 64, 2>(args, lens, s);
    case 64 * 8 + 3: return launch_one<KIND, 64, 3>(args, lens, s);
    case 128 * 8 + 0: return launch_one<KIND, 128, 0>(args, lens, s);
    case 128 * 8 + 1: return launch_one<KIND, 128, 1>(args, lens, s);
    case 128 * 8 + 2: return launch_one<KIND, 128, 2>(args, lens, s);
    case 128 * 8 + 3: return launch_one<KIND, 128, 3>(args, lens, s);
    case 256 * 8 + 0: return launch_one<KIND, 256, 0>(args, lens, s);
    case 256 * 8 + 1: return launch_one<KIND, 256, 1>(args, lens, s);
    case 256 * 8 + 2: return launch_one<KIND, 256, 2>(args, lens, s);
    case 256 * 8 + 3: return launch_one<KIND, 256, 3>(args, lens, s);
  }
  if constexpr (KIND == kF8) {
    if (cls == 4) return d == 64 ? launch_one<KIND, 64, 4>(args, lens, s) : launch_one<KIND, 128, 4>(args, lens, s);
  }
}

}  // namespace hrs
