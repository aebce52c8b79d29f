// Epilogue of a grouped product for one element (the tile kernels' scalar form
// of GroupArgs' description).
#pragma once
#include "common.cuh"
#include "kernels.h"

namespace mg {

template <typename T>
static __device__ __forceinline__ void group_epilogue(const GroupArgs& g, size_t o, float x) {
  auto round_t = [](float v) { return sizeof(T) == 2 ? __bfloat162float(__float2bfloat16_rn(v)) : v; };
  if (g.act || g.resid || g.out_z) x = round_t(x);
  if (g.out_z) st_elem(static_cast<T*>(g.out_z), o, x);
  if (g.act) x = apply_act(g.act, x);
  if (g.dact) x = round_t(x) * act_grad_from_saved(g.dact, ld_elem(static_cast<const T*>(g.saved), o));
  if (g.resid) x += ld_elem(static_cast<const T*>(g.resid), o);
  st_elem(static_cast<T*>(g.out), o, x);
}

}  // namespace mg
