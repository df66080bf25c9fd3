// What the append kernels with rotary axes share: a token's slot and positions.
#pragma once

#include "device_common.cuh"
#include "internal.h"
#include "num_dev.cuh"
#include "step_ops.h"

namespace pkv {
namespace append {

// What stops a token's key and value rows; reported by one thread.
struct Token {
  int slot;
  bool known, fits;   // every axis in use has a table row; the slot lies in the pool
};
__device__ __forceinline__ Token read_token(const AxesParams& p, int t) {
  Token k;
  k.slot = __ldg(p.slots + t);
  k.known = true;
  for (int a = 0; a < p.axes; ++a)
    if ((p.used_axes >> a) & 1u) {
      const int x = __ldg(p.pos + (int64_t)a * p.T + t);
      k.known = k.known && x >= 0 && x < p.P;
    }
  k.fits = k.slot < p.pool_rows;
  return k;
}
__device__ __forceinline__ void report(const AxesParams& p, const Token& k) {
  if (k.slot >= 0 && (!k.known || !k.fits))
    flag_status(p.status, (k.known ? 0 : PKV_DEV_BAD_POSITION) | (k.fits ? 0 : PKV_DEV_BAD_SLOT));
}

}  // namespace append
}  // namespace pkv
