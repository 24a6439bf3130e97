// How moe_kv_append's rows are shared out over warps, as arithmetic that the
// kernel and the host share (no CUDA header needed).  A warp takes `per` <= 32
// rows at a time, from `first` on in steps of `step`.  Unsigned: with N up to
// 2^31 - 1 rows the last step (at most 2^19 rows) passes 2^31 but not 2^32.
#pragma once

#ifdef __CUDACC__
#define MOE_HD __host__ __device__
#else
#define MOE_HD
#endif

namespace moe {

constexpr unsigned kAppendWarps = 8;     // of a CTA

struct AppendShape {
  unsigned per, ctas;
};

MOE_HD inline AppendShape append_shape(unsigned N, unsigned sms) {
  const unsigned cap = 8 * sms, all = cap * kAppendWarps;
  AppendShape a;
  a.per = (N + all - 1) / all;             // few rows: spread over the SMs
  if (a.per > 32) a.per = 32;
  a.ctas = (N + a.per * kAppendWarps - 1) / (a.per * kAppendWarps);
  if (a.ctas > cap) a.ctas = cap;
  return a;
}
MOE_HD inline unsigned append_first(const AppendShape& a, unsigned cta, unsigned warp) {
  return a.per * (cta * kAppendWarps + warp);
}
MOE_HD inline unsigned append_step(const AppendShape& a) { return a.per * a.ctas * kAppendWarps; }

}  // namespace moe
