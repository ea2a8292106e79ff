// Host side of the sampling from logits: how many CTAs a row gets, and whether rows that quick passes
// leave open go to a launch of their own. The kernel and the method are in ds_head_sample.cuh.
#include <algorithm>
#include <mutex>

#include "ds_head_sample.cuh"

namespace ds {
namespace {

using namespace sample;

struct SampleDevice {
  int sms;
};
std::once_flag g_sample_once[kMaxHeadDevices];
SampleDevice g_sample_device[kMaxHeadDevices];
cudaError_t g_sample_error[kMaxHeadDevices];

cudaError_t sample_device(SampleDevice* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxHeadDevices) return cudaErrorInvalidDevice;
  std::call_once(g_sample_once[dev], [dev] {
    cudaError_t& s = g_sample_error[dev];
    s = cudaDeviceGetAttribute(&g_sample_device[dev].sms, cudaDevAttrMultiProcessorCount, dev);
    for (auto prepare : {prepare_rows<float, kWhole>, prepare_rows<float, kQuick>,
                         prepare_rows<float, kRest>, prepare_rows<__nv_bfloat16, kWhole>,
                         prepare_rows<__nv_bfloat16, kQuick>, prepare_rows<__nv_bfloat16, kRest>})
      if (s == cudaSuccess) s = prepare();
  });
  *out = g_sample_device[dev];
  return g_sample_error[dev];
}

template <int MODE>
cudaError_t launch(int es, const SampleArgs& q, int C, int64_t clusters, int sms, cudaStream_t st) {
  return es == 4 ? launch_rows<float, MODE>(q, C, clusters, sms, st)
                 : launch_rows<__nv_bfloat16, MODE>(q, C, clusters, sms, st);
}

}  // namespace

cudaError_t launch_sample_logits(const ds_sample_logits_args& a, cudaStream_t st) {
  SampleDevice dev;
  cudaError_t e = sample_device(&dev);
  if (e != cudaSuccess) return e;
  const int es = a.dtype == DS_DTYPE_FP32 ? 4 : 2, per16 = 16 / es;
  const int64_t bytes = (a.vocab + per16) * es;
  // CTAs a row: as many rows side by side as two CTAs an SM allow, and with fewer rows more CTAs
  // each, down to shares of 8 KB. One CTA a row needs no exchange between CTAs, which costs about
  // as much as a pass over 30000 tokens: measured at 256 x 262144 bf16 with top-p and min-p, 8 / 1
  // CTAs a row: 190 / 85 us.
  int C = 1;
  while (C < kMaxCluster && a.rows * C * 2 <= 2 * dev.sms && bytes > C * 8192ll) C *= 2;
  // Rows that quick passes leave open take ten passes and more; where there are rows enough to fill
  // the GPU with few CTAs each, a second launch of larger clusters does those rows (2048 x 32749 fp32,
  // all settings mixed: one CTA each there 302 us, eight 243 us; with nothing left it takes 6 us).
  int C2 = C;
  while (C2 < kMaxCluster && a.vocab > C2 * 4096ll) C2 *= 2;
  const bool two = C2 > C && a.rows * C >= dev.sms / 2;
  int lg = 0;
  while ((1ll << lg) < a.vocab) ++lg;
  SampleArgs s{a.logits, a.temperature, a.top_p, a.min_p, a.u, a.top_k, a.done, a.token, a.prob,
               a.logits_stride, a.rows, (int)a.vocab, 0, ldexpf(1.f, kMassBits - lg),
               std::max(0, kListBits - (kMassBits - lg))};
  // rows in slices of what a grid holds
  const int64_t most = 1ll << 27;
  for (int64_t r0 = 0; r0 < a.rows; r0 += most) {
    SampleArgs q = s;
    q.rows = a.rows - r0 < most ? a.rows - r0 : most;
    q.logits = static_cast<const uint8_t*>(a.logits) + r0 * a.logits_stride * es;
    if (q.temperature) q.temperature += r0;
    if (q.top_k) q.top_k += r0;
    if (q.top_p) q.top_p += r0;
    if (q.min_p) q.min_p += r0;
    q.u += r0;
    if (q.done) q.done += r0;
    q.token += r0;
    if (q.prob) q.prob += r0;
    if (!two) {
      e = launch<kWhole>(es, q, C, q.rows, dev.sms, st);
    } else {
      e = launch<kQuick>(es, q, C, q.rows, dev.sms, st);
      if (e == cudaSuccess)
        e = launch<kRest>(es, q, C2, std::min<int64_t>(q.rows, std::max(1, 2 * dev.sms / C2)), dev.sms,
                          st);
    }
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace ds
