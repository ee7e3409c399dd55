// Host side of the decode attention: which instance a call takes, what the
// device holds of it, and the workspace's size.
#include <map>
#include <mutex>
#include <new>
#include <utility>

#include "internal.h"

namespace gwb {

namespace {
std::mutex g_mu;
std::map<std::pair<int, const void *>, AttnSetup> g_setup;   // per device and kernel

gwb_status sm_count(int *dev, int *sms) {
  cudaError_t e = cudaGetDevice(dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, *dev);
  return e == cudaSuccess ? GWB_OK : fail(GWB_ERR_CUDA, "device lookup: %s", cudaGetErrorString(e));
}
}  // namespace

gwb_status attn_setup(const void *kern, size_t smem, int threads, AttnSetup *out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(GWB_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  std::lock_guard<std::mutex> lk(g_mu);
  auto it = g_setup.find({dev, kern});
  if (it == g_setup.end()) {
    AttnSetup s{};
    const gwb_status st = sm_count(&dev, &s.sms);
    if (st != GWB_OK) return st;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&s.per_sm, kern, threads, smem);
    if (e != cudaSuccess) return fail(GWB_ERR_CUDA, "attn_decode setup: %s", cudaGetErrorString(e));
    if (s.per_sm < 1) return fail(GWB_ERR_CUDA, "attn_decode: %zu bytes of shared memory do not fit", smem);
    *out = s;
    try {
      g_setup.emplace(std::make_pair(dev, kern), s);
    } catch (const std::bad_alloc &) {               // looked up again by the next call
    }
    return GWB_OK;
  }
  *out = it->second;
  return GWB_OK;
}

// 16 heads a CTA where the group has more than 8 and the registers hold them
// (head_dim <= 128): the codes are unpacked once for both 8-head tiles.
int attn_tiles(int64_t group, int head_dim) { return group > 8 && head_dim <= 128 ? 2 : 1; }

// Short sequences are not cut (one launch, nothing to join): a pair goes to a CTA, or to a warp where the pairs
// are so many that the SMs want more of them at once.  us for B sequences of tables of L tokens (lengths L/2 .. L,
// 4 bits, head_dim 128, 8 kv heads; 444 CTAs resident), cut / a CTA a pair / a warp a pair:
//   B = 1    L = 128    7.3   5.0   8.6     512   10.6   8.9  22.6     1024   10.9  13.8
//   B = 64   L = 128   15.5  11.6  11.5     512   22.9  19.0  28.7     1024   29.3  27.7     2048   44.5  47.4
//   B = 128  L = 256   24.8  21.8  19.4     512   31.5  28.5  32.2     2048   74.7  75.1
//   B = 256  L = 128   30.1  28.4  19.3     512   58.8  51.0  45.0     1024   85.9  77.2  81.2     2048  142  127
// A longer table may hold one sequence that keeps its CTA busy behind all others, so it is always cut.
constexpr int64_t kAttnUncut = 512, kAttnPairs = 1 << 20;

AttnMode attn_mode(int64_t pairs, int64_t cap, int ctas) {
  if (pairs > kAttnPairs) return kAttnCut;
  if (cap <= kAttnUncut && cap * ctas <= 128 * pairs) return kAttnWarpPair;
  if (cap <= kAttnUncut || (cap <= 2048 && pairs >= 4 * (int64_t)ctas)) return kAttnCtaPair;
  return kAttnCut;
}

gwb_status attn_workspace_bytes(int64_t q_heads, int64_t kv_heads, int head_dim, int64_t B, int64_t max_tokens,
                                int64_t *bytes) {
  int dev = 0, sms = 0;
  const gwb_status s = sm_count(&dev, &sms);
  if (s != GWB_OK) return s;
  const int64_t group = q_heads / kv_heads, heads = 8 * attn_tiles(group, head_dim);
  // uncut whatever the number of resident CTAs, and for fewer sequences too: the table's width alone decides
  if (B > 0 && max_tokens > 0 && max_tokens <= kAttnUncut &&
      B <= kAttnPairs / (kv_heads * ((group + heads - 1) / heads))) {
    *bytes = 0;
    return GWB_OK;
  }
  // two partials (sums, max and total a head) and a 16-byte record a CTA
  *bytes = (int64_t)sms * kAttnMaxPerSm * (2 * 4 * heads * (head_dim + 2) + 16);
  return GWB_OK;
}

gwb_status launch_attn_decode(AttnCall c, cudaStream_t st) {
  c.tiles = attn_tiles(c.q_heads / c.cache.heads, c.cache.head_dim);
  if (c.cache.bits == 4) return c.f16 ? launch_attn_4_fp16(c, st) : launch_attn_4_bf16(c, st);
  return c.f16 ? launch_attn_8_fp16(c, st) : launch_attn_8_bf16(c, st);
}

}  // namespace gwb
