// Decode attention over 8-bit caches, fp16 queries and outputs (the kernel is in attn_decode.cuh).
#include "attn_decode.cuh"

namespace gwb {

gwb_status launch_attn_8_fp16(const AttnCall &c, cudaStream_t st) {
#define GWB_ATTN(D, GS, NT) \
  if (c.cache.head_dim == D && c.cache.gs == GS && c.tiles == NT) \
    return run_attn<8, D, GS, NT, true>(attn_args(c), c.ws_bytes, st);
  GWB_ATTN(64, 32, 1)
  GWB_ATTN(64, 32, 2)
  GWB_ATTN(64, 64, 1)
  GWB_ATTN(64, 64, 2)
  GWB_ATTN(128, 32, 1)
  GWB_ATTN(128, 32, 2)
  GWB_ATTN(128, 64, 1)
  GWB_ATTN(128, 64, 2)
  GWB_ATTN(128, 128, 1)
  GWB_ATTN(128, 128, 2)
  GWB_ATTN(256, 32, 1)
  GWB_ATTN(256, 64, 1)
  GWB_ATTN(256, 128, 1)
#undef GWB_ATTN
  return GWB_ERR_UNSUPPORTED;
}

}  // namespace gwb
