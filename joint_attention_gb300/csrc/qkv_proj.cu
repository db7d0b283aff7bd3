// qkv_proj.cu — the QKV projection from bf16 tokens and weights (qkv_proj.cuh),
// and the choice between its forms.
#include "qkv_proj.cuh"

namespace jattn {

// Pairs of CTAs once their tiles fill half of the GPU; below, tiles of one
// head by single CTAs (also under a cap of one CTA).
bool qkv_uses_pairs(const QkvLaunch& a) {
  const int sms = device_sm_count();
  if (sms < 2) return false;
  const int64_t cols = (3 * static_cast<int64_t>(a.H) * a.d + 255) / 256;
  const int64_t tiles = ((a.M[0] + 255) / 256 + (a.M[1] + 255) / 256) * cols;
  return 4 * tiles > sms;
}

cudaError_t launch_qkv_norm(const CUtensorMap (&maps)[4], const CUtensorMap (&out_maps)[5], const QkvLaunch& a,
                            uint32_t* dev_err, cudaStream_t st, const LoraLaunch* lora,
                            const CUtensorMap* lora_maps) {
  if (lora) return launch_qkv_norm_lora(maps, out_maps, a, dev_err, st, lora, lora_maps);
  if (a.e4m3) return launch_qkv_norm_e4m3(maps, out_maps, a, dev_err, st);
  return launch_qkv_form<kBf16>(maps, out_maps, a, dev_err, st, nullptr, nullptr);
}

}  // namespace jattn
