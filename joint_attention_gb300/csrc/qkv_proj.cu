// qkv_proj.cu — the QKV projection from bf16 tokens and weights (qkv_proj.cuh),
// and the choice between its forms.
#include "qkv_proj.cuh"

namespace jattn {

// Pairs of CTAs once their tiles fill half of the GPU; below, tiles of one
// head by single CTAs, which start some 3 us sooner (and under a cap of one
// CTA).  Tokens of one stream, pairs / single CTAs in us:
//   bf16, 12 heads of 64, C 768:   512 11.0 /  8.4,  768 11.0 / 11.9, 1536 11.5 / 15.7, 3000 16.9 / 26.9
//   bf16, 16 heads of 128, C 2048: 256 20.5 / 15.9,  512 20.1 / 25.3, 1536 32.5 / 44.5, 3000 56.6 / 82.9
//   e4m3, 12 heads of 64, C 768:   512  9.6 /  6.8, 1024  9.8 /  9.0, 1536 10.0 / 11.1, 3000 13.7 / 17.2
// The rule takes pairs from 1025 tokens on for the first and third, from 257 for the second.
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
