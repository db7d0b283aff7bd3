// qkv_proj.cu — the QKV projection from bf16 tokens and weights (qkv_proj.cuh),
// and the choice between its forms.
#include "qkv_proj.cuh"

namespace jattn {

// Pairs of CTAs once one CTA a tile of one head would take more than one tile
// on some SM; below that single CTAs, which start some 1.5 us sooner, also under
// a cap of one CTA.  Tokens of one stream, pairs / single CTAs in us:
//   bf16, 12 heads of 64, C 768:   512  9.2 /  7.8,  768  9.8 / 11.5, 1536 11.9 / 15.6, 3000 15.6 / 27.4
//   bf16, 16 heads of 128, C 2048: 256 16.2 / 15.0,  512 18.2 / 25.1, 1536 29.5 / 44.5, 3000 52.4 / 83.7
//   e4m3, 12 heads of 64, C 768:   512  7.8 /  6.1, 1024  8.5 /  8.4, 1536  9.9 / 10.6, 3000 13.1 / 17.3
//   bf16, 4 heads of 64, C 256:   1536  7.1 /  5.4, 3000  7.5 /  7.2
// The rule takes pairs from 513, 385, 513 and 1537 tokens on, for outputs at 16-byte
// boundaries too (17616 tokens of the first: pairs 52.4, single CTAs 130 us).
bool qkv_uses_pairs(const QkvLaunch& a) {
  const int sms = device_sm_count();
  if (sms < 2) return false;
  const int64_t row_tiles = (a.M[0] + 127) / 128 + (a.M[1] + 127) / 128;
  return row_tiles * 3 * a.H > sms;
}

cudaError_t launch_qkv_norm(const CUtensorMap (&maps)[4], const QkvLaunch& a,
                            uint32_t* dev_err, cudaStream_t st, const LoraLaunch* lora,
                            const CUtensorMap* lora_maps) {
  if (lora) return launch_qkv_norm_lora(maps, a, dev_err, st, lora, lora_maps);
  if (a.e4m3) return launch_qkv_norm_e4m3(maps, a, dev_err, st);
  return launch_qkv_form<kBf16>(maps, a, dev_err, st, nullptr, nullptr);
}

}  // namespace jattn
