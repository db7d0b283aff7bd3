// qkv_fp8.cu — the QKV projection from e4m3 tokens and weights (qkv_proj.cuh).
#include "qkv_proj.cuh"

namespace jattn {

cudaError_t launch_qkv_norm_e4m3(const CUtensorMap (&maps)[4], const QkvLaunch& a,
                                 uint32_t* dev_err, cudaStream_t st) {
  return launch_qkv_form<kE4m3>(maps, a, dev_err, st, nullptr, nullptr);
}

}  // namespace jattn
