// prefill_masked.cu -- pa_prefill_masked: the choice among the kernels (prefill_masked.cuh)
// that mask, cap and bias, and the one that only masks (windows and prefixes).
#include <string.h>

#include "prefill_masked_launch.cuh"

namespace pa {

// tanh(x) ~ sum c_k x^(2 k + 1), minimax fits (Lawson's iteration): 4 terms for |x| <= 1/2, off by
// 2^-22.9 at most, 6 terms for |x| <= 1, off by 2^-22.0 (in fp32 2^-22.4 and 2^-21.6).
// Of the raw scores, x = f s with f = scale / cap, the terms are cap_log2 c_k f^(2 k + 1).
static void set_tanh(PrefillMaskedParams& p) {
  constexpr double kNear[4] = {0.9999976761923924, -0.33320655217201633, 0.131451456485501, -0.0433724834987327};
  constexpr double kWide[6] = {0.9999968538800571, -0.33324003803682367, 0.13253525316763984,
                               -0.05097286452796889, 0.016114182103335564, -0.0028394659261702696};
  const double f = p.scale_log2;
  auto pairs = [&](const double* c, int n, uint64_t* out) {
    for (int k = 0; k < n; ++k) {
      const float v = static_cast<float>(p.cap_log2 * c[k] * pow(f, 2 * k + 1));
      uint32_t bits;
      memcpy(&bits, &v, 4);
      out[k] = static_cast<uint64_t>(bits) << 32 | bits;
    }
  };
  pairs(kNear, 4, p.tanh_near);
  pairs(kWide, 6, p.tanh_wide);
  // (factors whose powers would leave fp32's range: the third form always)
  const bool fine = f >= 0x1p-11 && f <= 0x1p8 && p.cap_log2 >= 0x1p-4f && p.cap_log2 <= 0x1p16f;
  p.tanh_near_to = fine ? static_cast<float>(0.5 / f) : -1.f;
  p.tanh_wide_to = fine ? static_cast<float>(1.0 / f) : -1.f;
}

cudaError_t launch_prefill_masked(int dtype, int head_size, int block_size, const PrefillMaskedParams& p,
                                  cudaStream_t stream, int* launches) {
  if (p.cap_log2 != 0.f) {
    PrefillMaskedParams q = p;
    set_tanh(q);
    return (p.slopes ? launch_prefill_capped_biased : launch_prefill_capped)(dtype, head_size, block_size, q, stream,
                                                                             launches);
  }
  if (p.slopes) return launch_prefill_biased(dtype, head_size, block_size, p, stream, launches);
  return launch_prefill_masked_kind<0>(dtype, head_size, block_size, p, stream, launches);
}

}  // namespace pa
