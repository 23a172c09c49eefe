// prefill_masked.cu -- pa_prefill_masked: the choice among the kernels (prefill_masked.cuh)
// that mask, cap and bias, and the one that only masks (windows and prefixes).
#include <string.h>

#include "prefill_masked_launch.cuh"

namespace pa {

// tanh(x) ~ sum c_k x^(2 k + 1), minimax in relative error (Lawson's iteration): 4 terms for |x| <= 1/2 (tanh_ratio's),
// off by 2^-20.8 at most, 6 terms for |x| <= 1, off by 2^-20.7 (in fp32 2^-20.6 and 2^-20.4).
// Of the raw scores s, x = f s with f = scale / cap, the terms are cap_log2 c_k f^(2 k + 1) = scale_log2 c_k f^(2 k).
// What a term's coefficient is off by as an fp32 number (2^-150 where it is that small) comes into the score with s^7, or
// s^11: for any cap that is below 2^-29 where |s| <= 2^16, or, with 6 terms, 2^11.  So large caps have the 4 terms up to
// that score or to cap / 2, whichever is less, and the form that serves every score beyond.
static void set_tanh(PrefillMaskedParams& p) {
  constexpr double kNear[4] = {kTanhRatio0, kTanhRatio1, kTanhRatio2, kTanhRatio3};
  constexpr double kWide[6] = {0.9999994135992479, -0.33329042378480966, 0.1328143388034517,
                               -0.05160567399125354, 0.01674311505139179, -0.0030670603216316227};
  const double f = static_cast<double>(p.scale_log2) / p.cap_log2;
  auto pairs = [&](const double* c, int n, uint64_t* out) {
    for (int k = 0; k < n; ++k) {
      const float v = static_cast<float>(p.scale_log2 * c[k] * pow(f, 2 * k));
      uint32_t bits;
      memcpy(&bits, &v, 4);
      out[k] = static_cast<uint64_t>(bits) << 32 | bits;
    }
  };
  pairs(kNear, 4, p.tanh_near);
  pairs(kWide, 6, p.tanh_wide);
  // (a scale that no model has, or a cap below scale / 256: coefficients past fp32, or scores past the cap anyway)
  const bool fine = f <= 0x1p8 && p.scale_log2 <= 0x1p24f;
  p.tanh_near_to = fine ? static_cast<float>(fmin(0.5 / f, 0x1p16)) : -1.f;
  p.tanh_exp = static_cast<float>(fmin(f * 2.8853900817779268, 0x1p126));
  p.tanh_wide_to = fine && f >= 0x1p-11 ? static_cast<float>(1.0 / f) : p.tanh_near_to;
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
