// Shared pieces of the 8-bit cache kernels: the e4m3 conversions, the cache's
// geometry and the walk over sequences of different lengths.
#pragma once
#include "fa_common.cuh"
#include "fa_kernels.h"

namespace fa {

constexpr int kCacheBlock = 64;          // tokens per cache block

// Two e4m3 codes (low byte first) to two halves; exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t codes) {
  const uint32_t h = e4m3x2_to_f16x2(codes);
  float2 f;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(f.x), "=f"(f.y) : "r"(h));
  return f;
}

// The smallest power of two s, at least 2^-126, with amax / s <= 448 = 1.75 * 2^8
// (amax finite, >= 0): amax = 1.m * 2^e fits 2^(e-8) while 1.m <= 1.75. 0 for amax = 0.
// A power of two makes x / s exact and a later growth of the scale a mere
// shift of the codes' exponents: only codes that become subnormal lose bits.
__device__ __forceinline__ float power_scale(float amax) {
  if (!(amax > 0.f)) return 0.f;
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);   // biased
  return __uint_as_float(static_cast<uint32_t>(max(e, 1)) << 23);
}

// Tokens a sequence holds, as the kernels take it: within its block table.
__device__ __forceinline__ int cache_length(const int* lengths, int b, int max_blocks) {
  return max(0, min(lengths[b], max_blocks * kCacheBlock));
}

// Launch that may be set up while the kernel before it in the stream still runs
// (programmatic dependent launch): a kernel launched so calls wait_before(), which
// returns when that one has ended and its writes are seen, before it reads or
// writes anything that is not its own, and in every CTA before it ends: the kernels behind
// are ordered behind this one only. One that calls let_next() allows the next
// kernel's set-up from there on.
__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <typename... Params, typename... Args>
inline cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute early[1];
  early[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = early;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Params>(args)...);
}

}  // namespace fa
