// Eviction from the 8-bit cache by accumulated attention weight.
//
// Per (sequence, KV head) of n tokens, `keep` of them stay: the last `recent`
// and, of the others, the keep - recent with the largest weights (ties to the
// lower position), all in their order. Two launches:
//  1. cache8_select_kernel  one CTA per (sequence, head): the weights' order
//     as integers, the smallest kept one by four passes over 8 bits each
//     (histograms), then the positions, in order, by block-wide counts.
//  2. cache8_gather_kernel  one CTA per (destination block, head, K or V): the
//     kept tokens' codes, re-encoded with a scale of their own.
#include "fa_cache8.cuh"

namespace fa {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kGatherThreads = 128;
constexpr int kMaxChunks = kCacheBlock * 256 / 16 / kGatherThreads;   // 16-code chunks per thread, d <= 256

// Floats as integers of the same order; -0 as 0, NaN above everything.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) cache8_select_kernel(const Cache8EvictParams p) {
  __shared__ int hist[256];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  __shared__ int warp_eq[32], warp_sel[32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.y, h = blockIdx.x;
  let_next();
  wait_before();
  const int n = cache_length(p.lengths, b, p.max_blocks);
  int* const kept = p.kept + (static_cast<size_t>(b) * p.c.Hkv + h) * p.keep;
  if (h == 0 && tid == 0) p.new_lengths[b] = min(n, p.keep);
  if (n <= p.keep) {
    for (int i = tid; i < p.keep; i += kSelThreads) kept[i] = i < n ? i : -1;
    return;
  }
  const int nc = n - p.recent;                   // candidates
  const int need_all = p.keep - p.recent;        // to choose among them, < nc
  const int* const table = p.table + static_cast<long long>(b) * p.max_blocks;
  auto key_at = [&](int i) -> uint32_t {
    const int page = table[i / kCacheBlock];
    if (page < 0 || page >= p.c.num_blocks) return order_key(0.f);
    return order_key(p.c.weight[(static_cast<size_t>(page) * p.c.Hkv + h) * kCacheBlock + i % kCacheBlock]);
  };
  if (need_all > 0) {
    // the key of the last one chosen, digit by digit from the top
    uint32_t prefix = 0;
    int need = need_all;
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      const uint32_t high = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
      for (int i = tid; i < nc; i += kSelThreads) {
        const uint32_t key = key_at(i);
        if ((key & high) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1);
      }
      __syncthreads();
      if (warp == 0) {
        // bins from the largest down, 8 per lane: the bin where the count reaches `need`
        int sum = 0;
        for (int e = 0; e < 8; ++e) sum += hist[255 - (lane * 8 + e)];
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += y;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, incl >= need);
        if (lane == __ffs(hit) - 1) {
          int left = need - (incl - sum);
          for (int e = 0; e < 8; ++e) {
            const int bin = 255 - (lane * 8 + e);
            if (hist[bin] >= left) {
              s_prefix = prefix | static_cast<uint32_t>(bin) << shift;
              s_need = left;
              break;
            }
            left -= hist[bin];
          }
        }
      }
      __syncthreads();
      prefix = s_prefix;
      need = s_need;
    }
    // positions in order: keys above `prefix`, and the first `need` equal to it
    int eq_base = 0, sel_base = 0;
    for (int i0 = 0; i0 < nc; i0 += kSelThreads) {
      const int i = i0 + tid;
      const uint32_t key = i < nc ? key_at(i) : 0u;
      const bool eq = i < nc && key == prefix, above = i < nc && key > prefix;
      const unsigned beq = __ballot_sync(0xffffffffu, eq), bab = __ballot_sync(0xffffffffu, above);
      if (lane == 0) {
        warp_eq[warp] = __popc(beq);
        warp_sel[warp] = __popc(bab);
      }
      __syncthreads();
      int eq_before = eq_base, above_before = 0, eq_total = 0, above_total = 0;
      for (int w = 0; w < 32; ++w) {
        if (w < warp) {
          eq_before += warp_eq[w];
          above_before += warp_sel[w];
        }
        eq_total += warp_eq[w];
        above_total += warp_sel[w];
      }
      const unsigned below = (1u << lane) - 1u;
      eq_before += __popc(beq & below);
      above_before += __popc(bab & below);
      // chosen before this one: all above, and the equal ones within the first `need`
      const int at = sel_base + above_before + min(eq_before, need) - min(eq_base, need);
      if (above || (eq && eq_before < need)) kept[at] = i;
      sel_base += above_total + min(eq_base + eq_total, need) - min(eq_base, need);
      eq_base += eq_total;
      __syncthreads();
    }
  }
  for (int i = tid; i < p.recent; i += kSelThreads) kept[need_all + i] = nc + i;
}

__global__ void __launch_bounds__(kGatherThreads) cache8_gather_kernel(const Cache8EvictParams p) {
  __shared__ float warp_max[kGatherThreads / 32];
  __shared__ long long src[kCacheBlock];          // (block * Hkv + h) * 64 + slot of a kept token, -1: no such block
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x / p.to_blocks, blk = blockIdx.x - b * p.to_blocks;
  const int h = blockIdx.y, which = blockIdx.z;
  let_next();
  wait_before();
  const int n = cache_length(p.lengths, b, p.max_blocks);
  const int cnt = min(kCacheBlock, min(n, p.keep) - blk * kCacheBlock);
  if (cnt <= 0) return;
  const int page = p.to_table[static_cast<long long>(b) * p.to_blocks + blk];
  if (page < 0 || page >= p.c.num_blocks) return;
  const size_t ph = static_cast<size_t>(page) * p.c.Hkv + h;
  if (tid < cnt) {
    const int i = p.kept[(static_cast<size_t>(b) * p.c.Hkv + h) * p.keep + blk * kCacheBlock + tid];
    const int from = p.table[static_cast<long long>(b) * p.max_blocks + i / kCacheBlock];
    const bool ok = from >= 0 && from < p.c.num_blocks;
    const long long at = (static_cast<long long>(from) * p.c.Hkv + h) * kCacheBlock + i % kCacheBlock;
    src[tid] = ok ? at : -1;
    if (which == 0) p.c.weight[ph * kCacheBlock + tid] = ok ? p.c.weight[at] : 0.f;
  }
  __syncthreads();
  const uint8_t* const codes = which ? p.c.v : p.c.k;
  float* const scales = which ? p.c.v_scale : p.c.k_scale;
  const int cpr = p.c.d / 16, chunks = cnt * cpr;
  uint4 val[kMaxChunks];
  float sc[kMaxChunks];
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < kMaxChunks; ++k) {
    const int c = tid + k * kGatherThreads;
    val[k] = make_uint4(0, 0, 0, 0);
    sc[k] = 0.f;
    if (c < chunks) {
      const int row = c / cpr, col = c - row * cpr;
      const long long at = src[row];
      if (at >= 0) {
        val[k] = *reinterpret_cast<const uint4*>(codes + at * p.c.d + col * 16);
        sc[k] = scales[at / kCacheBlock];
      }
      const uint32_t w[4] = {val[k].x, val[k].y, val[k].z, val[k].w};
      uint32_t m = 0;                             // the largest code without its sign; 0x7F is NaN
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const uint32_t code = (w[e / 4] >> (8 * (e % 4))) & 0x7Fu;
        m = max(m, code == 0x7Fu ? 0u : code);
      }
      amax = fmaxf(amax, e4m3x2_to_float2(m).x * sc[k]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (lane == 0) warp_max[warp] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kGatherThreads / 32; ++w) amax = fmaxf(amax, warp_max[w]);
  float now = power_scale(amax);
  if (!(now > 0.f)) now = 1.f;
  if (tid == 0) scales[ph] = now;
  const float inv = __fdiv_rn(1.f, now);
  uint8_t* const dst = (which ? p.c.v : p.c.k) + ph * kCacheBlock * p.c.d;
#pragma unroll
  for (int k = 0; k < kMaxChunks; ++k) {
    const int c = tid + k * kGatherThreads;
    if (c >= chunks) continue;
    const uint32_t w[4] = {val[k].x, val[k].y, val[k].z, val[k].w};
    uint32_t r[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 a = e4m3x2_to_float2(w[e] & 0xFFFFu), z = e4m3x2_to_float2(w[e] >> 16);
      r[e] = pack_e4m3x2(a.x * sc[k] * inv, a.y * sc[k] * inv) | pack_e4m3x2(z.x * sc[k] * inv, z.y * sc[k] * inv) << 16;
    }
    *reinterpret_cast<uint4*>(dst + c * 16) = make_uint4(r[0], r[1], r[2], r[3]);
  }
}

}  // namespace

cudaError_t launch_cache8_evict(const Cache8EvictParams& p, cudaStream_t stream) {
  const cudaError_t e = launch_early(cache8_select_kernel, dim3(p.c.Hkv, p.B), dim3(kSelThreads), 0, stream, p);
  if (e != cudaSuccess) return e;
  return launch_early(cache8_gather_kernel, dim3(p.B * p.to_blocks, p.c.Hkv, 2), dim3(kGatherThreads), 0, stream, p);
}

}  // namespace fa
