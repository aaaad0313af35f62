// Eviction from the 8-bit cache by accumulated attention weight.
//
// Per (sequence, KV head) of n tokens, `keep` of them stay: the last `recent`
// and, of the others, the keep - recent with the largest weights (ties to the
// lower position), all in their order. Two launches:
//  1. cache8_select_kernel  one cluster per (sequence, head), a stretch of the tokens
//     to each of its CTAs: the weights, read once, lie in shared memory as integers of
//     the same order; the smallest kept one is found digit by digit (8 bits each;
//     histograms that the CTAs read from one another), then every warp counts the
//     tokens of its stretch that stay and writes their positions behind those before.
//  2. cache8_gather_kernel  one CTA per (destination block, head, K or V): the
//     kept tokens' codes, re-encoded with a scale of their own.
// Measured: 8 sequences of 8192 to 32768 tokens, 8 heads, d 128, cut to 4096: 46 us, of which the
// selection some 18 (7 MB; its rounds of histograms and barriers bound it: one CTA per head took
// 100, bins of 11 bits 40) and the gathering 27 (140 MB in rows of d bytes: 5 TB/s). 2 sequences
// of 517 tokens: 11 us, two launches and their chains of loads.
#include <cuda_fp16.h>

#include "fa_cache8.cuh"

namespace fa {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelCtas = 4;                     // CTAs of a cluster at most
constexpr int kBins = 256;
constexpr int kSelKeys = 49152;                 // keys of a CTA that stay in shared memory (192 KB)
constexpr int kGatherThreads = 64;

__device__ __forceinline__ __half2 as_half2(uint32_t x) {
  __half2 h;
  asm("mov.b32 %0, %1;" : "=r"(reinterpret_cast<uint32_t&>(h)) : "r"(x));
  return h;
}
// Two halves to e4m3 codes, rounded to nearest even, saturating to +-448.
__device__ __forceinline__ uint32_t pack_halves(__half2 x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(reinterpret_cast<uint32_t&>(x)));
  return r;
}

// Blocks that `keep` tokens take up. The gather runs over these alone, however wide to_table is: their
// slots stay within an int, and none but theirs can be written.
__host__ __device__ __forceinline__ int dest_blocks(int keep) { return (keep - 1) / kCacheBlock + 1; }

// Floats as integers of the same order; -0 as 0, NaN above everything.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// All CTAs of the cluster meet; what they wrote before is seen after.
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Address of this CTA's shared memory address `a` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t a, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ int load_cluster(uint32_t a) {
  int v;
  asm volatile("ld.shared::cluster.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ int warp_scan(int x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// Grid (cluster, heads, sequences). `room`: keys that shared memory holds.
__global__ void __launch_bounds__(kSelThreads) cache8_select_kernel(const Cache8EvictParams p, int room) {
  extern __shared__ __align__(16) uint32_t keys[];       // [room] of this CTA's stretch; 0, below all keys, behind it
  __shared__ int hist[2][kBins];
  __shared__ int warp_sum[kBins / 32];
  __shared__ int warp_eq[kSelWarps], warp_above[kSelWarps];
  __shared__ int counts[2];                              // this CTA's: equal, above
  __shared__ uint32_t s_digit;
  __shared__ int s_need;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.z, h = blockIdx.y, rank = blockIdx.x, ctas = gridDim.x;
  let_next();
  wait_before();
  const int n = cache_length(p.lengths, b, p.max_blocks);
  int* const kept = p.kept + (static_cast<size_t>(b) * p.c.Hkv + h) * p.keep;
  const int me = rank * kSelThreads + tid, all = ctas * kSelThreads;
  if (h == 0 && me == 0) p.new_lengths[b] = min(n, p.keep);
  if (n <= p.keep) {                                     // (all CTAs of the cluster)
    // (unsigned: the step past the largest `keep` is no int)
    for (unsigned i = me; i < static_cast<unsigned>(p.keep); i += all) kept[i] = i < static_cast<unsigned>(n) ? static_cast<int>(i) : -1;
    return;
  }
  const int nc = n - p.recent;                           // candidates
  const int need_all = p.keep - p.recent;                // to choose among them, < nc
  for (int i = me; i < p.recent; i += all) kept[need_all + i] = nc + i;
  if (need_all == 0) return;
  // this CTA's stretch [i0, i1), and each warp's: whole blocks of 64 tokens
  const int cta_blocks = (nc + kCacheBlock * ctas - 1) / (kCacheBlock * ctas);
  const int warp_blocks = (cta_blocks + kSelWarps - 1) / kSelWarps;
  const int i0 = min(nc, rank * cta_blocks * kCacheBlock), i1 = min(nc, i0 + cta_blocks * kCacheBlock);
  const int w0 = warp * warp_blocks * kCacheBlock, w1 = min(cta_blocks * kCacheBlock, w0 + warp_blocks * kCacheBlock);
  const int* const table = p.table + static_cast<long long>(b) * p.max_blocks;
  // four keys from token i0 + at on (at a multiple of 4), from memory
  auto keys_at = [&](int at) -> uint4 {
    const int i = i0 + at;
    if (i >= i1) return make_uint4(0, 0, 0, 0);
    const int page = table[i / kCacheBlock];
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f);
    if (page >= 0 && page < p.c.num_blocks)
      w = *reinterpret_cast<const float4*>(p.c.weight + (static_cast<size_t>(page) * p.c.Hkv + h) * kCacheBlock + i % kCacheBlock);
    return make_uint4(order_key(w.x), i + 1 < i1 ? order_key(w.y) : 0u, i + 2 < i1 ? order_key(w.z) : 0u,
                      i + 3 < i1 ? order_key(w.w) : 0u);
  };
  // (a stretch longer than shared memory's room is read again where it does not fit)
  auto keys4 = [&](int at) -> uint4 { return at < room ? *reinterpret_cast<const uint4*>(keys + at) : keys_at(at); };
  const int held = min(room, cta_blocks * kCacheBlock);
  if (tid < kBins) hist[0][tid] = hist[1][tid] = 0;
  __syncthreads();

  // the key of the last one chosen, digit by digit from the top
  uint32_t prefix = 0, mask = 0;
  int need = need_all;
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    int* const bins = hist[(shift >> 3) & 1];
    auto add = [&](const uint4& k4) {
      const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if ((k[e] & mask) == prefix) atomicAdd(&bins[(k[e] >> shift) & 255u], 1);
    };
    int at = tid * 4;
    if (shift == 24) {
#pragma unroll 2
      for (; at < held; at += kSelThreads * 4) {
        const uint4 k4 = keys_at(at);
        *reinterpret_cast<uint4*>(keys + at) = k4;
        add(k4);
      }
    }
    for (; at < cta_blocks * kCacheBlock; at += kSelThreads * 4) add(keys4(at));
    cluster_meet();
    // bins from the largest down, one per thread: the one where the count reaches `need`
    int sum = 0, incl = 0;
    if (tid < kBins) {
      // (the other histogram has been read by all: they were here)
      hist[((shift >> 3) + 1) & 1][tid] = 0;
      const uint32_t mine = smem_addr(&bins[kBins - 1 - tid]);
#pragma unroll
      for (int r = 0; r < kSelCtas; ++r)
        if (r < ctas) sum += load_cluster(in_cta(mine, r));
      incl = warp_scan(sum, lane);
      if (lane == 31) warp_sum[warp] = incl;
    }
    __syncthreads();
    if (tid < kBins) {
#pragma unroll
      for (int w = 0; w < kBins / 32; ++w)
        if (w < warp) incl += warp_sum[w];
      if (incl >= need && incl - sum < need) {           // one thread: at least `need` keys have the prefix
        s_digit = static_cast<uint32_t>(kBins - 1 - tid);
        s_need = need - (incl - sum);
      }
    }
    __syncthreads();
    prefix |= s_digit << shift;
    mask |= 255u << shift;
    need = s_need;
  }

  // keys above `prefix` and those equal to it, of the warps and of the CTAs
  int eq = 0, above = 0;
  for (int at = w0; at < w1; at += 128) {
    const uint4 k4 = at + 4 * lane < w1 ? keys4(at + 4 * lane) : make_uint4(0, 0, 0, 0);
    const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      eq += k[e] == prefix;
      above += k[e] > prefix;
    }
  }
  eq = __reduce_add_sync(0xffffffffu, eq);
  above = __reduce_add_sync(0xffffffffu, above);
  if (lane == 0) {
    warp_eq[warp] = eq;
    warp_above[warp] = above;
  }
  __syncthreads();
  if (warp == 0) {
    const int e = __reduce_add_sync(0xffffffffu, lane < kSelWarps ? warp_eq[lane] : 0);
    const int a = __reduce_add_sync(0xffffffffu, lane < kSelWarps ? warp_above[lane] : 0);
    if (lane == 0) {
      counts[0] = e;
      counts[1] = a;
    }
  }
  cluster_meet();
  int eq_before = 0, above_before = 0;
#pragma unroll
  for (int r = 0; r < kSelCtas; ++r)
    if (r < rank) {
      eq_before += load_cluster(in_cta(smem_addr(&counts[0]), r));
      above_before += load_cluster(in_cta(smem_addr(&counts[1]), r));
    }
#pragma unroll
  for (int w = 0; w < kSelWarps; ++w)
    if (w < warp) {
      eq_before += warp_eq[w];
      above_before += warp_above[w];
    }
  // chosen: all above, and the equal ones within the first `need`; positions in order
  for (int at = w0; at < w1; at += 128) {
    const int mine = at + 4 * lane;
    const uint4 k4 = mine < w1 ? keys4(mine) : make_uint4(0, 0, 0, 0);
    const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
    int e4 = 0, a4 = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      e4 += k[e] == prefix;
      a4 += k[e] > prefix;
    }
    // both counts in one scan: at most 128 of each
    const int both = warp_scan(e4 | a4 << 16, lane);
    int eqs = eq_before + (both & 0xffff) - e4, aboves = above_before + (both >> 16) - a4;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool same = k[e] == prefix, over = k[e] > prefix;
      if (over || (same && eqs < need)) kept[aboves + min(eqs, need)] = i0 + mine + e;
      eqs += same;
      aboves += over;
    }
    const int last = __shfl_sync(0xffffffffu, both, 31);
    eq_before += last & 0xffff;
    above_before += last >> 16;
  }
  cluster_meet();                                        // until the others have read this CTA's counts
}

// D: 128 or 256, d at most that.
template <int D>
__global__ void __launch_bounds__(kGatherThreads, D == 128 ? 18 : 8) cache8_gather_kernel(const Cache8EvictParams p) {
  constexpr int kMaxChunks = kCacheBlock * D / 16 / kGatherThreads;    // 16-code chunks per thread
  __shared__ float warp_max[kGatherThreads / 32];
  __shared__ long long src[kCacheBlock];          // (block * Hkv + h) * 64 + slot of a kept token, -1: no such block
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int blocks = dest_blocks(p.keep), b = blockIdx.x / blocks, blk = blockIdx.x - b * blocks;
  const int h = blockIdx.y, which = blockIdx.z;
  let_next();
  wait_before();
  // (one round of loads for all three)
  const int n = cache_length(p.lengths, b, p.max_blocks);
  const int page = p.to_table[static_cast<long long>(b) * p.to_blocks + blk];
  const int slot = blk * kCacheBlock + tid;
  const int i = tid < kCacheBlock && slot < p.keep ? p.kept[(static_cast<size_t>(b) * p.c.Hkv + h) * p.keep + slot] : -1;
  const int cnt = min(kCacheBlock, min(n, p.keep) - blk * kCacheBlock);
  if (cnt <= 0 || page < 0 || page >= p.c.num_blocks) return;
  const size_t ph = static_cast<size_t>(page) * p.c.Hkv + h;
  if (tid < cnt) {
    const int from = p.table[static_cast<long long>(b) * p.max_blocks + i / kCacheBlock];
    const bool ok = from >= 0 && from < p.c.num_blocks;
    const long long at = (static_cast<long long>(from) * p.c.Hkv + h) * kCacheBlock + i % kCacheBlock;
    src[tid] = ok ? at : -1;
    if (which == 0) p.c.weight[ph * kCacheBlock + tid] = ok ? p.c.weight[at] : 0.f;
  }
  __syncthreads();
  const uint8_t* const codes = which ? p.c.v : p.c.k;
  float* const scales = which ? p.c.v_scale : p.c.k_scale;
  const int cpr = p.c.d / 16;                     // chunks per token
  // this thread's chunks: tid, tid + kGatherThreads, ... as (row, column)
  const int drow = kGatherThreads / cpr, dcol = kGatherThreads - drow * cpr;
  uint4 val[kMaxChunks];
  float sc[kMaxChunks];
  int row = tid / cpr, col = tid - row * cpr;
#pragma unroll
  for (int k = 0; k < kMaxChunks; ++k) {
    val[k] = make_uint4(0, 0, 0, 0);
    sc[k] = 0.f;
    if (row < cnt) {
      const long long at = src[row];
      if (at >= 0) {
        val[k] = *reinterpret_cast<const uint4*>(codes + at * p.c.d + col * 16);
        sc[k] = scales[at / kCacheBlock];
      }
    }
    row += drow;
    col += dcol;
    if (col >= cpr) {
      col -= cpr;
      ++row;
    }
  }
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < kMaxChunks; ++k) {
    // the largest magnitude of 16 codes, as halves, exact; a maximum passes over NaN
    const uint32_t w[4] = {val[k].x, val[k].y, val[k].z, val[k].w};
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) m = __vimax3_u16x2(m, w[e] & 0x7F007F00u, (w[e] << 8) & 0x7F007F00u);
    m = max(m & 0xFFFFu, m >> 16) >> 8;
    if (m == 0x7Fu) {
      m = 0;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const uint32_t code = (w[e / 4] >> (8 * (e % 4))) & 0x7Fu;
        m = max(m, code == 0x7Fu ? 0u : code);
      }
    }
    // (rounded up: above 448 times a power of two if and only if the exact product is)
    amax = fmaxf(amax, __fmul_ru(e4m3x2_to_float2(m).x, sc[k]));
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
    if (c >= cnt * cpr) continue;
    const uint32_t w[4] = {val[k].x, val[k].y, val[k].z, val[k].w};
    uint32_t r[4];
    const float ratio = sc[k] * inv;
    // Scales that are powers of two, as fa_cache8_append makes them: the codes as halves
    // times the ratio, exact down to 2^-24, where every code has long become 0.
    if ((__float_as_uint(ratio) & 0x807FFFFFu) == 0 && ratio >= 0x1p-14f && ratio <= 0x1p15f) {
      const __half2 f = __float2half2_rn(ratio);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        r[e] = pack_halves(__hmul2(as_half2(e4m3x2_to_f16x2(w[e])), f)) |
               pack_halves(__hmul2(as_half2(e4m3x2_to_f16x2(w[e] >> 16)), f)) << 16;
    } else {
      // the ratio is exact, or so small that every code becomes 0, or past all floats where every code is 0
      const float f = fminf(ratio, 0x1p127f);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 a = e4m3x2_to_float2(w[e]), z = e4m3x2_to_float2(w[e] >> 16);
        r[e] = pack_e4m3x2(a.x * f, a.y * f) | pack_e4m3x2(z.x * f, z.y * f) << 16;
      }
    }
    *reinterpret_cast<uint4*>(dst + c * 16) = make_uint4(r[0], r[1], r[2], r[3]);
  }
}

}  // namespace

cudaError_t launch_cache8_evict(const Cache8EvictParams& p, cudaStream_t stream) {
  // One CTA per (sequence, head) or a cluster of four, whichever fills the SMs. Both kernels, us, one / four / eight:
  // 16 of them, 2048 tokens 11.3 / 11.3 / 13.7, 4608 13.9 / 11.8 / 14.8, 32768 40 / 22 / 23;
  // 64, 4608 17 / 18 / 22, 8192 24 / 20 / 25, 32768 72 / 56 / 57; 256, 8192 56 / 64 / 91, 16384 115 / 105 / 127.
  const bool many = static_cast<long long>(p.B) * p.c.Hkv > kCache8Sms;
  const int ctas = p.max_blocks > (many ? 128 : 64) ? kSelCtas : 1;
  const int most = (p.max_blocks + ctas - 1) / ctas;     // blocks per CTA, more than it will have
  const int room = most < kSelKeys / kCacheBlock ? most * kCacheBlock : kSelKeys;
  static PerDeviceOnce attr;
  cudaError_t e = attr.run([] {
    return cudaFuncSetAttribute(cache8_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelKeys * 4);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas, p.c.Hkv, p.B);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(room) * 4;
  cfg.stream = stream;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = ctas;
  attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, cache8_select_kernel, p, room);
  if (e != cudaSuccess) return e;
  return launch_early(p.c.d > 128 ? cache8_gather_kernel<256> : cache8_gather_kernel<128>,
                      dim3(p.B * dest_blocks(p.keep), p.c.Hkv, 2), dim3(kGatherThreads), 0, stream, p);
}

}  // namespace fa
