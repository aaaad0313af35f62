// Writing the 8-bit cache: bf16 K and V tokens of several sequences appended
// as e4m3 codes with one scale per block of 64 tokens and KV head.
//
// code = e4m3(x / s), s the smallest power of two that holds the block's
// largest magnitude within 448. When a block that already holds tokens gets a
// larger one, its scale grows and the codes there are re-encoded by the ratio
// (a power of two). HBM-bound: each new value is read once (2 bytes) and
// written once (1 byte). One CTA of 128 threads per block, head and K or V, eight
// 16-byte loads in flight per thread; 256 threads with four each spent a third more
// instructions on finding their block (35 us). 30011 tokens of 8 heads, d 128: 31 us, 6.0 TB/s;
// one token each for 64 sequences 5.3 us, which is the launch and two rounds of loads. Every CTA looks through
// the sequences 32 at a time: 256 sequences take 21 us, 1024 131, 4096 1475.
#include "fa_cache8.cuh"

namespace fa {
namespace {

constexpr int kThreads = 128;

// Largest finite magnitude of two bf16; infinities and NaN are left out.
__device__ __forceinline__ uint32_t finite_max(uint32_t m, uint32_t x) {
  const uint32_t lo = x & 0x7FFFu, hi = (x >> 16) & 0x7FFFu;
  m = max(m, lo < 0x7F80u ? lo : 0u);
  return max(m, hi < 0x7F80u ? hi : 0u);
}
// Largest magnitudes of the lower and of the upper halves of eight bf16 and m; NaN are left out.
__device__ __forceinline__ uint32_t max2(uint32_t m, const uint4& x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[e] & 0x7FFF7FFFu));
  return m;
}

__device__ __forceinline__ uint2 encode8(const uint4& x, float inv) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t q[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    q[e] = pack_e4m3x2(__uint_as_float(w[e] << 16) * inv, __uint_as_float(w[e] & 0xFFFF0000u) * inv);
  return make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
}

// The same where the scale is no power of two, a held one of the caller's: x / s rounded once to fp32, then to
// the code. (1 / s would round twice, and is infinite for the smallest s.) A call, so that its divisions stay out of the way.
__device__ __noinline__ uint2 divide8(uint4 x, float s) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t q[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    q[e] = pack_e4m3x2(__fdiv_rn(__uint_as_float(w[e] << 16), s), __fdiv_rn(__uint_as_float(w[e] & 0xFFFF0000u), s));
  return make_uint2(q[0] | q[1] << 16, q[2] | q[3] << 16);
}

// One CTA per (touched block, KV head, K or V). D: 128 or 256, d at most that.
template <int D>
__global__ void __launch_bounds__(kThreads, D == 128 ? 8 : 4) cache8_append_kernel(const Cache8AppendParams p) {
  constexpr int kMaxChunks = kCacheBlock * D / 8 / kThreads;   // 16-byte chunks of one block per thread
  __shared__ float warp_max[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  let_next();
  wait_before();
  const long long cap = static_cast<long long>(p.max_blocks) * kCacheBlock;
  // Tokens [a, e) of sequence b go to positions from s on. Every warp looks for the
  // CTA's block by itself: one round of loads, and no barrier before the next.
  int b = -1, blk = 0, a = 0, e = 0, s = 0;
  for (int b0 = 0, base = 0; b0 < p.B && b < 0; b0 += 32) {
    int cnt = 0, first = 0;
    if (b0 + lane < p.B) {
      a = max(0, min(p.cu[b0 + lane], p.T));
      e = max(a, min(p.cu[b0 + lane + 1], p.T));
      s = static_cast<int>(max(0LL, min(static_cast<long long>(p.start[b0 + lane]), cap)));
      e = static_cast<int>(min(static_cast<long long>(e), a + (cap - s)));  // behind the table's end: not written
      first = s / kCacheBlock;
      if (e > a) cnt = (s + (e - a) - 1) / kCacheBlock - first + 1;
    }
    int incl = cnt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const int i = static_cast<int>(blockIdx.x) - base;
    const unsigned hit = __ballot_sync(0xffffffffu, i < incl);
    if (hit) {
      const int src = __ffs(hit) - 1;
      b = b0 + src;
      blk = __shfl_sync(0xffffffffu, first + i - (incl - cnt), src);
      a = __shfl_sync(0xffffffffu, a, src);
      e = __shfl_sync(0xffffffffu, e, src);
      s = __shfl_sync(0xffffffffu, s, src);
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  if (b < 0) return;
  const int lo = max(0, s - blk * kCacheBlock);
  const int hi = min(kCacheBlock, s + (e - a) - blk * kCacheBlock);
  const int tok0 = a + (blk * kCacheBlock + lo - s);
  const int h = blockIdx.y, which = blockIdx.z;
  const int cpr = p.c.d / 8;                                  // chunks of eight values per token
  const int chunks = (hi - lo) * cpr;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(which ? p.v : p.k) +
                           h * (which ? p.v_sh : p.k_sh);
  const long long st = which ? p.v_st : p.k_st;
  const int page = p.table[static_cast<long long>(b) * p.max_blocks + blk];   // (needed after the values)

  uint4 val[kMaxChunks];
  // this thread's chunks: tid, tid + kThreads, ... as (row, column)
  const int drow = kThreads / cpr, dcol = kThreads - drow * cpr;
  int row = tid / cpr, col = tid - row * cpr;
#pragma unroll
  for (int i = 0; i < kMaxChunks; ++i) {
    val[i] = row < hi - lo ? *reinterpret_cast<const uint4*>(x + (tok0 + row) * st + col * 8) : make_uint4(0, 0, 0, 0);
    row += drow;
    col += dcol;
    if (col >= cpr) {
      col -= cpr;
      ++row;
    }
  }
  if (page < 0 || page >= p.c.num_blocks) return;
  const size_t ph = static_cast<size_t>(page) * p.c.Hkv + h;
  uint8_t* codes = (which ? p.c.v : p.c.k) + ph * kCacheBlock * p.c.d;
  float* scale = (which ? p.c.v_scale : p.c.k_scale) + ph;
  const float old = lo > 0 ? *scale : 0.f;                    // read before the barrier, written after it
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kMaxChunks; ++i) top = max2(top, val[i]);
  top = max(top & 0xFFFFu, top >> 16);
  if (top >= 0x7F80u) {                                       // an infinity: the largest of the others
    top = 0;
    for (int i = 0; i < kMaxChunks; ++i) top = finite_max(finite_max(finite_max(finite_max(top, val[i].x), val[i].y), val[i].z), val[i].w);
  }
  float amax = __uint_as_float(top << 16);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if (lane == 0) warp_max[warp] = amax;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) amax = fmaxf(amax, warp_max[w]);
  float now = fmaxf(old, power_scale(amax));
  if (!(now > 0.f)) now = 1.f;
  if (lo > 0 && now != old) {
    // the tokens there, 8 codes at a time, by the ratio of the scales
    const float ratio = __fdiv_rn(old, now);
    for (int c = tid; c < lo * cpr; c += kThreads) {
      uint2 w = *reinterpret_cast<const uint2*>(codes + c * 8);
      uint32_t r[4] = {w.x & 0xFFFFu, w.x >> 16, w.y & 0xFFFFu, w.y >> 16};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = e4m3x2_to_float2(r[k]);
        r[k] = pack_e4m3x2(f.x * ratio, f.y * ratio);
      }
      *reinterpret_cast<uint2*>(codes + c * 8) = make_uint2(r[0] | r[1] << 16, r[2] | r[3] << 16);
    }
  }
  if (tid == 0) *scale = now;
  if ((__float_as_uint(now) & 0x7FFFFFu) == 0) {                              // a normal power of two, as all made here are: 1 / now is exact
    const float inv = __fdiv_rn(1.f, now);
#pragma unroll
    for (int i = 0; i < kMaxChunks; ++i) {
      const int c = tid + i * kThreads;
      if (c < chunks) *reinterpret_cast<uint2*>(codes + (lo * cpr + c) * 8) = encode8(val[i], inv);
    }
  } else {
#pragma unroll
    for (int i = 0; i < kMaxChunks; ++i) {
      const int c = tid + i * kThreads;
      if (c < chunks) *reinterpret_cast<uint2*>(codes + (lo * cpr + c) * 8) = divide8(val[i], now);
    }
  }
  if (which == 0 && p.c.weight != nullptr && lo + tid < hi) p.c.weight[ph * kCacheBlock + lo + tid] = 0.f;
}

}  // namespace

cudaError_t launch_cache8_append(const Cache8AppendParams& p, cudaStream_t stream) {
  // n tokens touch at most (n + 126) / 64 blocks of a sequence, and no more than n
  const long long most = (static_cast<long long>(p.T) + 126LL * p.B) / kCacheBlock;
  const unsigned items = static_cast<unsigned>(most < p.T ? most : p.T);
  return launch_early(p.c.d > 128 ? cache8_append_kernel<256> : cache8_append_kernel<128>, dim3(items, p.c.Hkv, 2), dim3(kThreads), 0, stream, p);
}

}  // namespace fa
