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
//
// With rotation K's pairs of columns are turned by their positions on the way, in fp32, and the block's scale is that of the
// rotated values, so K is rounded once. The angles are the same for all heads of a token: a CTA computes them once for
// several. K's kernel then has 60% of the issue slots busy (about 20 instructions per value) and 2.1 waves of CTAs.
#include "fa_cache8.cuh"
#include "fa_rope.cuh"

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

// The codes of a block's tokens [0, lo) when its scale grows, eight at a time.
__device__ __forceinline__ void rescale_codes(uint8_t* codes, int chunks, float ratio, int tid, int threads) {
  for (int c = tid; c < chunks; c += threads) {
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

// Where a CTA's block lies: slots [lo, hi) of page `page` get the tokens from tok0 on; the first is position pos0.
struct NewTokens {
  int lo, hi, tok0, pos0, page;
};

// K, and with kBoth V, of one block for heads [h0, h1), each pair of K's columns turned by its angle on the way. A thread has
// four pairs (eight columns) of up to kUnits tokens; their cosines and sines are computed once, kept in shared
// memory where it has only this thread's, and serve all its heads. The rotated values stay in fp32 until they are codes. The
// next head's loads are under way meanwhile.
template <int D, int N, bool kBoth, bool kApart>
__device__ __forceinline__ void append_rotated(const Cache8AppendParams& p, const NewTokens& n, int h0, int h1, float2 (*warp_max)[N / 32], float4* table) {
  constexpr int kUnits = kCacheBlock * D / 8 / N;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int upt = p.c.d / 8, slots = N / upt;               // units of a token, tokens at a time
  const int slot = tid / upt, c = tid - slot * upt;
  const bool turned = 4 * c < p.rope.pairs;
  // kApart: a pair's columns lie p.rope.pairs apart; otherwise, and behind the pairs, the thread's eight side by side
  const int ca = kApart && turned ? 4 * c : 8 * c, cb = kApart && turned ? ca + p.rope.pairs : ca + 4;
  const int count = n.hi - n.lo;
  auto row_of = [&](int i) { return slot + i * slots; };
  auto mine = [&](int i) { return slot < slots && row_of(i) < count; };
  uint2 raw[kUnits][2];
  uint4 raw_v[kBoth ? kUnits : 1];
  const __nv_bfloat16* next_k = static_cast<const __nv_bfloat16*>(p.k) + h0 * p.k_sh + static_cast<long long>(n.tok0 + slot) * p.k_st;
  const __nv_bfloat16* next_v = static_cast<const __nv_bfloat16*>(p.v) + h0 * p.v_sh + static_cast<long long>(n.tok0 + slot) * p.v_st + 8 * c;
  const long long step_k = slots * p.k_st, step_v = slots * p.v_st;
  auto load = [&]() {                                        // the next head's
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      raw[i][0] = raw[i][1] = make_uint2(0, 0);
      if (kBoth) raw_v[kBoth ? i : 0] = make_uint4(0, 0, 0, 0);
      if (mine(i)) {
        raw[i][0] = *reinterpret_cast<const uint2*>(next_k + i * step_k + ca);
        raw[i][1] = *reinterpret_cast<const uint2*>(next_k + i * step_k + cb);
        if (kBoth) raw_v[kBoth ? i : 0] = *reinterpret_cast<const uint4*>(next_v + i * step_v);
      }
    }
    next_k += p.k_sh;
    next_v += p.v_sh;
  };
  load();
  unsigned long long turns[4] = {0, 0, 0, 0};
  const int* at[4] = {nullptr, nullptr, nullptr, nullptr};
  if (turned) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      turns[e] = static_cast<unsigned long long>(p.rope.turns[4 * c + e]);
      const int axis = p.rope.axis == nullptr ? 0 : max(0, min(p.rope.axis[4 * c + e], p.rope.axes - 1));
      if (p.rope.positions != nullptr) at[e] = p.rope.positions + axis * p.rope.pos_sa + n.tok0;
    }
  }
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    float2 cs[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      int pos = n.pos0 + row_of(i);
      if (at[e] != nullptr && mine(i)) pos = at[e][row_of(i)];
      cs[e] = cos_sin_turns(turns[e], pos);
    }
    table[(2 * i) * N + tid] = make_float4(cs[0].x, cs[1].x, cs[2].x, cs[3].x);
    table[(2 * i + 1) * N + tid] = make_float4(cs[0].y, cs[1].y, cs[2].y, cs[3].y);
  }
  if (n.page < 0 || n.page >= p.c.num_blocks) return;
  for (int h = h0; h < h1; ++h) {
    const size_t ph = static_cast<size_t>(n.page) * p.c.Hkv + h;
    uint8_t* const codes = p.c.k + ph * kCacheBlock * p.c.d;
    uint8_t* const codes_v = p.c.v + ph * kCacheBlock * p.c.d;
    // read before the barrier, written after it
    const float old = n.lo > 0 ? p.c.k_scale[ph] : 0.f, old_v = kBoth && n.lo > 0 ? p.c.v_scale[ph] : 0.f;
    float fa[kUnits][4], fb[kUnits][4];                     // the first and the second columns of the four pairs
    uint4 v[kBoth ? kUnits : 1];
    float2 amax = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      const uint32_t w[4] = {raw[i][0].x, raw[i][0].y, raw[i][1].x, raw[i][1].y};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float lower = __uint_as_float(w[e] << 16), upper = __uint_as_float(w[e] & 0xFFFF0000u);
        if (kApart) {
          (e < 2 ? fa : fb)[i][2 * (e & 1)] = lower;
          (e < 2 ? fa : fb)[i][2 * (e & 1) + 1] = upper;
        } else {
          fa[i][e] = lower;
          fb[i][e] = upper;
        }
      }
      if (turned) {
        const float4 co = table[(2 * i) * N + tid], si = table[(2 * i + 1) * N + tid];
        rotate2(fa[i][0], fa[i][1], fb[i][0], fb[i][1], co.x, co.y, si.x, si.y);
        rotate2(fa[i][2], fa[i][3], fb[i][2], fb[i][3], co.z, co.w, si.z, si.w);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) amax.x = fmaxf(amax.x, fmaxf(fabsf(fa[i][e]), fabsf(fb[i][e])));   // (NaN are left out)
      if (kBoth) v[kBoth ? i : 0] = raw_v[kBoth ? i : 0];
    }
    if (!(amax.x < INFINITY)) {                             // an infinity: the largest of the others
      amax.x = 0.f;
#pragma unroll
      for (int i = 0; i < kUnits; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = fabsf(fa[i][e]), y = fabsf(fb[i][e]);
          amax.x = fmaxf(amax.x, fmaxf(x < INFINITY ? x : 0.f, y < INFINITY ? y : 0.f));
        }
    }
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < (kBoth ? kUnits : 0); ++i) top = max2(top, v[i]);
    top = max(top & 0xFFFFu, top >> 16);
    if (kBoth && top >= 0x7F80u) {
      top = 0;
      for (int i = 0; i < (kBoth ? kUnits : 0); ++i) top = finite_max(finite_max(finite_max(finite_max(top, v[i].x), v[i].y), v[i].z), v[i].w);
    }
    if (h + 1 < h1) load();
    // (non-negative floats order like their bits)
    amax.x = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax.x)));
    if (kBoth) amax.y = __uint_as_float(__reduce_max_sync(0xffffffffu, top << 16));
    float2* const maxima = warp_max[(h - h0) & 1];          // (the other buffer may still be read for the head before)
    if (lane == 0) maxima[warp] = amax;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < N / 32; ++w) {
      amax.x = fmaxf(amax.x, maxima[w].x);
      amax.y = fmaxf(amax.y, maxima[w].y);
    }
    auto grown = [&](float before, float most) {
      const float s = fmaxf(before, power_scale(most));
      return s > 0.f ? s : 1.f;
    };
    const float now = grown(old, amax.x), now_v = grown(old_v, amax.y);
    if (n.lo > 0 && now != old) rescale_codes(codes, n.lo * upt, __fdiv_rn(old, now), tid, N);
    if (kBoth && n.lo > 0 && now_v != old_v) rescale_codes(codes_v, n.lo * upt, __fdiv_rn(old_v, now_v), tid, N);
    if (tid == 0) {
      p.c.k_scale[ph] = now;
      if (kBoth) p.c.v_scale[ph] = now_v;
    }
    // powers of two, as all made here are (2^126 at most): 1 / now is exact, and its exponent the other's opposite
    auto is_power = [](float s) { return (__float_as_uint(s) & 0x7FFFFFu) == 0 && s < 1.7014118e38f; };
    const bool power = is_power(now), power_v = is_power(now_v);
    const float inv = __uint_as_float(0x7F000000u - __float_as_uint(now)), inv_v = __uint_as_float(0x7F000000u - __float_as_uint(now_v));
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
      if (!mine(i)) continue;
      if (power) {
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          mul2_bc(fa[i][e], fa[i][e + 1], inv);
          mul2_bc(fb[i][e], fb[i][e + 1], inv);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          fa[i][e] = __fdiv_rn(fa[i][e], now);
          fb[i][e] = __fdiv_rn(fb[i][e], now);
        }
      }
      const int at = (n.lo + row_of(i)) * p.c.d;
      uint32_t first, second;
      if (kApart) {
        first = pack_e4m3x2(fa[i][0], fa[i][1]) | pack_e4m3x2(fa[i][2], fa[i][3]) << 16;
        second = pack_e4m3x2(fb[i][0], fb[i][1]) | pack_e4m3x2(fb[i][2], fb[i][3]) << 16;
      } else {
        first = pack_e4m3x2(fa[i][0], fb[i][0]) | pack_e4m3x2(fa[i][1], fb[i][1]) << 16;
        second = pack_e4m3x2(fa[i][2], fb[i][2]) | pack_e4m3x2(fa[i][3], fb[i][3]) << 16;
      }
      *reinterpret_cast<uint32_t*>(codes + at + ca) = first;
      *reinterpret_cast<uint32_t*>(codes + at + cb) = second;
      if (kBoth) *reinterpret_cast<uint2*>(codes_v + at + 8 * c) = power_v ? encode8(v[kBoth ? i : 0], inv_v) : divide8(v[kBoth ? i : 0], now_v);
    }
    if (p.c.weight != nullptr && tid < count) p.c.weight[ph * kCacheBlock + n.lo + tid] = 0.f;
  }
}

// D: 128 or 256, d at most that. kRotate 0: one CTA of kThreads per (touched block, KV head, K or V; V alone where K is
// rotated). 1: K rotated, one CTA of N threads per block and `heads` KV heads. 2: V too, as it is. 5 and 6: the same for pairs
// side by side.
template <int D, int kRotate, int N>
__global__ void __launch_bounds__(N, kRotate == 0 ? (D == 128 ? 8 : 4) : (kRotate & 1) && D == 128 ? 3 : 512 / N) cache8_append_kernel(const Cache8AppendParams p) {
  constexpr int kThreads = N;
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
  if constexpr (kRotate > 0) {
    __shared__ float2 maxima[2][N / 32];
    const int h0 = static_cast<int>(blockIdx.y) * p.heads;
    const NewTokens n{lo, hi, tok0, blk * kCacheBlock + lo, p.table[static_cast<long long>(b) * p.max_blocks + blk]};
    extern __shared__ float4 table[];
    append_rotated<D, N, (kRotate & 2) != 0, kRotate < 4>(p, n, h0, min(h0 + p.heads, p.c.Hkv), maxima, table);
    return;
  }
  const int h = blockIdx.y, which = p.rope.pairs > 0 ? 1 : blockIdx.z;
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
    // the tokens there, by the ratio of the scales
    rescale_codes(codes, lo * cpr, __fdiv_rn(old, now), tid, kThreads);
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

template <int D, int kRotate, int N>
static cudaError_t rotate_as(const Cache8AppendParams& p, unsigned items, cudaStream_t stream) {
  constexpr int kTable = 2 * ((kCacheBlock * D / 8 + N - 1) / N) * N * static_cast<int>(sizeof(float4));
  static PerDeviceOnce attr;
  const cudaError_t e = attr.run([] {
    return cudaFuncSetAttribute(cache8_append_kernel<D, kRotate, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTable);
  });
  if (e != cudaSuccess) return e;
  return launch_early(cache8_append_kernel<D, kRotate, N>, dim3(items, (p.c.Hkv + p.heads - 1) / p.heads), dim3(N), kTable, stream, p);
}

// kRotate 1 or 2
template <int D, int kRotate, int N>
static cudaError_t rotating(const Cache8AppendParams& p, unsigned items, cudaStream_t stream) {
  return p.rope.interleaved ? rotate_as<D, kRotate + 4, N>(p, items, stream) : rotate_as<D, kRotate, N>(p, items, stream);
}

cudaError_t launch_cache8_append(const Cache8AppendParams& p, cudaStream_t stream) {
  // n tokens touch at most (n + 126) / 64 blocks of a sequence, and no more than n
  const long long most = (static_cast<long long>(p.T) + 126LL * p.B) / kCacheBlock;
  const unsigned items = static_cast<unsigned>(most < p.T ? most : p.T);
  const bool wide = p.c.d > 128;
  auto plain = [&](int z) {
    return launch_early(wide ? cache8_append_kernel<256, 0, kThreads> : cache8_append_kernel<128, 0, kThreads>, dim3(items, p.c.Hkv, z),
                        dim3(kThreads), 0, stream, p);
  };
  if (p.rope.pairs == 0) return plain(2);
  Cache8AppendParams r = p;
  if (static_cast<long long>(items) * p.c.Hkv <= 1216) {
    // few blocks (a decoding step): K and V of a head together, in one launch
    r.heads = 1;
    return wide ? rotating<256, 2, 512>(r, items, stream) : rotating<128, 2, 256>(r, items, stream);
  }
  // Many: V by the kernel that has nothing else to do, eight CTAs per SM, and K by one whose registers are few enough for
  // three, four heads to a CTA, for which the angles are computed once. (30011 tokens of 8 heads, d 128: 49 us, with two
  // heads to a CTA 51, with eight 53; K and V together at two CTAs per SM 64.)
  const cudaError_t e = plain(1);
  if (e != cudaSuccess) return e;
  r.heads = 4;
  return wide ? rotating<256, 1, 512>(r, items, stream) : rotating<128, 1, 256>(r, items, stream);
}

}  // namespace fa
