// Rotary positions for Q and K in one launch: each pair of columns of a head's
// vector turned by position * frequency, or back (the gradient, since a rotation's
// transpose is its inverse).
//
// HBM-bound: every value is read once and written once. A CTA takes a few tokens and all
// their heads: the tokens' cosines and sines are computed once (about 30
// instructions each, one per thread) into shared memory and serve Hq + Hkv heads. A
// thread holds both columns of its pairs (two 16-byte vectors where a pair's columns lie
// pairs apart), so the result may go where the input was.
#include "fa_rope.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 4;                  // rows whose loads a thread has under way together
constexpr int kRopeCtas = 4 * 152;        // fewer leave SMs idle

// E values of a row as fp32.
template <typename T, int E>
struct Vec {
  static constexpr int kWords = E * static_cast<int>(sizeof(T)) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWords == 4) {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      w[0] = u.x;
      w[1] = u.y;
      w[2] = u.z;
      w[3] = u.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      w[0] = u.x;
      w[1] = u.y;
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kWords == 4)
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
  __device__ __forceinline__ void get(float (&f)[E]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = __uint_as_float(w[e]);
    } else {
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        f[2 * e] = __uint_as_float(w[e] << 16);
        f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
      }
    }
  }
  __device__ __forceinline__ void set(const float (&f)[E]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < E; ++e) w[e] = __float_as_uint(f[e]);
    } else {
#pragma unroll
      for (int e = 0; e < E / 2; ++e) w[e] = pack_bf16x2(f[2 * e], f[2 * e + 1]);   // one rounding, to nearest
    }
  }
};

// kAdjacent: 0 pairs are columns i and i + pairs, 1 columns 2 i and 2 i + 1. threadIdx.x: unit of a row (rotated
// vectors, or pairs of them, then the vectors behind them); threadIdx.y: row.
template <typename T, int E, int kAdjacent>
__global__ void __launch_bounds__(kThreads, 4) rope_kernel(const RopeParams p) {
  constexpr int kP = kAdjacent ? E / 2 : E;              // pairs of a unit
  extern __shared__ float2 table[];                      // [token][kP][units]: neighbouring threads read neighbouring entries
  const int units = p.rope.pairs / kP;
  const int tiles = (p.T + p.tokens - 1) / p.tokens;
  const int b = static_cast<int>(blockIdx.x) / tiles;
  const int t0 = (static_cast<int>(blockIdx.x) - b * tiles) * p.tokens;
  const int tokens = min(p.tokens, p.T - t0);
  const int h0 = blockIdx.y * p.heads, heads = min(p.heads, p.x[0].H + p.x[1].H - h0);
  const int u = threadIdx.x, slots = blockDim.y;
  const bool turned = u < units;
  const int ca = turned ? u * E : 2 * p.rope.pairs + (u - units) * E;   // the unit's columns
  const int cb = ca + p.rope.pairs;

  auto angles = [&]() {
    const int n = tokens * p.rope.pairs;
    for (int i = threadIdx.y * blockDim.x + u; i < n; i += blockDim.x * slots) {
      const int t = i / p.rope.pairs, pair = i - t * p.rope.pairs;
      float2 cs = rope_at(p.rope, pair, b, t0 + t);
      if (p.inverse) cs.y = -cs.y;
      table[(t * kP + pair % kP) * units + pair / kP] = cs;
    }
  };

  // this thread's rows: (token, head) in the order of memory, `slots` apart
  const int rows = tokens * heads, step_t = slots / heads, step_h = slots - step_t * heads;
  int t = threadIdx.y / heads, h = threadIdx.y - t * heads;
  bool first = true;
  for (int row = threadIdx.y; first || row < rows; row += kRows * slots) {
    Vec<T, E> va[kRows], vb[kRows];
    T* dst[kRows];
    int tt[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      tt[i] = t;
      dst[i] = nullptr;
      if (row + i * slots < rows) {
        const int head = h0 + h;
        const bool is_k = head >= p.x[0].H;
        const RopeTensor& x = p.x[is_k ? 1 : 0];
        const int hx = is_k ? head - p.x[0].H : head;
        const T* const src = static_cast<const T*>(x.in) + b * x.in_sb + hx * x.in_sh + (t0 + t) * x.in_st;
        T* const out = static_cast<T*>(x.out) + b * x.out_sb + hx * x.out_sh + (t0 + t) * x.out_st;
        if (turned || src != out) {                      // (in place, the columns behind the pairs are there)
          dst[i] = out;
          va[i].load(src + ca);
          if (!kAdjacent && turned) vb[i].load(src + cb);
        }
      }
      t += step_t;
      h += step_h;
      if (h >= heads) {
        h -= heads;
        ++t;
      }
    }
    if (first) {                                         // (while the first rows are on their way)
      angles();
      __syncthreads();
      first = false;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      if (dst[i] == nullptr) continue;
      if (turned) {
        const float2* const cs = table + tt[i] * p.rope.pairs + u;
        float a[E], c[E];
        va[i].get(a);
        if (kAdjacent) {
#pragma unroll
          for (int e = 0; e < kP; ++e) rotate(a[2 * e], a[2 * e + 1], cs[e * units]);
        } else {
          vb[i].get(c);
#pragma unroll
          for (int e = 0; e < kP; ++e) rotate(a[e], c[e], cs[e * units]);
          vb[i].set(c);
          vb[i].store(dst[i] + cb);
        }
        va[i].set(a);
      }
      va[i].store(dst[i] + ca);
    }
  }
}

template <typename T, int E, int kAdjacent>
cudaError_t launch(RopeParams p, cudaStream_t stream) {
  constexpr int kP = kAdjacent ? E / 2 : E;
  const int units = p.rope.pairs / kP + (p.d - 2 * p.rope.pairs) / E;
  const int slots = kThreads / units, all = p.x[0].H + p.x[1].H;
  // One cosine and sine per thread where tokens are many; where they are few, a CTA per token
  // and as many heads as it has rows of threads.
  const int most = kThreads / p.rope.pairs > 1 ? kThreads / p.rope.pairs : 1;
  const long long n = static_cast<long long>(p.B) * p.T;
  p.tokens = most;
  p.heads = all;
  while (p.tokens > 1 && (n + p.tokens - 1) / p.tokens < kRopeCtas) p.tokens /= 2;
  if (p.tokens == 1 && n < kRopeCtas && all > slots) p.heads = slots;
  const long long ctas = static_cast<long long>(p.B) * ((p.T + p.tokens - 1) / p.tokens);
  rope_kernel<T, E, kAdjacent><<<dim3(static_cast<unsigned>(ctas), (all + p.heads - 1) / p.heads), dim3(units, slots),
                                 static_cast<size_t>(p.tokens) * p.rope.pairs * sizeof(float2), stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(int elt_bytes, const RopeParams& p, cudaStream_t stream) {
  if (elt_bytes == 4) return p.rope.interleaved ? launch<float, 4, 1>(p, stream) : launch<float, 4, 0>(p, stream);
  if (p.rope.interleaved) return launch<__nv_bfloat16, 8, 1>(p, stream);
  return p.rope.pairs % 8 == 0 ? launch<__nv_bfloat16, 8, 0>(p, stream) : launch<__nv_bfloat16, 4, 0>(p, stream);
}

}  // namespace fa
