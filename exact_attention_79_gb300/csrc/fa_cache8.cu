// Attention of a few new queries per sequence over the 8-bit block cache.
//
// For sequence b, KV head h the R = (Hq / Hkv) * Nq query rows that share the
// head are the columns of two tensor-core products per 16 keys:
//   S^T [16 keys x R] = K [16 x d] Q^T,   O^T [d x R] += V^T [d x 16] P^T,
// so K and V, read once, fill the M side of mma.m16n8k16 and the few rows
// cost N = 8 columns at a time. e4m3 codes become halves exactly; the block's
// K scale multiplies the logits, its V scale is folded into P's exponent. Q is
// brought to [2^14, 2^15) by a power of two per row, where every bf16 value
// down to 2^-29 of the row's largest is an exact half.
//
// Each warp keeps its own online softmax over the 16-key slices it takes (two
// references per column: ml for the sum of probabilities, mo for O, whose
// terms carry the V scales; both trail the true maximum by at most 2^8, and
// are only looked up across lanes when one would trail further). P is rounded
// to half relative to mo (2^-11 relative), O and the sums are fp32.
//
// HBM-bound: 2 d bytes per cached token and KV head, against which Q and O
// are small. The work is a line of units, one per (sequence, KV head, chunk of
// rows, block of 64 tokens), cut into equal parts for the CTAs whatever the
// sequences' lengths; a row whose units fall to several CTAs is joined from
// their partial results by a second kernel.
#include <cuda_fp16.h>

#include "fa_cache8.cuh"

namespace fa {
namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr float kShift = 6.f;             // P is taken times 2^6: at most 2^14 as a half, normal down to 2^-20

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 matrix of halves spread over the warp.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The codes of one 16-key slice as a lane (g = lane / 4, t = lane % 4) feeds
// them to the products. K: rows g and g + 8, bytes 64 c + 16 t .. + 15 of each
// 64-byte piece c; word w of a piece is the operand of product step 4 c + w
// (which columns of d a step covers is free as long as Q agrees). V: tokens
// 2t, 2t+1, 2t+8, 2t+9, a lane's D / 8 columns of d as words.
template <int D>
struct Slice {
  uint4 k[2][D / 64];
  uint32_t v[4][D / 32];
};

// column of d that word w, byte e of a lane's V words holds
template <int D>
__device__ __forceinline__ int v_column(int g, int w) {
  if constexpr (D == 64) return 8 * g + 4 * w;
  else return 128 * (w >> 2) + 16 * g + 4 * (w & 3);
}

template <int D>
__device__ __forceinline__ void load_slice(Slice<D>& s, const uint8_t* k, const uint8_t* v, int d, int tokens, int lane) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const int row = g + 8 * r, col = 64 * c + 16 * t;
      s.k[r][c] = (row < tokens && col < d) ? __ldg(reinterpret_cast<const uint4*>(k + row * d + col)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 2 * t + (i & 1) + 8 * (i >> 1);
    if constexpr (D == 64) {
      const int col = 8 * g;
      const uint2 x = (row < tokens && col < d) ? __ldg(reinterpret_cast<const uint2*>(v + row * d + col)) : make_uint2(0, 0);
      s.v[i][0] = x.x;
      s.v[i][1] = x.y;
    } else {
#pragma unroll
      for (int c = 0; c < D / 128; ++c) {
        const int col = 128 * c + 16 * g;
        const uint4 x = (row < tokens && col < d) ? __ldg(reinterpret_cast<const uint4*>(v + row * d + col)) : make_uint4(0, 0, 0, 0);
        s.v[i][4 * c] = x.x;
        s.v[i][4 * c + 1] = x.y;
        s.v[i][4 * c + 2] = x.z;
        s.v[i][4 * c + 3] = x.w;
      }
    }
  }
}

// The query rows [row0, row0 + ncols) of the group as product operands in
// shared memory: for column n, step j and lane l the two registers at
// sq[((n / 8) * (D / 16) + j) * 32 + l]; rows past R and columns past d are 0.
// qs[n]: the power of two by which the row was divided.
template <int D>
__device__ __forceinline__ void stage_queries(uint2* sq, float* qs, const __nv_bfloat16* q, int R, int row0, int ncols,
                                              int d, int warp, int lane) {
  for (int n = warp; n < ncols; n += kWarps) {
    const int row = row0 + n;
    float x[D / 128 < 1 ? 1 : D / 128][4];
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < (D + 127) / 128; ++c) {
      const int col = 128 * c + 4 * lane;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[c][e] = 0.f;
      if (row < R && col < d) {
        const uint2 u = *reinterpret_cast<const uint2*>(q + static_cast<size_t>(row) * d + col);
        x[c][0] = __uint_as_float(u.x << 16);
        x[c][1] = __uint_as_float(u.x & 0xFFFF0000u);
        x[c][2] = __uint_as_float(u.y << 16);
        x[c][3] = __uint_as_float(u.y & 0xFFFF0000u);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) amax = fmaxf(amax, fabsf(x[c][e]));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    // exponent that brings the largest to [2^14, 2^15); bounded so that both powers are normal
    const int e2 = amax > 0.f ? max(-100, min(100, static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 14)) : 0;
    const float down = __uint_as_float(static_cast<uint32_t>(127 - e2) << 23);
    if (lane == 0) qs[n] = __uint_as_float(static_cast<uint32_t>(127 + e2) << 23);
#pragma unroll
    for (int c = 0; c < (D + 127) / 128; ++c) {
      const int col = 128 * c + 4 * lane;
      if (col < D) {
        const int j = 4 * (col / 64) + (col % 16) / 4, t = (col % 64) / 16;
        sq[((n >> 3) * (D / 16) + j) * 32 + (n & 7) * 4 + t] =
            make_uint2(pack_f16x2(x[c][0] * down, x[c][1] * down), pack_f16x2(x[c][2] * down, x[c][3] * down));
      }
    }
  }
}

// S^T of one slice for NT column tiles (before any scale).
template <int D, int NT>
__device__ __forceinline__ void scores(float (&s)[NT][4], const uint4 (&k)[2][D / 64], const uint2* sq, int lane) {
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
  for (int j = 0; j < D / 16; ++j) {
    const uint4 x = k[0][j / 4], y = k[1][j / 4];
    const uint32_t wx = j % 4 == 0 ? x.x : j % 4 == 1 ? x.y : j % 4 == 2 ? x.z : x.w;
    const uint32_t wy = j % 4 == 0 ? y.x : j % 4 == 1 ? y.y : j % 4 == 2 ? y.z : y.w;
    const uint32_t a0 = e4m3x2_to_f16x2(wx), a1 = e4m3x2_to_f16x2(wy);
    const uint32_t a2 = e4m3x2_to_f16x2(wx >> 16), a3 = e4m3x2_to_f16x2(wy >> 16);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint2 b = sq[(n * (D / 16) + j) * 32 + lane];
      mma_f16(s[n], a0, a1, a2, a3, b.x, b.y);
    }
  }
}

// Where a unit of the line lies, and the whole line's length. A sequence has
// at least one block of units, so that rows without keys are written too.
struct Line {
  long long total;
  __device__ __forceinline__ static int blocks(const Cache8Params& p, int b) {
    return max(1, (cache_length(p.lengths, b, p.max_blocks) + kCacheBlock - 1) / kCacheBlock);
  }
  // all lanes of a warp together
  __device__ __forceinline__ Line(const Cache8Params& p, int per_block, int lane) {
    long long sum = 0;
    for (int b = lane; b < p.B; b += 32) sum += blocks(p, b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    total = sum * per_block;
  }
  // parts it is cut into by a grid of `ctas`: none of them empty, so that
  // every part between a row's first and last has a partial result of it
  __device__ __forceinline__ long long parts(long long ctas) const { return min(ctas, total); }
  // sequence of unit u, and the units before that sequence
  __device__ __forceinline__ static void find(const Cache8Params& p, int per_block, long long u, int lane, int& b,
                                              long long& before) {
    long long base = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int cnt = b0 + lane < p.B ? blocks(p, b0 + lane) : 0;
      long long incl = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, u < (base + incl) * per_block);
      if (hit) {
        const int src = __ffs(hit) - 1;
        b = b0 + src;
        before = (base + __shfl_sync(0xffffffffu, incl - cnt, src)) * per_block;
        return;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    b = p.B - 1;
    before = 0;
  }
};
__device__ __forceinline__ long long part_begin(long long total, long long i, long long parts) { return total * i / parts; }
// the part that unit u belongs to
__device__ __forceinline__ long long part_of(long long total, long long u, long long parts) {
  return ((u + 1) * parts - 1) / total;
}

template <int D, int NT>
struct Cfg {
  static constexpr int kCols = 8 * NT;
  static constexpr int kQBytes = NT * (D / 16) * 32 * 8;
  static constexpr int kRedBytes = kWarps * kCols * D * 4;
  static constexpr int kStatBytes = (3 * kWarps + 4) * kCols * 4;
  static constexpr int kSmem = kQBytes + kRedBytes + kStatBytes;
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads) cache8_fwd_kernel(const Cache8Params p) {
  using C = Cfg<D, NT>;
  extern __shared__ __align__(16) uint8_t smem[];
  uint2* const sq = reinterpret_cast<uint2*>(smem);
  float* const red = reinterpret_cast<float*>(smem + C::kQBytes);                 // [warp][column][D]
  float* const st_ml = reinterpret_cast<float*>(smem + C::kQBytes + C::kRedBytes);  // [warp][column]
  float* const st_l = st_ml + kWarps * C::kCols;
  float* const st_mo = st_l + kWarps * C::kCols;
  float* const f_ml = st_mo + kWarps * C::kCols;                                  // [column]
  float* const f_l = f_ml + C::kCols;
  float* const f_mo = f_l + C::kCols;
  float* const qs = f_mo + C::kCols;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int per_block = p.c.Hkv * p.chunks;

  const Line line(p, per_block, lane);
  const long long parts = line.parts(gridDim.x);
  if (blockIdx.x >= parts) return;
  const long long u0 = part_begin(line.total, blockIdx.x, parts), u1 = part_begin(line.total, blockIdx.x + 1, parts);
  int b;
  long long before;
  Line::find(p, per_block, u0, lane, b, before);
  for (long long u = u0; u < u1;) {
    // ---- segment: blocks [blk0, blk1) of row group (b, h, chunk)
    const int nblk = Line::blocks(p, b);
    const int len = cache_length(p.lengths, b, p.max_blocks);
    const int row = static_cast<int>((u - before) / nblk);                        // head * chunks + chunk
    const int blk0 = static_cast<int>((u - before) - static_cast<long long>(row) * nblk);
    const int blk1 = static_cast<int>(min(static_cast<long long>(nblk), blk0 + (u1 - u)));
    const int h = row / p.chunks, chunk = row - h * p.chunks;
    const int row0 = chunk * C::kCols;
    const size_t qrow = (static_cast<size_t>(b) * p.Hq + static_cast<size_t>(h) * p.G) * p.Nq;   // first of the R rows
    __syncthreads();                                     // the previous segment's shared memory is free
    stage_queries<D>(sq, qs, p.q + qrow * p.c.d, p.R, row0, C::kCols, p.c.d, warp, lane);
    __syncthreads();

    float o[NT][D / 16][4];
    float ml[NT][2], mo[NT][2], l[NT][2], qsc[NT][2];
    int lim[NT][2];                                      // keys visible to the column
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][j][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int col = 8 * n + 2 * t + e;
        ml[n][e] = mo[n][e] = -INFINITY;
        l[n][e] = 0.f;
        qsc[n][e] = qs[col] * p.scale_log2;
        lim[n][e] = p.causal ? min(len, max(0, len - p.Nq + (row0 + col) % p.Nq + 1)) : len;
      }
    }
    const int all = p.causal ? max(0, len - p.Nq + 1) : len;     // keys below it are visible to every column
    const int* const table = p.table + static_cast<long long>(b) * p.max_blocks;

    for (int s = blk0 * 4 + warp; s < blk1 * 4; s += kWarps) {
      const int blk = s >> 2;
      const int key0 = s * 16;
      if (key0 >= len) break;
      const int page = table[blk];
      if (page < 0 || page >= p.c.num_blocks) continue;          // no such block: its tokens are absent
      const size_t ph = static_cast<size_t>(page) * p.c.Hkv + h;
      const size_t off = (ph * kCacheBlock + (s & 3) * 16) * p.c.d;
      Slice<D> sl;
      load_slice<D>(sl, p.c.k + off, p.c.v + off, p.c.d, len - key0, lane);
      const float ks = __ldg(p.c.k_scale + ph), vs = __ldg(p.c.v_scale + ph);
      const float lvs = log2f(vs);
      float x[NT][4];
      scores<D, NT>(x, sl.k, sq, lane);
      bool grow = false;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[n][e] *= ks * qsc[n][e & 1];
          if (key0 + 16 > all && key0 + g + 8 * (e >> 1) >= lim[n][e & 1]) x[n][e] = -INFINITY;
          grow |= x[n][e] > ml[n][e & 1] + 8.f || x[n][e] + lvs > mo[n][e & 1] + 8.f;
        }
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(x[n][e], x[n][e + 2]);
#pragma unroll
            for (int sh = 4; sh < 32; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
            if (mx > ml[n][e]) {
              l[n][e] *= ex2_approx(ml[n][e] - mx);
              ml[n][e] = mx;
            }
            if (mx + lvs > mo[n][e]) {
              const float alpha = ex2_approx(mo[n][e] - (mx + lvs));
              mo[n][e] = mx + lvs;
#pragma unroll
              for (int j = 0; j < D / 16; ++j) {
                o[n][j][e] *= alpha;
                o[n][j][e + 2] *= alpha;
              }
            }
          }
      }
      uint32_t pb[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float po[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = ml[n][e & 1], c = mo[n][e & 1];
          l[n][e & 1] += ex2_approx(x[n][e] - (a == -INFINITY ? 0.f : a));
          po[e] = ex2_approx(x[n][e] + (lvs - (c == -INFINITY ? 0.f : c) + kShift));
        }
        pb[n][0] = movmatrix(pack_f16x2(po[0], po[1]));
        pb[n][1] = movmatrix(pack_f16x2(po[2], po[3]));
      }
#pragma unroll
      for (int w = 0; w < D / 32; ++w)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t sel = half ? 0x7362u : 0x5140u;
          const uint32_t x01 = __byte_perm(sl.v[0][w], sl.v[1][w], sel), x89 = __byte_perm(sl.v[2][w], sl.v[3][w], sel);
          const uint32_t a0 = e4m3x2_to_f16x2(x01), a1 = e4m3x2_to_f16x2(x01 >> 16);
          const uint32_t a2 = e4m3x2_to_f16x2(x89), a3 = e4m3x2_to_f16x2(x89 >> 16);
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_f16(o[n][2 * w + half], a0, a1, a2, a3, pb[n][0], pb[n][1]);
        }
    }

    // ---- join the warps
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float sum = l[n][e];
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, sh);
        const int col = 8 * n + 2 * t + e;
        if (g == 0) {
          st_ml[warp * C::kCols + col] = ml[n][e];
          st_mo[warp * C::kCols + col] = mo[n][e];
          st_l[warp * C::kCols + col] = sum;
        }
        float* const dst = red + (warp * C::kCols + col) * D;
#pragma unroll
        for (int w = 0; w < D / 32; ++w)
          *reinterpret_cast<float4*>(dst + v_column<D>(g, w)) =
              make_float4(o[n][2 * w][e], o[n][2 * w][e + 2], o[n][2 * w + 1][e], o[n][2 * w + 1][e + 2]);
      }
    __syncthreads();
    if (tid < C::kCols) {
      float a = -INFINITY, c = -INFINITY, sum = 0.f;
      for (int w = 0; w < kWarps; ++w) {
        a = fmaxf(a, st_ml[w * C::kCols + tid]);
        c = fmaxf(c, st_mo[w * C::kCols + tid]);
      }
      for (int w = 0; w < kWarps; ++w) {
        const float m = st_ml[w * C::kCols + tid];
        const float lw = st_l[w * C::kCols + tid];
        sum += m == -INFINITY ? lw : lw * ex2_approx(m - a);    // (a NaN stays)
        const float mw = st_mo[w * C::kCols + tid];
        st_mo[w * C::kCols + tid] = mw == -INFINITY ? 1.f : ex2_approx(mw - c);
      }
      f_ml[tid] = a;
      f_l[tid] = sum;
      f_mo[tid] = c - kShift;
    }
    __syncthreads();
    const bool whole = blk0 == 0 && blk1 == nblk;
    const long long slot = (2LL * blockIdx.x + (u == u0 ? 0 : 1)) * C::kCols;
    for (int i = tid; i < C::kCols * (D / 4); i += kThreads) {
      const int col = i / (D / 4), c4 = (i - col * (D / 4)) * 4;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = st_mo[w * C::kCols + col];
        const float4 y = *reinterpret_cast<const float4*>(red + (w * C::kCols + col) * D + c4);
        a.x = fmaf(f, y.x, a.x);
        a.y = fmaf(f, y.y, a.y);
        a.z = fmaf(f, y.z, a.z);
        a.w = fmaf(f, y.w, a.w);
      }
      if (whole) {
        if (row0 + col < p.R && c4 < p.c.d) {
          const float sum = f_l[col];
          const float f = sum == 0.f ? 0.f : ex2_approx(f_mo[col] - f_ml[col]) / sum;
          *reinterpret_cast<uint2*>(p.o + (qrow + row0 + col) * p.c.d + c4) =
              make_uint2(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(a.z * f, a.w * f));
        }
      } else {
        *reinterpret_cast<float4*>(p.part_o + (slot + col) * D + c4) = a;
      }
    }
    if (tid < C::kCols) {
      if (whole) {
        if (row0 + tid < p.R) p.lse[qrow + row0 + tid] = f_l[tid] == 0.f ? -INFINITY : (f_ml[tid] + log2f(f_l[tid])) * kLn2;
      } else {
        float* const s3 = p.part_s + (slot + tid) * 3;
        s3[0] = f_ml[tid];
        s3[1] = f_l[tid];
        s3[2] = f_mo[tid];
      }
    }
    u += blk1 - blk0;
    if (u - before >= static_cast<long long>(nblk) * per_block) {                 // the next sequence
      before += static_cast<long long>(nblk) * per_block;
      ++b;
    }
  }
}

// Joins the rows whose units went to several CTAs: one CTA per row.
template <int D>
__global__ void __launch_bounds__(D / 4 < 32 ? 32 : D / 4) cache8_join_kernel(const Cache8Params p, int cols, int ctas) {
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.y, h = blockIdx.x / p.R, r = blockIdx.x - h * p.R;
  const int per_block = p.c.Hkv * p.chunks;
  const Line line(p, per_block, lane);
  const long long parts = line.parts(ctas);
  long long before = 0;
  for (int i = lane; i < b; i += 32) before += Line::blocks(p, i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) before += __shfl_xor_sync(0xffffffffu, before, o);
  const int nblk = Line::blocks(p, b), chunk = r / cols;
  const long long ua = before * per_block + static_cast<long long>(h * p.chunks + chunk) * nblk;
  const long long c0 = part_of(line.total, ua, parts), c1 = part_of(line.total, ua + nblk - 1, parts);
  if (c0 == c1) return;                                       // written whole
  const int first = part_begin(line.total, c0, parts) == ua ? 0 : 1;
  float ml = -INFINITY, mo = -INFINITY;
  for (long long c = c0; c <= c1; ++c) {
    const float* const s3 = p.part_s + ((2 * c + (c == c0 ? first : 0)) * cols + r % cols) * 3;
    ml = fmaxf(ml, s3[0]);
    mo = fmaxf(mo, s3[2]);
  }
  float sum = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  const int c4 = threadIdx.x * 4;
  for (long long c = c0; c <= c1; ++c) {
    const long long slot = (2 * c + (c == c0 ? first : 0)) * cols + r % cols;
    const float* const s3 = p.part_s + slot * 3;
    sum += s3[0] == -INFINITY ? s3[1] : s3[1] * ex2_approx(s3[0] - ml);
    const float f = s3[2] == -INFINITY ? 1.f : ex2_approx(s3[2] - mo);   // (no term yet: O is 0, or a NaN that stays)
    if (c4 < D) {
      const float4 y = *reinterpret_cast<const float4*>(p.part_o + slot * D + c4);
      a.x = fmaf(f, y.x, a.x);
      a.y = fmaf(f, y.y, a.y);
      a.z = fmaf(f, y.z, a.z);
      a.w = fmaf(f, y.w, a.w);
    }
  }
  const size_t row = (static_cast<size_t>(b) * p.Hq + static_cast<size_t>(h) * p.G) * p.Nq + r;
  const float f = sum == 0.f ? 0.f : ex2_approx(mo - ml) / sum;
  if (c4 < p.c.d)
    *reinterpret_cast<uint2*>(p.o + row * p.c.d + c4) = make_uint2(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(a.z * f, a.w * f));
  if (threadIdx.x == 0) p.lse[row] = sum == 0.f ? -INFINITY : (ml + log2f(sum)) * kLn2;
}

// ------------------------------------------------------------------ weights
// weight_j = decay weight_j + sum over the group's rows of exp(s_rj - LSE_r):
// the scores once more from K (the probabilities need the whole row's LSE).
// Units are (sequence, KV head, block).
template <int D>
__global__ void __launch_bounds__(kThreads) cache8_weight_kernel(const Cache8Params p) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int ntiles = (p.R + 7) / 8;
  uint2* const sq = reinterpret_cast<uint2*>(smem);
  float* const qs = reinterpret_cast<float*>(smem + ntiles * (D / 16) * 32 * 8);   // [columns]
  float* const lse2 = qs + ntiles * 8;                                             // [columns], +inf past R
  int* const lim = reinterpret_cast<int*>(lse2 + ntiles * 8);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int per_block = p.c.Hkv;
  const Line line(p, per_block, lane);
  const long long parts = line.parts(gridDim.x);
  if (blockIdx.x >= parts) return;
  const long long u0 = part_begin(line.total, blockIdx.x, parts), u1 = part_begin(line.total, blockIdx.x + 1, parts);
  int b;
  long long before;
  Line::find(p, per_block, u0, lane, b, before);
  for (long long u = u0; u < u1;) {
    const int nblk = Line::blocks(p, b);
    const int len = cache_length(p.lengths, b, p.max_blocks);
    const int h = static_cast<int>((u - before) / nblk);
    const int blk0 = static_cast<int>((u - before) - static_cast<long long>(h) * nblk);
    const int blk1 = static_cast<int>(min(static_cast<long long>(nblk), blk0 + (u1 - u)));
    const size_t qrow = (static_cast<size_t>(b) * p.Hq + static_cast<size_t>(h) * p.G) * p.Nq;
    __syncthreads();
    stage_queries<D>(sq, qs, p.q + qrow * p.c.d, p.R, 0, ntiles * 8, p.c.d, warp, lane);
    for (int col = tid; col < ntiles * 8; col += kThreads) {
      lse2[col] = col < p.R ? p.lse[qrow + col] * kLog2e : INFINITY;
      lim[col] = p.causal ? min(len, max(0, len - p.Nq + col % p.Nq + 1)) : len;
    }
    __syncthreads();
    const int* const table = p.table + static_cast<long long>(b) * p.max_blocks;
    for (int s = blk0 * 4 + warp; s < blk1 * 4; s += kWarps) {
      const int key0 = s * 16;
      if (key0 >= len) break;
      const int page = table[s >> 2];
      if (page < 0 || page >= p.c.num_blocks) continue;
      const size_t ph = static_cast<size_t>(page) * p.c.Hkv + h;
      const uint8_t* const k = p.c.k + (ph * kCacheBlock + (s & 3) * 16) * p.c.d;
      uint4 kk[2][D / 64];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const int row = g + 8 * r, col = 64 * c + 16 * t;
          kk[r][c] = (key0 + row < len && col < p.c.d) ? __ldg(reinterpret_cast<const uint4*>(k + row * p.c.d + col))
                                                       : make_uint4(0, 0, 0, 0);
        }
      const float ks = __ldg(p.c.k_scale + ph) * p.scale_log2;
      float w0 = 0.f, w1 = 0.f;                               // keys key0 + g, key0 + g + 8
      for (int n = 0; n < ntiles; ++n) {
        float x[1][4];
        scores<D, 1>(x, kk, sq + n * (D / 16) * 32, lane);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = 8 * n + 2 * t + (e & 1);
          const int key = key0 + g + 8 * (e >> 1);
          const float l2 = lse2[col];
          // a row that sees no key has LSE -inf and adds nothing
          const float pr = key < lim[col] && l2 != -INFINITY ? ex2_approx(x[0][e] * (ks * qs[col]) - l2) : 0.f;
          if (e < 2) w0 += pr;
          else w1 += pr;
        }
      }
#pragma unroll
      for (int sh = 1; sh < 4; sh <<= 1) {
        w0 += __shfl_xor_sync(0xffffffffu, w0, sh);
        w1 += __shfl_xor_sync(0xffffffffu, w1, sh);
      }
      if (t < 2) {
        const int key = key0 + g + 8 * t;
        float* const dst = p.c.weight + ph * kCacheBlock + (s & 3) * 16 + g + 8 * t;
        // (a decay of 0 drops what was there, a NaN too)
        if (key < len) *dst = (p.decay == 0.f ? 0.f : p.decay * *dst) + (t ? w1 : w0);
      }
    }
    u += blk1 - blk0;
    if (u - before >= static_cast<long long>(nblk) * per_block) {
      before += static_cast<long long>(nblk) * per_block;
      ++b;
    }
  }
}

template <int D, int NT>
cudaError_t launch_fwd(const Cache8Params& p, int parts, cudaStream_t stream) {
  static PerDeviceOnce attr;
  const cudaError_t e = attr.run([] {
    return cudaFuncSetAttribute(cache8_fwd_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, NT>::kSmem);
  });
  if (e != cudaSuccess) return e;
  cache8_fwd_kernel<D, NT><<<parts, kThreads, Cfg<D, NT>::kSmem, stream>>>(p);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_all(const Cache8Params& p, int parts, cudaStream_t stream) {
  const int cols = cache8_columns(p.c.d, p.R);
  cudaError_t e = cudaErrorInvalidValue;
  if (cols == 8) e = launch_fwd<D, 1>(p, parts, stream);
  else if (cols == 16) e = launch_fwd<D, 2>(p, parts, stream);
  else if constexpr (D <= 128) e = launch_fwd<D, 4>(p, parts, stream);
  if (e != cudaSuccess) return e;
  if (parts > 1) {
    cache8_join_kernel<D><<<dim3(p.c.Hkv * p.R, p.B), D / 4 < 32 ? 32 : D / 4, 0, stream>>>(p, cols, parts);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess || !p.add_weights) return e;
  static PerDeviceOnce attr;
  e = attr.run([] {
    return cudaFuncSetAttribute(cache8_weight_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (kCache8MaxRows / 8) * (D / 16) * 256 + kCache8MaxRows * 12);
  });
  if (e != cudaSuccess) return e;
  const int ntiles = (p.R + 7) / 8;
  const long long units = static_cast<long long>(p.B) * p.c.Hkv * p.max_blocks;
  const int grid = static_cast<int>(units < kCache8Parts ? units : kCache8Parts);
  cache8_weight_kernel<D><<<grid, kThreads, ntiles * ((D / 16) * 256 + 96), stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

int cache8_columns(int d, int R) { return R <= 8 ? 8 : R <= 16 || d > 128 ? 16 : 32; }

int cache8_parts(int B, int Hkv, int chunks, int max_blocks) {
  const long long units = static_cast<long long>(B) * Hkv * chunks * max_blocks;
  return static_cast<int>(units < kCache8Parts ? units : kCache8Parts);
}

cudaError_t launch_cache8_fwd(const Cache8Params& p, cudaStream_t stream) {
  const int parts = cache8_parts(p.B, p.c.Hkv, p.chunks, p.max_blocks);
  if (p.c.d <= 64) return launch_all<64>(p, parts, stream);
  if (p.c.d <= 128) return launch_all<128>(p, parts, stream);
  return launch_all<256>(p, parts, stream);
}

}  // namespace fa
