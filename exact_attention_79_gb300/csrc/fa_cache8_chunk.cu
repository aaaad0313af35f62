// Attention of chunks of new tokens over the 8-bit block cache: any number of
// new tokens per sequence, different in each, behind any number of cached ones.
//
// Rows. For KV head h, a row tile is up to 128 rows: tt = 128 / G neighbouring tokens of
// the G query heads that share it, row r being token r / G, head r % G. So all rows of a
// tile see nearly the same keys (the causal border falls within tt tokens), and few new tokens still
// fill tiles. An item is kGroups row tiles of one sequence and KV head, which read the same
// K and V.
//
// Products, per tile of 128 keys (two cache blocks), on the tensor cores:
//   S [128 x 128 keys] = Q K^T   8-bit (kind::f8f6f4): K's codes as they are, Q in two terms, e4m3 and e5m2,
//      q = q0 + q1 of the row scaled by a power of two to [128, 256). From 2^-6 on q0 has four of bf16's eight
//      significant bits, and what it leaves is at most eight units of the last, which three bits hold (e5m2, down to
//      2^-16): exact down to 2^-13 of the row's largest value. Below that 2^-10 at most is left, off by 2^-14: 2^-21 of the
//      row's largest. Two terms at the 8-bit rate cost what one bf16 product does.
//   O [128 x d] += P V           f16 (kind::f16): V's codes as halves (exact), P in f16.
// A block's K scale multiplies its logits, its V scale its P, by a factor that keeps them within f16:
// hence two references per row, ml for the sum of probabilities and mo for O, P' = 2^(x - ml) 2^(ml - mo) vs <= 2^15, each
// P' within 2^-11 of itself or 2^-31 of the row's largest. O's error against 64 bits is then its own rounding to bf16.
// (P in two e4m3 terms would save V's conversion but is 2^-8, and three cost half as much again.)
//
// K goes from memory into the product untouched (TMA). V passes through converting
// warps: 16 codes a thread at a time from the landing buffer to the MN-major f16 tile; they
// clear keys that are not there (P is 0, but 0 x NaN is not) and also lay out Q.
//
// The work is a line of units, one per (item, key tile), cut into equal parts for a
// persistent grid of one CTA per SM, whatever the lengths (a unit is a unit, of one row tile or of two: by a model of
// the line the longest part is 16% above the mean for a piece beside single tokens, 8% for several prompts' pieces,
// nothing for one prompt); an item whose units fall to several CTAs is joined from partial results by a second
// kernel. An item of no more than one row tile gives its even key tiles to one softmax group and its odd ones to
// the other, joined in TMEM.
//
// Warps: 0-3 and 4-7 the softmax groups (one thread per row), 8 producer (block table, scales,
// TMA), 9 tensor-core issuer, 10 ring watcher, 11 scheduler, 12-15 converters. At d > 128 (kGroups = 1) O takes half of
// TMEM, S is double-buffered, warps 4-7 convert too and there is no watcher. The loops of all roles are about 20 KB of
// code, more than the instruction cache holds: each line that has gone costs some 230 cycles, and the order of
// the roles below is the best of ten (4096 tokens at the end of 32768, 32 heads on 8, d 128: 1434 to 1812 us).
//
// What bounds it. There (1463 to 1526 us from one GPU to the next, 1.35 to 1.41 PFLOP/s, 70 to 73% of the bf16
// rate) a step of two row tiles takes 3300 cycles, 2100 of them products: each group's S, softmax (1600), P V and the
// hand-offs between follow one another, and two groups do not cover it all. At d 64 a step takes 2900. A change of
// items costs some 15000 (Q's terms, the diagonal's mask, O's way out).
#include <type_traits>

#include "fa_cache8.cuh"

namespace fa {
namespace {

constexpr int kThreads = 512;
constexpr float kTrailL = 8.f;            // log2 of how far the references may trail
constexpr float kTopO = 7.f, kTrailO = 15.f;   // P' of the row's largest is 2^7 where mo is set, at most 2^15
constexpr float kNoKey = -1.f;            // factor of O for a row that sees no key
constexpr int kInfo = 8;                  // tiles whose scales wait in shared memory
constexpr int kItems = 4;                 // segments that the scheduler may be ahead
constexpr int kItemInts = 12;
// Places that a change of items takes up on the line, so that parts of many items have fewer key tiles. (Not what it costs,
// four to five key tiles' time: the line does not weigh items of one row tile less either, and both go together. With 1, 4 and
// 9: 7 prompts' pieces 315, 308, 305 us; a piece and 24 single tokens 348, 345, 352; wide heads 280, 281, 286.)
constexpr int kTurn = 1;

template <int D>
struct Cfg {
  static constexpr int kGroups = D == 128 ? 2 : 1;
  static constexpr int kCh = D / 128;                      // 128-byte columns of codes
  static constexpr int kRows = 128 * kGroups;              // of an item
  static constexpr int kConv = kGroups == 2 ? 4 : 8;       // converting warps: 12-15, with one group 4-7 too
  static constexpr int kReaders = 2 + (kGroups == 2 ? 1 : 0) + kConv + 4 * kGroups;   // warps that read a segment: producer, issuer, watcher, converters, softmax
  static constexpr int kKeysV = D == 128 ? 128 : 64;       // keys of a V stage
  static constexpr int kPerTile = 128 / kKeysV;            // V stages of a key tile
  static constexpr int kQTerm = 16384 * kCh;               // one term of a row tile
  static constexpr int kQBytes = kGroups * 2 * kQTerm;
  static constexpr int kTileK = 16384 * kCh;
  static constexpr int kRingK = D == 128 ? 3 : 2;
  static constexpr int kCodesV = 16384, kHalfV = 32768;    // a V stage as codes and as halves
  static constexpr int kRingV = 2;
  static constexpr int kBoxV = kKeysV * 128;               // 64 columns of halves
  static constexpr int kOffK = kQBytes, kOffCodes = kOffK + kRingK * kTileK, kOffHalf = kOffCodes + kRingV * kCodesV;
  static constexpr int kOffStat = kOffHalf + kRingV * kHalfV;
  static constexpr int kStat = kRows * 4 + (kGroups == 2 ? 128 * 12 : 0) + kInfo * 32 + kItems * kItemInts * 4;
  static constexpr int kLayout = kOffStat + kStat + 272;
  static constexpr int kSmem = kLayout + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  // setmaxnreg, of the 512 x 128 launched: without spills, which L1 beside so much shared memory does not hold
  static constexpr uint32_t kRegsSoftmax = D == 128 ? 192 : 168, kRegsOther = D == 128 ? 64 : 112;
  static_assert(kGroups * kRegsSoftmax + (4 - kGroups) * kRegsOther <= 512, "register split");
  static __device__ __forceinline__ uint32_t col_s(int i) { return 128u * i; }
  static __device__ __forceinline__ uint32_t col_o(int i) { return 256u + 128u * i; }
};

// Bounded wait whose limit starts at its own first look at the timer.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned long long limit_ns) {
  uint32_t polls = 0;
  uint64_t until = 0;
  while (!mbar_try_wait(bar, parity)) {
    if ((++polls & 255u) == 0) {
      if (*abort_flag) return false;
      const uint64_t now = global_timer_ns();
      if (until == 0) until = now + limit_ns;
      if (now > until) {
        *abort_flag = 1;
        return false;
      }
    }
  }
  return true;
}

// ------------------------------------------------------------------ the line of units
// A sequence's new tokens (rows row0 .. row0 + n - 1 of the packed ones) and length.
struct Sequence {
  int row0, n, len;
  __device__ __forceinline__ Sequence(const ChunkParams& p, int b) {
    row0 = max(0, min(p.cu[b], p.T));
    n = max(0, min(p.cu[b + 1], p.T) - row0);
    len = cache_length(p.lengths, b, p.max_blocks);
  }
  // keys that its tokens below `last` see
  __device__ __forceinline__ int seen(const ChunkParams& p, int last) const { return p.causal ? len - n + last : len; }
  __device__ __forceinline__ int items(const ChunkParams& p) const { return static_cast<int>((n + static_cast<unsigned>(p.span) - 1) / p.span); }
  // key tiles of the tokens below `last`; a row without keys has one, so that it is written
  __device__ __forceinline__ int tiles(const ChunkParams& p, int last) const { return max(1, (seen(p, last) + 127) >> 7); }
  __device__ __forceinline__ int end_of(const ChunkParams& p, int item) const {
    return static_cast<int>(min(static_cast<long long>(n), (item + 1LL) * p.span));
  }
};
// sum over j < n of floor((a j + b) / m), by the well-known steps of Euclid's algorithm on (a, m)
__device__ __forceinline__ long long floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) {
  long long sum = 0;
  while (n > 0) {
    sum += static_cast<long long>(n) * (n - 1LL) / 2 * (a / m) + static_cast<long long>(n) * (b / m);
    a %= m;
    b %= m;
    const unsigned y = a * n + b;                          // a n is at most about T
    n = y / m;
    b = y % m;
    const unsigned t = m;
    m = a;
    a = t;
    if (m == 0) break;
  }
  return sum;
}
// Key tiles of the first x items of one KV head, x at most the sequence's items.
__device__ __forceinline__ long long tiles_before(const ChunkParams& p, const Sequence& s, int x) {
  if (x == 0) return 0;
  if (!p.causal) return static_cast<long long>(x) * s.tiles(p, s.n);
  long long sum = 0;
  if (x == s.items(p)) {                                   // the last item may end early
    --x;
    sum = s.tiles(p, s.n);
  }
  if (x == 0) return sum;
  // item i has max(1, ceil(((i + 1) span + past) / 128)): 1 for the first `ones`
  const int past = s.len - s.n;
  const int ones = past > 128 ? 0 : static_cast<int>(min(static_cast<long long>(x), (128LL - past) / p.span));
  sum += ones;
  if (x > ones)
    sum += floor_sum(x - ones, 128, p.span, static_cast<unsigned>((ones + 1LL) * p.span + past + 127));
  return sum;
}
// Places of a sequence on one KV head: `turn` more for every item, the time that a change of items costs.
__device__ __forceinline__ long long places(const ChunkParams& p, const Sequence& s, int turn) {
  const int n = s.items(p);
  return tiles_before(p, s, n) + static_cast<long long>(turn) * n;
}
__device__ __forceinline__ long long warp_sum(long long x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The line, cut into `parts` equal parts. A part is at least twice a turn long, so that it
// has units, and where it begins in a turn its first units are that item's.
struct Line {
  long long total;
  int turn, parts;
  // by a whole warp
  __device__ __forceinline__ Line(const ChunkParams& p, int lane) {
    long long units = 0, items = 0;
    for (int b = lane; b < p.B; b += 32) {
      const Sequence s(p, b);
      units += places(p, s, 0);
      items += s.items(p);
    }
    units = warp_sum(units) * p.c.Hkv;
    items = warp_sum(items) * p.c.Hkv;
    turn = static_cast<int>(min(static_cast<long long>(kTurn), units / (2 * p.ctas)));
    total = units + turn * items;
    parts = static_cast<int>(min(static_cast<long long>(p.ctas), total));
  }
  __device__ __forceinline__ long long begin(int i) const { return total * i / parts; }
  __device__ __forceinline__ int part_of(long long u) const { return static_cast<int>(((u + 1) * parts - 1) / total); }
};

// A place of the line: `off` places into an item (its turn, then its units).
struct Place {
  int b = 0, h = 0, item = 0, off = 0;
  long long start = 0;                                     // places before the item
  // by a whole warp; u below the total
  __device__ __forceinline__ void find(const ChunkParams& p, int turn, long long u, int lane) {
    long long before = 0, each = 0;
    b = p.B - 1;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      long long cnt = 0;
      if (b0 + lane < p.B) cnt = places(p, Sequence(p, b0 + lane), turn);
      long long incl = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, u < before + incl * p.c.Hkv);
      if (hit) {
        const int src = __ffs(hit) - 1;
        b = b0 + src;
        each = __shfl_sync(0xffffffffu, cnt, src);
        before += __shfl_sync(0xffffffffu, incl - cnt, src) * p.c.Hkv;
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31) * p.c.Hkv;
    }
    const Sequence s(p, b);
    h = static_cast<int>((u - before) / each);
    before += h * each;
    // the last item that does not begin behind u, 32 at a time
    int lo = 0, n = s.items(p);
    while (n > 1) {
      const int step = (n + 31) / 32, i = lo + min(lane * step, n - 1);
      const bool not_behind = before + tiles_before(p, s, i) + static_cast<long long>(turn) * i <= u;
      const int k = __popc(__ballot_sync(0xffffffffu, not_behind && lane * step < n)) - 1;
      const int left = n - k * step;
      lo += k * step;
      n = min(step, left);
    }
    item = lo;
    start = before + tiles_before(p, s, lo) + static_cast<long long>(turn) * lo;
    off = static_cast<int>(u - start);
  }
};

// An item's share of a part: key tiles [t0, t1) of `tiles`.
struct Segment {
  int b, h, row0, n, len;
  int tok0;                                                // the item's first token, counted from the sequence's first new one
  int t0, t1, tiles;
  bool split;                                              // one row tile, whose key tiles alternate between the groups
  int n0;                                                  // group 0's key tiles (not split): its rows see fewer
};
// From the part's first place on, segment by segment.
struct Walk {
  int b, h, item, off, turn;
  long long left;
  Sequence s;
  __device__ __forceinline__ Walk(const ChunkParams& p, const Place& at, int line_turn, long long length)
      : b(at.b), h(at.h), item(at.item), off(at.off), turn(line_turn), left(length), s(p, at.b) {}
  template <int kGroups>
  __device__ __forceinline__ bool next(const ChunkParams& p, Segment& g) {
    if (left <= 0) return false;
    g.b = b;
    g.h = h;
    g.row0 = s.row0;
    g.n = s.n;
    g.len = s.len;
    g.tok0 = item * p.span;
    g.tiles = s.tiles(p, s.end_of(p, item));
    const int take = static_cast<int>(min(left, static_cast<long long>(turn + g.tiles - off)));
    g.t0 = max(0, off - turn);
    g.t1 = off + take - turn;
    g.split = kGroups == 2 && g.tok0 + p.tt >= s.n;
    g.n0 = max(0, min(s.tiles(p, min(s.n, g.tok0 + p.tt)), g.t1) - g.t0);
    left -= take;
    off = 0;
    if (++item == s.items(p)) {
      item = 0;
      if (++h == p.c.Hkv) {
        h = 0;
        while (left > 0 && ++b < p.B) {
          s = Sequence(p, b);
          if (s.n > 0) break;
        }
        if (b >= p.B) left = 0;
      }
    }
    return g.t1 > g.t0;                                    // (false: the part ends in a turn)
  }
};

// A segment as the scheduler hands it on: the ints of its slot, and what most roles go by.
enum { kB, kH, kRow0, kNew, kLen, kTok0, kT0, kN, kN0, kSplit, kWhole };
struct Item {
  int n, n0;                                               // key tiles; group 0's (not split)
  bool split;
};

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_to_e5m2x2(uint32_t x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f16x2 %0, %1;" : "=h"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void mul2_b(float& d0, float& d1, float a0, float a1, float b) {
  asm("{\n\t.reg .b64 a, b, d;\n\t"
      "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\t"
      "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
      : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b));
}
__device__ __forceinline__ void store16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" :: "r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
// The lower half of an operand's descriptor (start address and leading offset), and the whole: eight-row groups 1024 bytes
// apart, 128-byte swizzle.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo_bytes) {
  return static_cast<uint32_t>(smem_desc_sw128(saddr, lbo_bytes, 1024));
}
__device__ __forceinline__ uint64_t desc_of(uint32_t lo) { return static_cast<uint64_t>(1024u >> 4 | 1u << 14 | 2u << 29) << 32 | lo; }
__device__ __forceinline__ float times_factor(float o, float factor) { return factor == kNoKey ? 0.f : o * factor; }

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
cache8_chunk_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const ChunkParams p) {
  using C = Cfg<D>;
  constexpr int kGroups = C::kGroups;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  auto s_q = [&](int group, int term) { return base + (group * 2 + term) * C::kQTerm; };
  auto s_k = [&](int i) { return base + C::kOffK + i * C::kTileK; };
  auto s_codes = [&](int i) { return base + C::kOffCodes + i * C::kCodesV; };
  auto s_half = [&](int i) { return base + C::kOffHalf + i * C::kHalfV; };
  float* const row_scale = reinterpret_cast<float*>(gbase + C::kOffStat);           // [kRows] what Q's rows were divided by
  float* const other = row_scale + C::kRows;                                       // [3][128] group 1's ml, mo, l (split)
  volatile float* const info = reinterpret_cast<volatile float*>(other + (kGroups == 2 ? 3 * 128 : 0));   // [kInfo][8]: per half K scale times scale_digits, log2 of V's, there
  volatile int* const items = reinterpret_cast<volatile int*>(gbase + C::kOffStat + C::kStat - kItems * kItemInts * 4);
  const uint32_t bars = base + C::kOffStat + C::kStat;
  uint8_t* const gbars = gbase + (bars - base);
  auto bar_k_full = [&](int i) { return bars + 8u * i; };              // 3
  auto bar_k_empty = [&](int i) { return bars + 24u + 8u * i; };       // 3
  auto bar_c_full = [&](int i) { return bars + 48u + 8u * i; };        // V's codes
  auto bar_c_empty = [&](int i) { return bars + 64u + 8u * i; };
  auto bar_v_full = [&](int i) { return bars + 80u + 8u * i; };        // V's halves
  auto bar_v_empty = [&](int i) { return bars + 96u + 8u * i; };
  auto bar_s_full = [&](int i) { return bars + 112u + 8u * i; };
  auto bar_p_ready = [&](int i) { return bars + 128u + 8u * i; };
  auto bar_o_final = [&](int i) { return bars + 144u + 8u * i; };
  const uint32_t bar_q_full = bars + 160u, bar_q_empty = bars + 168u;
  const uint32_t bar_other_full = bars + 176u, bar_other_empty = bars + 184u;
  auto bar_item_full = [&](int i) { return bars + 192u + 8u * i; };    // kItems
  auto bar_item_empty = [&](int i) { return bars + 224u + 8u * i; };
  const uint32_t bar_stall = bars + 256u;                              // nothing arrives (timeout test)
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gbars + 264);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(gbars + 268);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < C::kRingK; ++i) {
      mbar_init(bar_k_full(i), 1);
      mbar_init(bar_k_empty(i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_c_full(i), 1);
      mbar_init(bar_c_empty(i), C::kConv);
      mbar_init(bar_v_full(i), C::kConv);
      mbar_init(bar_v_empty(i), 1);
      mbar_init(bar_s_full(i), 1);
      mbar_init(bar_p_ready(i), kGroups == 2 ? 129 : 128);   // + the watcher
      mbar_init(bar_o_final(i), 1);
    }
    mbar_init(bar_q_full, C::kConv);
    mbar_init(bar_q_empty, 1 + 4 * kGroups);               // its products done, its scales read by every softmax warp
    mbar_init(bar_other_full, 128);
    mbar_init(bar_other_empty, 128);
    for (int i = 0; i < kItems; ++i) {
      mbar_init(bar_item_full(i), 1);
      mbar_init(bar_item_empty(i), C::kReaders);
    }
    mbar_init(bar_stall, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;

  // What the scheduler says of segment n of this part, as a thread or a warp reads it; false: there is none, or a wait ran
  // out. `done` gives its slot back, once per warp.
  auto take_one = [&](int n, Item& it) -> bool {
    if (!wait(bar_item_full(n % kItems), (n / kItems) & 1, abort_flag, p.timeout_ns)) return false;
    const volatile int* const m = items + (n % kItems) * kItemInts;
    it.n = m[kN];
    it.n0 = m[kN0];
    it.split = m[kSplit];
    return it.n > 0;
  };
  auto take = [&](int n, Item& it) -> bool {
    const bool ok = wait(bar_item_full(n % kItems), (n / kItems) & 1, abort_flag, p.timeout_ns);
    if (!__all_sync(0xffffffffu, ok)) return false;
    const volatile int* const m = items + (n % kItems) * kItemInts;
    it.n = m[kN];
    it.n0 = m[kN0];
    it.split = m[kSplit];
    return it.n > 0;
  };
  auto field = [&](int n, int which) { return items[(n % kItems) * kItemInts + which]; };
  auto done = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar_item_empty(n % kItems));
  };

  if (warp == 11) {
    // ------------------------------------------------------------ scheduler
    // Finds this part's segments ahead of time: one warp's look-up instead of all roles', whose code for it would come
    // from memory at every change. And brings the segment's rows of Q into L2.
    setmaxnreg_dec<C::kRegsOther>();
    const Line line(p, lane);
    bool ok = true;
    long long u = 0, length = 0;
    Place place;
    if (static_cast<int>(blockIdx.x) < line.parts) {
      u = line.begin(blockIdx.x);
      length = line.begin(blockIdx.x + 1) - u;
      place.find(p, line.turn, u, lane);
    }
    Walk walk(p, place, line.turn, length);
    if (p.joins != nullptr) {
      // for the second kernel: the item that this part is the second one of
      int c0 = 0, c1 = -1, slot = 0;
      if (length > 0 && place.off > line.turn) {
        c0 = line.part_of(place.start + line.turn);
        if (c0 == static_cast<int>(blockIdx.x) - 1)
          c1 = line.part_of(place.start + line.turn + walk.s.tiles(p, walk.s.end_of(p, place.item)) - 1);
        slot = line.begin(c0) >= place.start ? 0 : 1;      // the item is that part's first or not
      }
      if (lane == 0) {
        int4* const join = reinterpret_cast<int4*>(p.joins) + 2 * blockIdx.x;
        join[0] = make_int4(c0, c1, slot, place.h);
        join[1] = make_int4(walk.s.row0, walk.s.n, place.item * p.span, 0);
      }
    }
    Segment s;
    for (int n = 0; ok; ++n) {
      const bool more = walk.next<kGroups>(p, s);
      if (n >= kItems) ok = wait(bar_item_empty(n % kItems), ((n / kItems) & 1) ^ 1, abort_flag, p.timeout_ns);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane == 0) {
        volatile int* const m = items + (n % kItems) * kItemInts;
        m[kB] = s.b;
        m[kH] = s.h;
        m[kRow0] = s.row0;
        m[kNew] = s.n;
        m[kLen] = s.len;
        m[kTok0] = s.tok0;
        m[kT0] = s.t0;
        m[kN] = more ? s.t1 - s.t0 : 0;
        m[kN0] = s.n0;
        m[kSplit] = s.split;
        m[kWhole] = s.t0 == 0 && s.t1 == s.tiles;
        mbar_arrive(bar_item_full(n % kItems));
      }
      __syncwarp();
      if (!more) break;
      for (int r = lane; r < (s.split ? 128 : C::kRows); r += 32) {
        const int row = r & 127, tok = row / p.G, token = s.tok0 + (r >> 7) * p.tt + tok;
        if (tok >= p.tt || token >= s.n) continue;
        const __nv_bfloat16* const src =
            p.q + (s.h * p.G + (row - tok * p.G)) * p.q_sh + (static_cast<long long>(s.row0) + token) * p.q_st;
        for (int c = 0; c < p.c.d; c += 64) asm volatile("prefetch.global.L2 [%0];" :: "l"(src + c));
      }
    }
    __syncwarp();
  } else if (warp < 4 * kGroups) {
    // ------------------------------------------------------------ softmax groups
    setmaxnreg_inc<C::kRegsSoftmax>();
    const int g = warp >> 2;
    const int quarter = warp & 3;                          // TMEM lane quarter this warp may access
    const int row = quarter * 32 + lane;                   // of the row tile
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    uint32_t tile = 0;                                     // tiles before the segment
    uint32_t par = 0;                                      // parities: bit 0 S, 1 O final, 2 group 1's results, 3 Q
    bool ok = true;
    for (int seg = 0; ok; ++seg) {
      uint32_t at, end;                                    // this group's tiles at, at + dx, ... below end, counted from the kernel's start
      int dx, lim;                                         // lim: keys that this row sees from the tile on
      {
        Item it;
        if (!take(seg, it)) break;
        at = tile + (it.split ? g : 0);
        dx = it.split ? 2 : 1;
        end = tile + (it.split || g == 1 || kGroups == 1 ? it.n : it.n0);
        tile += it.n;
        const int len = field(seg, kLen), last = field(seg, kTok0) + (it.split ? 0 : g * p.tt) + row / p.G + 1;   // tokens up to this row's
        lim = (p.causal ? min(len, len - field(seg, kNew) + last) : len) - (field(seg, kT0) + (it.split ? g : 0)) * 128;
      }
      const bool any = at < end, split = dx == 2;
      ok = wait(bar_q_full, par >> 3 & 1u, abort_flag, p.timeout_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      par ^= 8u;
      const float rs = p.scale_power * row_scale[(split ? 0 : g * 128) + row];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_q_empty);
      bool rescale = false;                                // O holds something
      float ml = -INFINITY, mo = -INFINITY;                // references, log2 units of the logits
      float l = 0.f;                                       // running sum relative to ml
      for (; at < end; at += dx, lim -= 128 * dx) {
        const int buf = kGroups == 1 ? at & 1 : g;
        ok = wait(bar_s_full(buf), kGroups == 1 ? at >> 1 & 1u : par & 1u, abort_flag, p.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        par ^= 1u;
        tc_fence_after();
        const volatile float* const sc = info + (at % kInfo) * 8;
        // (at least the smallest normal number: a K scale of 0 makes 0 of every logit, but would make NaN of the -inf of
        // keys that are not there)
        const float ka = fmaxf(sc[0] * rs, 1.17549435e-38f), kb = fmaxf(sc[4] * rs, 1.17549435e-38f);
        const float lva = sc[1], lvb = sc[5];
        const bool here_a = sc[2] != 0.f, here_b = sc[6] != 0.f;
        const uint32_t t_s = tbase + lane_off + C::col_s(buf);
        const uint32_t t_o = tbase + lane_off + C::col_o(g);
        uint32_t sr[4][32];
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) tmem_ld_32x32b_x32(t_s + q4 * 32, sr[q4]);
        tmem_wait_ld();
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) reg_fence_x32(sr[q4]);
        float v[128];
#pragma unroll
        for (int i = 0; i < 128; ++i) v[i] = __uint_as_float(sr[i >> 5][i & 31]);
        if (lim < 128 || !here_a || !here_b) {
#pragma unroll
          for (int q4 = 0; q4 < 4; ++q4) {
            const int n = (q4 < 2 ? here_a : here_b) ? lim - 32 * q4 : 0;
#pragma unroll
            for (int i = 0; i < 32; ++i) v[32 * q4 + i] = i < n ? v[32 * q4 + i] : -INFINITY;
          }
        }
        float mk[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float* w = v + 32 * k;
          float a = fmax3(w[0], w[1], w[2]);
#pragma unroll
          for (int e = 3; e < 31; e += 2) a = fmax3(a, w[e], w[e + 1]);
          mk[k] = fmaxf(a, w[31]);
        }
        const float xa = fmaxf(mk[0], mk[1]) * ka, xb = fmaxf(mk[2], mk[3]) * kb;
        const float xl = fmaxf(xa, xb), xo = fmaxf(xa + lva, xb + lvb);
        const bool grow_l = xl > ml + kTrailL;             // also true on the first tile with a key (ml = -inf)
        const bool grow_o = xo > mo + kTrailO;
        const float ml_new = grow_l ? xl : ml, mo_new = grow_o ? xo - kTopO : mo;
        const float alpha_l = grow_l ? ex2_approx(ml - ml_new) : 1.f;
        const float alpha_o = grow_o ? ex2_approx(mo - mo_new) : 1.f;
        ml = ml_new;
        mo = mo_new;
        const float neg_m = ml == -INFINITY ? 0.f : -ml;
        float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
          const float k = h2 ? kb : ka;
          // V's scale relative to mo (0 where mo is not set: no V so far has a scale)
          const float f = mo == -INFINITY ? 0.f : ex2_approx(fminf((h2 ? lvb : lva) - neg_m - mo, 126.f));
          uint32_t pr[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            float x0, x1, y0, y1;
            fma2_bc(x0, x1, v[h2 * 64 + 2 * i], v[h2 * 64 + 2 * i + 1], k, neg_m);
            const float p0 = ex2_approx(x0);
            const float p1 = ex2_approx(x1);
            add2_acc(sum0, sum1, p0, p1);
            mul2_b(y0, y1, p0, p1, f);
            pr[i] = pack_f16x2(y0, y1);                    // within 2^-11; l sums P unrounded
          }
          tmem_st_32x32b_x32(t_s + h2 * 32, pr);
        }
        l = l * alpha_l + (sum0 + sum1);
        // O <- alpha_o O; the P V before it is done: it was issued before the S just waited for (one group:
        // before the S of the tile after this one, so it has to be waited for)
        if (rescale && __any_sync(0xffffffffu, grow_o)) {
          if (kGroups == 1) {
            const uint32_t c = at * C::kPerTile - 1;       // V's stage that the product before read last
            ok = wait(bar_v_empty(c % C::kRingV), (c / C::kRingV) & 1, abort_flag, p.timeout_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
          }
#pragma unroll
          for (int c0 = 0; c0 < D; c0 += 32) {
            if (c0 >= p.c.d) continue;
            uint32_t o[32];
            tmem_ld_32x32b_x32(t_o + c0, o);
            tmem_wait_ld();
            reg_fence_x32(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha_o);
            tmem_st_32x32b_x32(t_o + c0, o);
          }
        }
        rescale = true;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar_p_ready(buf));
      }
      if (!ok) break;
      // ---------------------------------------------------------- the item's result
      if (any) {
        ok = wait(bar_o_final(g), par >> 1 & 1u, abort_flag, p.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        par ^= 2u;
        tc_fence_after();
      }
      if (split && g == 1) {
        // group 0 joins both: this group's O stays in TMEM until it has
        other[row] = ml;
        other[128 + row] = mo;
        other[256 + row] = l;
        tc_fence_before();
        mbar_arrive(bar_other_full);
        ok = wait(bar_other_empty, par >> 2 & 1u, abort_flag, p.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        par ^= 4u;
        tc_fence_after();
        done(seg);
        continue;
      }
      float f0 = 1.f, f1 = kNoKey;                         // factors of this group's O and of the other's
      float root = 1.f;                                    // of both: V's scale itself may be below the normal numbers
      if (l == 0.f) f0 = kNoKey;
      if (kGroups == 2 && split) {
        ok = wait(bar_other_full, par >> 2 & 1u, abort_flag, p.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        par ^= 4u;
        tc_fence_after();
        const float ml1 = other[row], mo1 = other[128 + row], l1 = other[256 + row];
        if (l1 != 0.f) {
          const float m = fmaxf(ml, ml1), mm = fmaxf(mo, mo1);
          // (a reference that is not set has nothing summed)
          l = (l == 0.f ? 0.f : l * ex2_approx(ml - m)) + l1 * ex2_approx(ml1 - m);
          f0 = f0 == kNoKey ? kNoKey : mo == -INFINITY ? 0.f : ex2_approx(mo - mm);
          f1 = mo1 == -INFINITY ? 0.f : ex2_approx(mo1 - mm);
          ml = m;
          mo = mm;
        }
      }
      const bool whole = field(seg, kWhole);
      const int tok = row / p.G, token = field(seg, kTok0) + (split ? 0 : g * p.tt) + tok;   // counted from the sequence's first new one
      const bool real = tok < p.tt && token < field(seg, kNew);
      const int head = field(seg, kH) * p.G + (row - tok * p.G);
      const long long at_row = static_cast<long long>(field(seg, kRow0)) + token;
      const int slot_row = (split ? 0 : g * 128) + row;
      float* part = nullptr;
      if (whole) {
        root = l == 0.f ? 0.f : ex2_approx(0.5f * (mo - ml));   // (0 where mo is not set)
        const float factor = l == 0.f ? 0.f : root / l;
        f0 = f0 == kNoKey ? kNoKey : f0 * factor;
        f1 = f1 == kNoKey ? kNoKey : f1 * factor;
        if (real) p.lse[static_cast<long long>(head) * p.T + at_row] = l == 0.f ? -INFINITY : (ml + log2f(l)) * kLn2;
      } else {
        const int slot = 2 * blockIdx.x + (seg > 0);
        part = p.part_o + static_cast<long long>(slot) * C::kRows * D;
        float* const st = p.part_s + static_cast<long long>(slot) * C::kRows * 3;
        if (real) {
          st[slot_row] = ml;
          st[C::kRows + slot_row] = mo;
          st[2 * C::kRows + slot_row] = l;
        }
      }
      done(seg);
      __nv_bfloat16* const dst = p.o + head * p.o_sh + at_row * p.o_st;
#pragma unroll 1
      for (int c0 = 0; c0 < p.c.d; c0 += 32) {
        uint32_t o[32], o1[32];
        tmem_ld_32x32b_x32(tbase + lane_off + C::col_o(g) + c0, o);
        if (kGroups == 2 && split) tmem_ld_32x32b_x32(tbase + lane_off + C::col_o(1) + c0, o1);
        tmem_wait_ld();
        reg_fence_x32(o);
        float y[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) y[i] = times_factor(__uint_as_float(o[i]), f0);
        if (kGroups == 2 && split) {
          reg_fence_x32(o1);
#pragma unroll
          for (int i = 0; i < 32; ++i) y[i] += times_factor(__uint_as_float(o1[i]), f1);
        }
#pragma unroll
        for (int i = 0; i < 32; i += 2) mul2_b(y[i], y[i + 1], y[i], y[i + 1], root);
        if (!real) continue;
        if (whole) {
#pragma unroll
          for (int i = 0; i < 32; i += 8)
            if (c0 + i < p.c.d)
              *reinterpret_cast<uint4*>(dst + c0 + i) = make_uint4(pack_bf16x2(y[i], y[i + 1]), pack_bf16x2(y[i + 2], y[i + 3]),
                                                                   pack_bf16x2(y[i + 4], y[i + 5]), pack_bf16x2(y[i + 6], y[i + 7]));
        } else {
#pragma unroll
          for (int i = 0; i < 32; i += 4)
            if (c0 + i < p.c.d)
              reinterpret_cast<float4*>(part)[((c0 + i) / 4) * C::kRows + slot_row] = make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]);
        }
      }
      tc_fence_before();
      if (kGroups == 2 && split) mbar_arrive(bar_other_empty);
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ tensor-core issuer
    setmaxnreg_dec<C::kRegsOther>();
    if (lane == 0) {
      const uint32_t id_s = make_idesc(0, 128, 128, 0, 0);             // e4m3, both K-major
      const uint32_t id_s1 = id_s | 1u << 7;                           // A e5m2: Q's second term
      const uint32_t id_o = make_idesc(0, 128, p.c.d, 0, 1);           // f16, V MN-major
      // The issuing thread paces the kernel: a product takes 64 cycles, and every other instruction of this one thread
      // about eight. So a step's products stand in a row with constant offsets, the steps between a segment's first and
      // last ones run in a loop of their own, and with two groups P-ready stands for V and the next K too (the
      // watcher's arrival) and the watcher hands the rings back.
      const int steps = (p.c.d + 31) / 32;                             // products over d that are not all zeros
      // Descriptors by their lower halves; the upper ones are the same for all.
      uint32_t tb = tbase;
      const uint32_t kd0 = desc_lo(s_k(0), 16), qd0 = desc_lo(s_q(0, 0), 16), vd0 = desc_lo(s_half(0), C::kBoxV);
      constexpr uint32_t kStepK = C::kTileK >> 4, kStepV = C::kHalfV >> 4;
      bool ok = !p.test_stall || wait(bar_stall, 0, abort_flag, p.timeout_ns);   // runs out by design
      uint32_t np = 0;                                                 // parities of the buffers' P-ready
      int tile = 0;                                                    // tiles before the segment
      // S of the rows behind descriptor qd with the K behind kd into buffer `buf`, d = 32 count at most
      auto scores = [&](auto count, int buf, uint32_t qd, uint32_t kd) {
        constexpr int n = decltype(count)::value;
        const uint32_t dst = tb + C::col_s(buf);
#pragma unroll
        for (int i = 0; i < 2 * n; ++i) {
          const int term = i / n, k = i % n, off = (k >> 2) * 16384 + (k & 3) * 32;
          mma_fp8_ss(dst, desc_of(qd + ((term * C::kQTerm + off) >> 4)), desc_of(kd + (off >> 4)), term ? id_s1 : id_s, i > 0);
        }
        mma_commit(bar_s_full(buf));
      };
      // O of `group` += P in buffer `buf` times the V stage behind vd, the x-th of its tile
      auto product = [&](int buf, int group, int x, uint32_t vd, bool acc) {
        const uint32_t src = tb + C::col_s(buf) + x * (C::kKeysV / 2);
#pragma unroll
        for (int k = 0; k < C::kKeysV / 16; ++k)
          mma_bf16_ts(tb + C::col_o(group), src + k * 8, desc_of(vd + (k * 2048 >> 4)), id_o, acc || k > 0);
      };
      auto k_there = [&](int t) {
        ok = wait(bar_k_full(t % C::kRingK), (t / C::kRingK) & 1, abort_flag, p.timeout_ns);
        tc_fence_after();
      };
      auto p_there = [&](int buf) {
        ok = wait(bar_p_ready(buf), np >> buf & 1u, abort_flag, p.timeout_ns);
        np ^= 1u << buf;
        tc_fence_after();
      };
      auto kd_of = [&](int t) { return kd0 + static_cast<uint32_t>(t % C::kRingK) * kStepK; };
      auto segments = [&](auto count) {
        Item it;
        for (int seg = 0; ok && take_one(seg, it); ++seg) {
          mbar_arrive(bar_item_empty(seg % kItems));
          const int n = it.n, n0 = it.n0;
          const bool split = it.split;
          ok = wait(bar_q_full, seg & 1, abort_flag, p.timeout_ns);
          if (!ok) break;
          if (kGroups == 1) {
            // S of the next tile is out before this one's P V
            for (int j = -1; j < n && ok; ++j) {
              const int t = tile + j;
              if (j + 1 < n) {
                k_there(t + 1);
                if (!ok) break;
                scores(count, (t + 1) & 1, qd0, kd_of(t + 1));
                mma_commit(bar_k_empty((t + 1) % C::kRingK));
              } else {
                mma_commit(bar_q_empty);
              }
              if (j < 0) continue;
              p_there(t & 1);
#pragma unroll
              for (int x = 0; x < C::kPerTile && ok; ++x) {
                const int c = t * C::kPerTile + x, slot = c % C::kRingV;
                ok = wait(bar_v_full(slot), (c / C::kRingV) & 1, abort_flag, p.timeout_ns);
                if (!ok) break;
                tc_fence_after();
                product(t & 1, 0, x, vd0 + slot * kStepV, j > 0 || x > 0);
                mma_commit(bar_v_empty(slot));
              }
            }
            if (ok) mma_commit(bar_o_final(0));
          } else {
            // Step i is group i & 1's P V of a tile and its S of the next one: split, tile i, then i + 2; else tile
            // i / 2 of either group, then the one behind it. The first two steps have no P V yet.
            const uint32_t qd1 = qd0 + (split ? 0 : 2 * C::kQTerm >> 4);
            const int all = split ? n : 2 * n;
            for (int i = -2; i < all; ++i) {
              if (i == 0) {
                // the steps that have a next one but not the last, two at a time: V and next K of group 0, of group 1
                const int pairs = split ? (n - 3) / 2 : n0 - 2;
                uint32_t va = vd0 + (tile & 1) * kStepV, vb = vd0 + ((tile + split) & 1) * kStepV;
                const uint32_t turn_v = split ? 0u : vd0 ^ (vd0 + kStepV);
                int ka = (tile + (split ? 2 : 1)) % C::kRingK, kb = split ? (ka + 1) % C::kRingK : ka;
                uint32_t kda = kd0 + ka * kStepK, kdb = kd0 + kb * kStepK;
                const uint32_t kd_end = kd0 + C::kRingK * kStepK;
                auto step = [&](uint32_t kd) {
                  kd += kStepK;
                  return kd == kd_end ? kd0 : kd;
                };
                uint32_t par = np & 1u, par1 = np >> 1, qa = qd0, qb = qd1;
                for (int j = 0; j < pairs; ++j) {
                  asm volatile("" : "+r"(qa), "+r"(qb), "+r"(tb));     // (or every product's offsets get registers of their own)
                  ok = wait(bar_p_ready(0), par, abort_flag, p.timeout_ns);
                  if (!ok) break;
                  tc_fence_after();
                  product(0, 0, 0, va, j > 0);
                  scores(count, 0, qa, kda);
                  ok = wait(bar_p_ready(1), par1, abort_flag, p.timeout_ns);
                  if (!ok) break;
                  tc_fence_after();
                  product(1, 1, 0, vb, j > 0);
                  scores(count, 1, qb, kdb);
                  par ^= 1u;
                  par1 ^= 1u;
                  va ^= turn_v;
                  vb ^= turn_v;
                  kda = step(kdb);
                  kdb = split ? step(kda) : kda;
                }
                if (!ok) break;
                if (pairs > 0) {
                  np = par | par1 << 1;
                  i = 2 * pairs;
                }
              }
              const int gr = i & 1, j = split ? i : i >> 1;
              const int mine = split || gr ? n : n0, next_j = split ? i + 2 : j + 1;
              const bool last = split || gr;
              if (j >= mine) continue;
              if (i >= 0) {
                p_there(gr);
                if (!ok) break;
                product(gr, gr, 0, vd0 + ((tile + j) & 1) * kStepV, split ? i > 1 : j > 0);
              } else if (next_j < mine && (split || !gr || n0 <= 0)) {
                k_there(tile + next_j);
                if (!ok) break;
              }
              if (next_j < mine) scores(count, gr, gr ? qd1 : qd0, kd_of(tile + next_j));
              else if (i >= 0) mma_commit(bar_o_final(gr));
              if (last && next_j + 1 == n) mma_commit(bar_q_empty);    // every S is out
            }
          }
          tile += n;
        }
      };
      // Two widths of code: d up to 64 and 128, up to 192 and 256. A d between runs in the next, over zeros of K and Q.
      constexpr int most = 4 * C::kCh;
      if (steps > most - 2) segments(std::integral_constant<int, most>());
      else segments(std::integral_constant<int, most - 2>());
    }
    __syncwarp();
  } else if (warp >= 12 || (kGroups == 1 && warp >= 4 && warp < 8)) {
    // ------------------------------------------------------------ converters
    setmaxnreg_dec<C::kRegsOther>();
    const int cw = warp >= 12 ? warp - 12 : warp;          // (with one group warps 4-7 are the converters 4-7)
    bool ok = true;
    int tile = 0;
    Item it;
    for (int seg = 0; ok && take(seg, it); ++seg) {
      const int len = field(seg, kLen), t0 = field(seg, kT0);
      // ---- Q, this warp's rows of each row tile. A row's bf16 values take as many bytes as its two terms: all rows come
      // at once by asynchronous copies (from L2: the scheduler) to where their terms will be, and are converted in place,
      // 16 bytes a lane. All wait for this once the last S is done, and its code comes from memory nearly every time, at about
      // 230 cycles for 128 bytes of it: so it is rolled up (unrolled eightfold it took 45000 cycles).
      ok = wait(bar_q_empty, (seg & 1) ^ 1, abort_flag, p.timeout_ns);
      if (!__all_sync(0xffffffffu, ok)) break;
      constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes; // lanes of a row, rows of a load
      constexpr int kMine = 128 / C::kConv;                // rows of a warp
      const int piece_q = lane % kLanes, sub = lane / kLanes;
      // where piece x of a row's bf16 values lands: the first half in the first term's row, the second in the second's
      const uint32_t raw_at = (piece_q / (kLanes / 2)) * C::kQTerm + (piece_q % (kLanes / 2) >> 3) * 16384;
      const int step_tok = kAtOnce / p.G, step_head = kAtOnce - step_tok * p.G;
      const long long step_plain = step_tok * p.q_st + step_head * p.q_sh, step_wrapped = step_plain + p.q_st - p.G * p.q_sh;
#pragma unroll 1
      for (int group = 0; group < (it.split ? 1 : kGroups); ++group) {
        int tok = (kMine * cw + sub) / p.G, head = kMine * cw + sub - tok * p.G;
        const int first_token = field(seg, kTok0) + group * p.tt, left = min(p.tt, field(seg, kNew) - first_token);
        const __nv_bfloat16* src = p.q + (static_cast<long long>(field(seg, kH)) * p.G + head) * p.q_sh +
                                   (static_cast<long long>(field(seg, kRow0)) + first_token + tok) * p.q_st + 8 * piece_q;
        const uint32_t dst = s_q(group, 0) + raw_at;
        if (8 * piece_q >= p.c.d) tok = p.tt;              // (columns behind d: zeros)
#pragma unroll 2
        for (int row = kMine * cw + sub; row < kMine * cw + kMine; row += kAtOnce) {
          const bool real = tok < left;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(swz128(dst, row, piece_q & 7)),
                       "l"(real ? src : p.q), "r"(real ? 16 : 0) : "memory");
          const bool wrap = head + step_head >= p.G;
          tok += step_tok + wrap;
          head += step_head - (wrap ? p.G : 0);
          src += wrap ? step_wrapped : step_plain;
        }
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
#pragma unroll 1
      for (int r = 0; r < (it.split ? 1 : kGroups) * kMine; r += 2 * kAtOnce) {
        const int group = r / kMine, row0 = kMine * cw + sub + r % kMine;   // and row0 + kAtOnce beside it
        uint32_t w[2][4], hi[2][2], lo[2][2];
#pragma unroll
        for (int e = 0; e < 2; ++e)
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[e][0]), "=r"(w[e][1]), "=r"(w[e][2]), "=r"(w[e][3])
                       : "r"(swz128(s_q(group, 0) + raw_at, row0 + e * kAtOnce, piece_q & 7)) : "memory");
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t m = 0;                                  // the largest magnitude, as bits
#pragma unroll
          for (int k = 0; k < 4; ++k) m = max(m, max(w[e][k] & 0x7FFFu, (w[e][k] >> 16) & 0x7FFFu));
          uint32_t amax = __reduce_max_sync(0xffffffffu, sub == 0 ? m : 0u);
          if (kAtOnce == 2) {
            const uint32_t second = __reduce_max_sync(0xffffffffu, sub == 1 ? m : 0u);
            if (sub == 1) amax = second;
          }
          // exponent that brings the largest to [128, 256); at least -126, so that both powers are normal: what is below 2^-119
          // comes to less than 128, down to 2^-7, and keeps all its bits (bf16's smallest is 2^-133). 120 is a finite row's largest
          // (without the min seven prompts' pieces take 326 us instead of 318: the code behind it lies otherwise).
          // A row with an infinity or NaN becomes NaN, as its logits are.
          const int e2 = amax > 0 ? max(-126, min(120, static_cast<int>(amax >> 7) - 127 - 7)) : 0;
          const float down = amax < 0x7F80u ? __uint_as_float(static_cast<uint32_t>(127 - e2) << 23) : NAN;
          if (piece_q == 0) row_scale[group * 128 + row0 + e * kAtOnce] = __uint_as_float(static_cast<uint32_t>(127 + e2) << 23);
          hi[e][0] = hi[e][1] = lo[e][0] = lo[e][1] = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // (eight significant bits and at most 256: f16, down to 2^-24, holds what the two terms can)
            const float x0 = __uint_as_float(w[e][k] << 16) * down, x1 = __uint_as_float(w[e][k] & 0xFFFF0000u) * down;
            const uint32_t c0 = pack_e4m3x2(x0, x1);
            hi[e][k >> 1] |= c0 << (16 * (k & 1));
            lo[e][k >> 1] |= f16x2_to_e5m2x2(sub_f16x2(pack_f16x2(x0, x1), e4m3x2_to_f16x2(c0))) << (16 * (k & 1));
          }
        }
        __syncwarp();                                      // all have read the rows
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t at = swz128((piece_q >> 4) * 16384, row0 + e * kAtOnce, (piece_q & 15) >> 1) + (piece_q & 1) * 8;
          asm volatile("st.shared.v2.b32 [%0], {%1, %2};" :: "r"(s_q(group, 0) + at), "r"(hi[e][0]), "r"(hi[e][1]) : "memory");
          asm volatile("st.shared.v2.b32 [%0], {%1, %2};" :: "r"(s_q(group, 1) + at), "r"(lo[e][0]), "r"(lo[e][1]) : "memory");
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_q_full);
      done(seg);
      // ---- V: 16 codes of a key at a time, from the codes' swizzled rows to two units of the halves' rows. Eight lanes, whose
      // 16 bytes go together, take four pieces of one box (64 columns) of keys k and k ^ 5: no bank twice, in the load
      // or in either store. A thread's keys are kApart apart, so one address each serves with constant offsets.
      constexpr int kBoxes = D / 64, kPieces = C::kKeysV * D / 16 / (32 * C::kConv);   // of a thread
      constexpr int kApart = 8 * C::kConv;
      const int quad = lane & 3, key0 = 2 * ((lane >> 3) + 4 * cw) ^ (lane & 4 ? 5 : 0);
      const uint32_t from = swz128(0, key0, quad), to = swz128(0, key0, 2 * quad);
      for (int j = t0; j < t0 + it.n && ok; ++j, ++tile) {
        const volatile float* const there = info + (tile % kInfo) * 8;
#pragma unroll
        for (int x = 0; x < C::kPerTile; ++x) {
          const int c = tile * C::kPerTile + x, slot = c % C::kRingV;
          if (ok) ok = wait(bar_c_full(slot), (c / C::kRingV) & 1, abort_flag, p.timeout_ns);
          if (ok) ok = wait(bar_v_empty(slot), ((c / C::kRingV) & 1) ^ 1, abort_flag, p.timeout_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          // keys of the stage that there are, in each of its blocks; the others become 0
          const int valid = len - j * 128 - x * C::kKeysV;
          const bool here0 = there[C::kPerTile == 1 ? 2 : 4 * x + 2] != 0.f, here1 = there[6] != 0.f;
          const uint32_t src = s_codes(slot) + from, dst = s_half(slot) + to;
          const bool all = valid >= C::kKeysV && here0 && (C::kPerTile == 2 || here1);
#pragma unroll 1
          for (int four = 0; four < kPieces / 4; ++four) {
            const int down = four * (4 / kBoxes) * kApart;
            uint4 w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int box = e % kBoxes, step = kApart * (e / kBoxes);
              if (64 * box >= p.c.d) continue;
              const uint32_t at = (src ^ ((box & 1) * 64)) + (box >> 1) * 8192 + (down + step) * 128;
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[e].x), "=r"(w[e].y), "=r"(w[e].z), "=r"(w[e].w) : "r"(at) : "memory");
            }
            if (!all) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int key = key0 + down + kApart * (e / kBoxes);
                if (!(key < valid && (key < 64 ? here0 : here1))) w[e] = make_uint4(0, 0, 0, 0);
              }
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int box = e % kBoxes, step = kApart * (e / kBoxes);
              if (64 * box >= p.c.d) continue;
              const uint32_t at = box * C::kBoxV + (down + step) * 128;
              store16(dst + at, e4m3x2_to_f16x2(w[e].x & 0xFFFFu), e4m3x2_to_f16x2(w[e].x >> 16), e4m3x2_to_f16x2(w[e].y & 0xFFFFu),
                      e4m3x2_to_f16x2(w[e].y >> 16));
              store16((dst ^ 16) + at, e4m3x2_to_f16x2(w[e].z & 0xFFFFu), e4m3x2_to_f16x2(w[e].z >> 16), e4m3x2_to_f16x2(w[e].w & 0xFFFFu),
                      e4m3x2_to_f16x2(w[e].w >> 16));
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar_c_empty(slot));
            mbar_arrive(bar_v_full(slot));
          }
        }
      }
    }
    __syncwarp();
  } else if (kGroups == 2 && warp == 10) {
    // ------------------------------------------------------------ ring watcher
    // One arrival on P-ready when V of its tile and K of the next S behind it have landed, and the rings' slots back when
    // the S that shows them read is done: K of that S, and V up to the tile whose product was issued before it. It
    // waits for every load in order, so no parity is taken for that of two phases earlier.
    setmaxnreg_dec<C::kRegsOther>();
    if (lane == 0) {
      Item s;
      bool ok = true;
      int tile = 0, k_seen = 0, v_back = 0;                // tiles before the segment, K tiles waited for, V stages handed back
      uint32_t ns0 = 0, ns1 = 0, np0 = 0, np1 = 0;         // phases of S and of P-ready
      auto hand = [&](int g) {
        uint32_t& np = g ? np1 : np0;
        // arrive for a phase only once the one before it has completed
        if (np > 0) ok = wait(bar_p_ready(g), (np - 1) & 1, abort_flag, p.timeout_ns);
        if (ok) mbar_arrive(bar_p_ready(g));
        ++np;
      };
      for (int seg = 0;; ++seg) {
        if (!ok || !take_one(seg, s)) break;
        mbar_arrive(bar_item_empty(seg % kItems));
        const int n = s.n;
        for (int x = 0; x < n && ok; ++x) {
          const int t = tile + x, g = s.split ? x & 1 : 1;
          auto k_there = [&](int last) {
            for (; k_seen <= last && ok; ++k_seen)
              ok = wait(bar_k_full(k_seen % C::kRingK), (k_seen / C::kRingK) & 1, abort_flag, p.timeout_ns);
          };
          auto s_done = [&]() {
            if (ok) ok = wait(bar_s_full(g), (g ? ns1 : ns0) & 1, abort_flag, p.timeout_ns);
            if (!ok) return;
            if (g) ++ns1;
            else ++ns0;
            mbar_arrive(bar_k_empty(t % C::kRingK));
            for (const int upto = s.split && x > 0 ? t - 2 : t - 1; v_back <= upto; ++v_back) mbar_arrive(bar_v_empty(v_back & 1));
          };
          // S before V where V of this tile may wait for the slot that goes back then: split, and at the segment's
          // start (whose first K comes before that, as its slot goes back too). Otherwise group 0's P is ready long
          // before this is: S of group 1 is done when P of group 0 nearly is, and each look costs 90 to 200 cycles.
          const bool s_first = s.split || x == 0;
          if (s_first) {
            k_there(t);
            s_done();
          }
          if (ok) ok = wait(bar_v_full(t & 1), (t >> 1) & 1, abort_flag, p.timeout_ns);
          k_there(tile + min(n - 1, s.split ? x + 2 : x + 1));
          if (ok && !s.split && x < s.n0) hand(0);
          if (!s_first) s_done();
          if (ok) hand(g);
        }
        if (!s.split) ns0 += s.n0;
        tile += n;
      }
    }
    __syncwarp();
  } else if (warp == 8) {
    // ------------------------------------------------------------ producer
    setmaxnreg_dec<C::kRegsOther>();
    if (lane == 0) {
      tma_prefetch_map(&map_k);
      tma_prefetch_map(&map_v);
    }
    int tile = 0;                                          // tiles so far
    bool ok = true;
    Item it;
    for (int seg = 0; ok && take(seg, it); ++seg) {
      const int blk0 = 2 * field(seg, kT0), blk1 = blk0 + 2 * it.n, h = field(seg, kH);
      const int* const table = p.table + static_cast<long long>(field(seg, kB)) * p.max_blocks;
      const int held = min(blk1, (field(seg, kLen) + kCacheBlock - 1) / kCacheBlock);
      done(seg);
      // 32 blocks at a time, one per lane; the next 32 are looked up while these are loaded
      auto page_of = [&](int blk) {
        const int page = blk + lane < held ? table[blk + lane] : -1;
        return page < p.c.num_blocks ? page : -1;
      };
      float ks = 0.f, vs = 0.f;
      int z = -1;
      auto scales_of = [&](int page) {
        const long long ph = page >= 0 ? static_cast<long long>(page) * p.c.Hkv + h : -1;
        ks = page >= 0 ? p.c.k_scale[ph] : 0.f;
        vs = page >= 0 ? p.c.v_scale[ph] : 0.f;
        z = static_cast<int>(ph);
      };
      scales_of(page_of(blk0));
      int va = -1, vb = -1;                                // the last tile's blocks, whose V is still to come
      auto load_v = [&](int t, int a, int b) {
#pragma unroll 1
        for (int x = 0; x < C::kPerTile && ok; ++x) {
          const int c = t * C::kPerTile + x, cs = c % C::kRingV, za = C::kPerTile == 1 || x == 0 ? a : b;
          ok = wait(bar_c_empty(cs), ((c / C::kRingV) & 1) ^ 1, abort_flag, p.timeout_ns);
          if (!ok) break;
          // a stage is two boxes: both blocks (d up to 128), or both halves of one block's columns
          const bool two = C::kPerTile == 1 ? b >= 0 : za >= 0;
          mbar_arrive_expect_tx(bar_c_full(cs), ((za >= 0) + two) * 8192);
          if (za >= 0) tma_load_3d(s_codes(cs), &map_v, bar_c_full(cs), 0, 0, za);
          if (two) tma_load_3d(s_codes(cs) + 8192, &map_v, bar_c_full(cs), C::kPerTile == 1 ? 0 : 128, 0, C::kPerTile == 1 ? b : za);
        }
      };
      for (int blk = blk0; blk < blk1 && ok; blk += 32) {
        const float ks_now = ks, vs_now = vs;
        const int z_now = z, next_page = page_of(blk + 32);
        for (int i = 0; i < 32 && blk + i < blk1 && ok; i += 2, ++tile) {
          const int za = __shfl_sync(0xffffffffu, z_now, i), zb = __shfl_sync(0xffffffffu, z_now, i + 1);
          const int slot = tile % C::kRingK;
          if (lane == 0) {
            ok = wait(bar_k_empty(slot), ((tile / C::kRingK) & 1) ^ 1, abort_flag, p.timeout_ns);
            if (ok) mbar_expect_tx(bar_k_full(slot), ((za >= 0) + (zb >= 0)) * 8192 * C::kCh);
            for (int ch = 0; ch < C::kCh && ok; ++ch) {
              if (za >= 0) tma_load_3d(s_k(slot) + ch * 16384, &map_k, bar_k_full(slot), ch * 128, 0, za);
              if (zb >= 0) tma_load_3d(s_k(slot) + ch * 16384 + 8192, &map_k, bar_k_full(slot), ch * 128, 0, zb);
            }
          }
          ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0);
          if (!ok) break;
          // The scales, ahead of the one arrival that K's barrier waits for beside its bytes: who sees K's product sees
          // them. Their slot is free: K's slot was, so S of tile - kRingK is done, which was issued behind the
          // product of the tile before it, or two before it: the softmax of that one and of all before is done.
          if (lane == i || lane == i + 1) {
            volatile float* const dst = info + (tile % kInfo) * 8 + (lane - i) * 4;
            dst[0] = ks_now * p.scale_digits;
            dst[1] = log2f(vs_now);
            dst[2] = z_now >= 0 ? 1.f : 0.f;
          }
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(bar_k_full(slot));
            // V a tile behind K: S of the next tile comes before this one's product
            if (blk + i > blk0) load_v(tile - 1, va, vb);
          }
          va = za;
          vb = zb;
          ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0);
          if (i == 16) scales_of(next_page);
        }
      }
      if (lane == 0 && ok) load_v(tile - 1, va, vb);
      ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0);
    }
    __syncwarp();
  } else {
    setmaxnreg_dec<C::kRegsOther>();
  }

  // ---------------------------------------------------------------- teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    if (threadIdx.x == 0) atomicOr(p.status, kDevTimeout);
    abort_grace_period();
  }
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tbase, 512);
}

// ------------------------------------------------------------------ second kernel
// Joins the items whose key tiles went to several parts: CTA (i, rows) the one whose second part is i + 1, by what that part's
// scheduler wrote down.
constexpr int kJoinRows = 32;
constexpr int kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) cache8_chunk_join_kernel(const ChunkParams p) {
  using C = Cfg<D>;
  const int4* const join = reinterpret_cast<const int4*>(p.joins) + 2 * (blockIdx.x + 1);
  const int4 parts = join[0], at = join[1];                // (c0, c1, first slot, head), (row0, new tokens, first token)
  const int c0 = parts.x, c1 = parts.y;
  if (c1 < c0) return;
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.y * kJoinRows + lane;             // row of the item
  const int group = r >> 7, tok = (r & 127) / p.G;
  const int token = at.z + group * p.tt + tok;
  if (tok >= p.tt || token >= at.y) return;
  auto slot = [&](int c) { return 2LL * c + (c == c0 ? parts.z : 0); };
  float ml = -INFINITY, mo = -INFINITY;
  for (int c = c0; c <= c1; ++c) {
    const float* const st = p.part_s + slot(c) * C::kRows * 3 + r;
    if (st[2 * C::kRows] == 0.f) continue;
    ml = fmaxf(ml, st[0]);
    mo = fmaxf(mo, st[C::kRows]);
  }
  // eight columns at a time
  constexpr int kWide = D / 8 / (kJoinThreads / 32);       // per thread
  float4 a[kWide][2];
#pragma unroll
  for (int x = 0; x < kWide; ++x) a[x][0] = a[x][1] = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
  for (int c = c0; c <= c1; ++c) {
    const float* const st = p.part_s + slot(c) * C::kRows * 3 + r;
    const float lc = st[2 * C::kRows], moc = st[C::kRows];
    if (lc == 0.f) continue;                               // no key: its O is not there either
    l += lc * ex2_approx(st[0] - ml);
    const float f = moc == -INFINITY ? 0.f : ex2_approx(moc - mo);
    const float4* const o = reinterpret_cast<const float4*>(p.part_o + slot(c) * C::kRows * D);
#pragma unroll
    for (int x = 0; x < kWide; ++x) {
      const int col = 8 * ((threadIdx.x >> 5) + x * (kJoinThreads / 32));
#pragma unroll
      for (int y = 0; y < 2; ++y)
        if (col < p.c.d) {
          const float4 v = o[(col / 4 + y) * C::kRows + r];
          a[x][y].x = fmaf(v.x, f, a[x][y].x);
          a[x][y].y = fmaf(v.y, f, a[x][y].y);
          a[x][y].z = fmaf(v.z, f, a[x][y].z);
          a[x][y].w = fmaf(v.w, f, a[x][y].w);
        }
    }
  }
  const int head = parts.w * p.G + ((r & 127) - tok * p.G);
  const long long at_row = static_cast<long long>(at.x) + token;
  const float root = l == 0.f ? 0.f : ex2_approx(0.5f * (mo - ml)), factor = l == 0.f ? 0.f : root / l;   // (V's scale itself may be below the normal numbers)
  if (threadIdx.x < 32) p.lse[static_cast<long long>(head) * p.T + at_row] = l == 0.f ? -INFINITY : (ml + log2f(l)) * kLn2;
  __nv_bfloat16* const dst = p.o + head * p.o_sh + at_row * p.o_st;
#pragma unroll
  for (int x = 0; x < kWide; ++x) {
    const int col = 8 * ((threadIdx.x >> 5) + x * (kJoinThreads / 32));
    if (col < p.c.d)
      *reinterpret_cast<uint4*>(dst + col) =
          make_uint4(pack_bf16x2(a[x][0].x * factor * root, a[x][0].y * factor * root), pack_bf16x2(a[x][0].z * factor * root, a[x][0].w * factor * root),
                     pack_bf16x2(a[x][1].x * factor * root, a[x][1].y * factor * root), pack_bf16x2(a[x][1].z * factor * root, a[x][1].w * factor * root));
  }
}

template <int D>
cudaError_t launch(const CUtensorMap& mk, const CUtensorMap& mv, ChunkParams p, cudaStream_t stream) {
  using C = Cfg<D>;
  static PerDeviceOnce attr;
  const cudaError_t e = attr.run(
      [] { return cudaFuncSetAttribute(cache8_chunk_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem); });
  if (e != cudaSuccess) return e;
  p.span = p.tt * C::kGroups;
  cache8_chunk_kernel<D><<<p.ctas, kThreads, C::kSmem, stream>>>(mk, mv, p);
  if (p.max_blocks > 2 && p.ctas > 1)                      // (of one key tile nothing is split)
    cache8_chunk_join_kernel<D><<<dim3(p.ctas - 1, C::kRows / kJoinRows), kJoinThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

int chunk_rows(int d) { return d <= 128 ? Cfg<128>::kRows : Cfg<256>::kRows; }

cudaError_t launch_cache8_chunk(const CUtensorMap& mk, const CUtensorMap& mv, const ChunkParams& p, cudaStream_t stream) {
  return p.c.d <= 128 ? launch<128>(mk, mv, p, stream) : launch<256>(mk, mv, p, stream);
}

}  // namespace fa
