// Attention of a few new queries per sequence over the 8-bit block cache, on
// the tensor cores with the cache's codes as they are.
//
// For sequence b, KV head h the R = (Hq / Hkv) * Nq query rows that share the
// head are columns of two e4m3 products (tcgen05 kind::f8f6f4) per tile of 128
// tokens, two blocks of the cache:
//   S^T [128 tokens x R] = K [128 x d] Q^T      O^T [d x R] += V^T [d x 128] P^T
// K and V go from memory to shared memory (TMA, 128-byte swizzle) and from
// there into the products; no thread ever touches them. What the threads make
// small enough for e4m3 are Q and P, as sums of e4m3 terms in columns of their own:
//   Q, times a power of two per row that brings it to [128, 256): q = q0 + q1 / 16, which
//      is exact for every bf16 value down to 2^-10 (2^-17 of the row's largest);
//   P, y = 2^(s - reference + 5) <= 256: y = y0 + y1 / 32 + y2 / 1024, each term the rounding
//      of what the one before left (at most 8, hence 32), 2^-12 relative and 2^-20 absolute,
//      which is 2^-25 of the row's largest P: 2^17 keys that small are off by 2^-8 together.
// fp32 accumulators in TMEM: S^T twice (the next tile's is computed while this one's
// softmax runs), O^T with three columns per row.
//
// One thread per token. A block's K scale multiplies its logits; its V scale is
// folded into P's exponent. Hence two references per row: ml for the sum of
// probabilities, mo for O. Both are common to the CTA and may trail the true
// maximum by up to 2^3; when a token exceeds that (told by the barrier that the
// softmax warps pass once a tile), all look up the maximum and rescale O in TMEM.
// (By 2^4: as fast, P one bit coarser; by 2^2: one bit finer, 3% slower over 32
// sequences of 8192.)
//
// HBM-bound: 2 d bytes per cached token and KV head, against which Q and O
// are small. Measured: 32 sequences of 2048 to 8192 tokens, 64 heads on 8, d 128: 65 us,
// 5.4 TB/s; two of 131072: 87 us, 5.8 TB/s; 6 of up to 5000, 16 heads, 4 queries, d 256: 34
// us, 4.3 TB/s. The steady state takes the memory's whole rate (a tile per CTA in 2700 cycles,
// 2000 of them softmax); lost are 8 us until the first tiles are there, the spread of the
// CTAs' ends (4 us), the changes of row groups and the join (3 us).
//
// The work is a line of units, one per (sequence, KV head, chunk of rows, block of
// 64 tokens), cut into equal parts for the CTAs (mostly two per SM, so that one's
// row changes hide behind the other's stream) whatever the sequences' lengths; a
// row whose units fall to several CTAs is joined from their partial results by a
// second kernel. Short row groups stay whole, one CTA each.
//
// Warps: 0-3 softmax, 4 producer (block table, scales, TMA), 5 tensor-core issuer, 6
// Q (reads, splits and lays out the next row group's queries).
#include "fa_cache8.cuh"

namespace fa {
namespace {

constexpr int kThreads = 224;
constexpr float kTrail = 3.f;             // log2 of how far a reference may trail
constexpr float kShift = 5.f;             // y = 2^(x - reference + kShift) <= 2^8
constexpr float kNoKey = -1.f;            // factor of O for a row that sees no key
constexpr int kWholeBlocks = 8;
constexpr int kTurn = 4;                  // blocks' time that a change of row groups costs
constexpr int kInfo = 8;                  // tiles whose scales wait in shared memory

// Whether `mine` holds for any of the softmax warps' 128 threads, which meet here.
__device__ __forceinline__ bool meet_or(bool mine) {
  int any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
      "selp.b32 %0, 1, 0, q;\n\t}"
      : "=r"(any) : "r"(static_cast<int>(mine)) : "memory");
  return any != 0;
}
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
               : "r"(taddr));
}
// Makes the registers depend on the tcgen05.wait::ld before.
__device__ __forceinline__ void reg_fence_x16(uint32_t (&r)[16]) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]) :: "memory");
}
__device__ __forceinline__ void store_byte(uint32_t addr, uint32_t x) {
  asm volatile("st.shared.b8 [%0], %1;" :: "r"(addr), "r"(x) : "memory");
}
// O of a row that sees no key is 0 whatever V holds: its P is 0, but 0 x NaN is not. (By a mark of its own: the
// factor of V scales of 0 is 0 as well.)
__device__ __forceinline__ float times_factor(float o, float factor) { return factor == kNoKey ? 0.f : o * factor; }
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

// The line of units: for sequence after sequence, row group (KV head, chunk)
// after row group, its blocks. A sequence has at least one block of units, so
// that rows without keys are written too.
__device__ __forceinline__ int blocks_of(int len) { return max(1, (len + kCacheBlock - 1) / kCacheBlock); }
__device__ __forceinline__ int line_blocks(const Cache8Params& p, int b) {
  return blocks_of(cache_length(p.lengths, b, p.max_blocks));
}
// All units; by a whole warp.
__device__ __forceinline__ int line_total(const Cache8Params& p, int lane) {
  int sum = 0;
  for (int b = lane; b < p.B; b += 32) sum += line_blocks(p, b);
  return __reduce_add_sync(0xffffffffu, sum) * p.c.Hkv * p.chunks;
}
// The line cut into equal parts for a grid of `ctas`. It is measured in units,
// but a CTA that goes on to another row group loses the time of a few blocks
// with the one's results and the other's queries: `turn` places more lie ahead
// of each group's units. (With units alone CTAs with three groups ended 6 us
// after those with one, of 59. Turns of 3 and 4 blocks measure alike, 2 and 8 slower.) A part is at least
// twice a turn long, so that it has units, and where it begins in a turn its
// first units are that group's; hence every part between a group's first and
// last has a partial result of it.
struct Line {
  int turn, total, parts;
  __device__ __forceinline__ Line(const Cache8Params& p, int units, int ctas) {
    turn = units >> 28 ? 0 : min(kTurn, units / (2 * ctas));
    total = units + turn * p.B * p.c.Hkv * p.chunks;
    parts = min(ctas, total);
  }
  __device__ __forceinline__ int begin(int i) const {
    return static_cast<int>(static_cast<long long>(total) * i / parts);
  }
  // the part that place u belongs to
  __device__ __forceinline__ int part_of(int u) const {
    return static_cast<int>(((u + 1LL) * parts - 1) / total);
  }
};

// A place on the line.
struct Place {
  int b, before;             // sequence, places before it
  int nblk, len;             // its blocks of units and tokens
  int turn;                  // as the line's; 0: places are units
  __device__ __forceinline__ void load(const Cache8Params& p) {
    len = cache_length(p.lengths, b, p.max_blocks);
    nblk = blocks_of(len);
  }
  // to the sequence of place u, by a whole warp
  __device__ __forceinline__ void find(const Cache8Params& p, int u, int lane) {
    const int per_block = p.c.Hkv * p.chunks;
    int base = 0;
    b = p.B - 1;
    before = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int cnt = b0 + lane < p.B ? line_blocks(p, b0 + lane) + turn : 0;
      int incl = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, u < (base + incl) * per_block);
      if (hit) {
        const int src = __ffs(hit) - 1;
        b = b0 + src;
        before = (base + __shfl_sync(0xffffffffu, incl - cnt, src)) * per_block;
        break;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    load(p);
  }
  // to the first place of part `i` of `ctas`, whose places are [u0, u1); false: no such part. By a
  // whole warp; one look at the lengths where a warp holds them all.
  __device__ __forceinline__ bool start(const Cache8Params& p, int i, int ctas, int lane, int& u0, int& u1) {
    const int per_block = p.c.Hkv * p.chunks;
    if (p.whole) {                                       // (the grid is B * per_block)
      b = i / per_block;
      load(p);
      turn = before = 0;
      if (p.scores != nullptr) {
        for (int x = lane; x < b; x += 32) before += line_blocks(p, x);
        before = __reduce_add_sync(0xffffffffu, before) * per_block;
      }
      u0 = before + (i - b * per_block) * nblk;
      u1 = u0 + nblk;
      return true;
    }
    int mine = 0, units;
    if (p.B <= 32) {
      mine = lane < p.B ? cache_length(p.lengths, lane, p.max_blocks) : -1;
      units = __reduce_add_sync(0xffffffffu, mine < 0 ? 0 : blocks_of(mine)) * per_block;
    } else {
      units = line_total(p, lane);
    }
    const Line line(p, units, ctas);
    if (i >= line.parts) return false;
    u0 = line.begin(i);
    u1 = line.begin(i + 1);
    turn = line.turn;
    if (p.B > 32) {
      find(p, u0, lane);
      return true;
    }
    int incl = mine < 0 ? 0 : blocks_of(mine) + turn;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    b = __ffs(__ballot_sync(0xffffffffu, u0 < incl * per_block)) - 1;
    len = __shfl_sync(0xffffffffu, mine, b);
    nblk = blocks_of(len);
    before = (__shfl_sync(0xffffffffu, incl, b) - nblk - turn) * per_block;
    return true;
  }
  // onwards to the sequence of place u (one that exists)
  __device__ __forceinline__ void go(const Cache8Params& p, int u) {
    const int per_block = p.c.Hkv * p.chunks;
    while (u - before >= (nblk + turn) * per_block) {
      before += (nblk + turn) * per_block;
      ++b;
      load(p);
    }
  }
};

// D: 128 or 256, d at most that; R: query rows a CTA takes at once, 4, 8 or 16; S: CTAs per SM.
template <int D, int R, int S>
struct Cfg {
  static_assert(R == 4 || R == 8 || R == 16, "rows");
  static constexpr int kChunks = D / 128;                  // 128-byte columns of K and V
  static constexpr int kNS = R < 8 ? 16 : 2 * R;           // S^T columns: two terms of Q (16 at least)
  static constexpr int kE = R < 8 ? R : 8;                 // rows dealt with together
  static constexpr int kNP = (3 * R + 15) / 16 * 16;       // O^T columns: three terms of P
  static constexpr int kPerSm = S;
  static constexpr int kTile = 16384 * kChunks;            // K or V of a tile
  static constexpr int kQBufs = 2;
  static constexpr int kQBytes = kNS * 128 * kChunks;
  static constexpr int kPBytes = kNP * 128;
  // references and their changes (4 R), the warps' maxima and sums (8 R), 1 / scale of Q per buffer
  static constexpr int kStatFloats = 4 * R + 8 * R + 2 * R;
  static constexpr int kFixed = kQBufs * kQBytes + 2 * kPBytes + kStatFloats * 4 + kInfo * 32 + 320;
  static constexpr int kBudget = (S == 3 ? 75 : S == 2 ? 113 : 227) * 1024;
  static constexpr int kFit = (kBudget - kFixed) / kTile;
  static constexpr int kRing = kFit < 8 ? kFit : 8;        // tiles of K or V
  static constexpr int kLayout = kRing * kTile + kFixed;
  static constexpr int kSmem = kLayout + 1024 <= kBudget ? kLayout + 1024 : kBudget;   // + what the base's alignment may take
  static constexpr uint32_t kColO = 2 * kNS;
  static constexpr int kCols = 2 * kNS + kNP * kChunks;
  static constexpr uint32_t kTmem = kCols <= 64 ? 64 : kCols <= 128 ? 128 : kCols <= 256 ? 256 : 512;
  static_assert(kRing >= 3 && kTmem * kPerSm <= 512, "shared memory or TMEM budget");
};

// A row group's share of a part: blocks [blk0, blk1) of (b, h, chunk), none where the
// part ends in the group's turn.
struct Segment {
  int b, h, chunk, blk0, blk1, nblk, len, tiles;
  int unit0;                 // units of the line before the group's
  int next;                  // place where the next segment begins
  __device__ __forceinline__ Segment(const Cache8Params& p, Place& at, int u, int u1) {
    at.go(p, u);
    b = at.b;
    nblk = at.nblk;
    len = at.len;
    const int span = nblk + at.turn, row = (u - at.before) / span;     // head * chunks + chunk
    const int off = u - at.before - row * span;
    next = min(u1, u + span - off);
    blk0 = max(0, off - at.turn);
    blk1 = off + (next - u) - at.turn;
    unit0 = at.before - at.turn * b * p.c.Hkv * p.chunks + row * nblk;
    h = row / p.chunks;
    chunk = row - h * p.chunks;
    tiles = (blk1 - blk0 + 1) / 2;
  }
};

template <int D, int R, int S>
__global__ void __launch_bounds__(kThreads, Cfg<D, R, S>::kPerSm)
cache8_fwd_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const Cache8Params p) {
  using C = Cfg<D, R, S>;
  extern __shared__ uint8_t smem_raw[];
  // This kernel may have been set up while the one before it still ran: nothing
  // in memory is read or written ahead of that one's end. From then on the second
  // kernel may be set up, which so may read what the caller's kernels wrote.
  wait_before();
  let_next();
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  if ((base - raw) + C::kLayout > static_cast<uint32_t>(C::kSmem)) {
    // the layout needs the dynamic window to start near a 1 KB boundary
    if (threadIdx.x == 0) atomicOr(p.status, kDevLayout);
    return;
  }
  const uint32_t s_q = base + C::kRing * C::kTile, s_p = s_q + C::kQBufs * C::kQBytes;
  auto s_kv = [&](int i) { return base + i * C::kTile; };
  constexpr int kOffStat = C::kRing * C::kTile + C::kQBufs * C::kQBytes + 2 * C::kPBytes;
  float* const ref_l = reinterpret_cast<float*>(gbase + kOffStat);     // [R] ml, then mo
  float* const ref_o = ref_l + R;
  float* const change_l = ref_o + R;                                   // [R] factors of the last change
  float* const change_o = change_l + R;
  float* const warp_l = change_o + R;                                  // [4][R] maxima of the warps (ml, mo); sums
  float* const warp_o = warp_l + 4 * R;
  float* const q_scale = warp_o + 4 * R;                               // [2][R] power of two the row was divided by
  volatile float* const info = reinterpret_cast<volatile float*>(q_scale + 2 * R);   // [kInfo][8]: per half K scale, V scale, there
  const uint32_t bars = base + kOffStat + C::kStatFloats * 4 + kInfo * 32;
  uint8_t* const gbars = gbase + (bars - base);
  auto bar_kv_full = [&](int i) { return bars + 8u * i; };             // 8
  auto bar_kv_empty = [&](int i) { return bars + 64u + 8u * i; };      // 8
  auto bar_info = [&](int i) { return bars + 128u + 8u * i; };         // kInfo
  auto bar_s_full = [&](int i) { return bars + 192u + 8u * i; };
  auto bar_p_ready = [&](int i) { return bars + 224u + 8u * i; };
  auto bar_p_empty = [&](int i) { return bars + 240u + 8u * i; };      // P V done
  auto bar_q_full = [&](int i) { return bars + 256u + 8u * i; };
  auto bar_q_empty = [&](int i) { return bars + 272u + 8u * i; };
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gbars + 296);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(gbars + 300);
  const uint32_t bar_stall = bars + 304;                               // nothing arrives (timeout test)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // (All warps find the part by the same code: a copy of it in each role costs
  // more than it saves, since code, too, comes from memory the first time.)
  int u0, u1;                                            // this part's units
  Place at;
  if (!at.start(p, blockIdx.x, gridDim.x, lane, u0, u1)) return;
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    for (int i = 0; i < C::kRing; ++i) {
      mbar_init(bar_kv_full(i), 1);
      mbar_init(bar_kv_empty(i), 1);
    }
    for (int i = 0; i < kInfo; ++i) mbar_init(bar_info(i), 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_s_full(i), 1);
      mbar_init(bar_p_ready(i), 128);
      mbar_init(bar_p_empty(i), 1);
      mbar_init(bar_q_full(i), 1);
      mbar_init(bar_q_empty(i), 2);                      // its products done, its scales read
    }
    mbar_init(bar_stall, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), C::kTmem);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;

  if (warp == 4) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      tma_prefetch_map(&map_k);
      tma_prefetch_map(&map_v);
    }
    int c = 0, tile = 0;                                 // loads and tiles so far
    bool ok = true;
    for (int u = u0; u < u1 && ok;) {
      const Segment s(p, at, u, u1);
      const int* const table = p.table + static_cast<long long>(s.b) * p.max_blocks;
      const int held = (s.len + kCacheBlock - 1) / kCacheBlock;        // blocks with tokens (nblk but for an empty sequence)
      for (int blk = s.blk0; blk < s.blk1 && ok; blk += 32) {
        // 32 blocks at a time, one per lane
        const int mine = blk + lane;
        int page = mine < s.blk1 && mine < held ? table[mine] : -1;
        if (page >= p.c.num_blocks) page = -1;
        const long long ph = page >= 0 ? static_cast<long long>(page) * p.c.Hkv + s.h : -1;
        // (not by the read-only path: the append before may still have been writing them when this kernel was set up)
        const float ks = page >= 0 ? p.c.k_scale[ph] : 0.f, vs = page >= 0 ? p.c.v_scale[ph] : 0.f;
        const int z = static_cast<int>(ph);
        for (int i = 0; i < 32 && blk + i < s.blk1 && ok; i += 2, ++tile) {
          const int za = __shfl_sync(0xffffffffu, z, i), zb = __shfl_sync(0xffffffffu, z, i + 1);
          const int there = (za >= 0) + (zb >= 0);
          if (lane == 0) {
            for (int kv = 0; kv < 2 && ok; ++kv, ++c) {
              const int slot = c % C::kRing;
              ok = wait(bar_kv_empty(slot), ((c / C::kRing) & 1) ^ 1, abort_flag, p.timeout_ns);
              if (!ok) break;
              mbar_arrive_expect_tx(bar_kv_full(slot), there * 8192 * C::kChunks);
              const CUtensorMap* const m = kv ? &map_v : &map_k;
              for (int ch = 0; ch < C::kChunks; ++ch) {
                if (za >= 0) tma_load_3d(s_kv(slot) + ch * 16384, m, bar_kv_full(slot), ch * 128, 0, za);
                if (zb >= 0) tma_load_3d(s_kv(slot) + ch * 16384 + 8192, m, bar_kv_full(slot), ch * 128, 0, zb);
              }
            }
          }
          ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0);
          // (the scales come after the loads are on their way: nothing before them needs them)
          if (lane == i || lane == i + 1) {
            volatile float* const dst = info + (tile % kInfo) * 8 + (lane - i) * 4;
            dst[0] = ks;
            dst[1] = vs;
            dst[2] = page >= 0 ? 1.f : 0.f;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_info(tile % kInfo));
        }
      }
      u = s.next;
    }
    __syncwarp();
  } else if (warp == 5) {
    // ------------------------------------------------------------ tensor-core issuer
    if (lane == 0) {
      const uint32_t id_s = make_idesc(0, 128, C::kNS, 0, 0);          // K tile and Q: both K-major
      const uint32_t id_o = make_idesc(0, 128, C::kNP, 1, 0);          // V tile: d contiguous, hence MN-major
      const int steps = (p.c.d + 31) / 32;                             // products over d that are not all zeros
      int tile = 0, seg = 0;
      bool ok = !p.test_stall || wait(bar_stall, 0, abort_flag, p.timeout_ns);   // runs out by design
      // S^T of tile `t`, whose K is load 2 t, with the queries of segment `g`
      auto scores = [&](int t, int g) {
        const int slot = (2 * t) % C::kRing;
        // (its buffer is free: S of two tiles before was read ahead of that tile's P-ready, long waited for)
        ok = wait(bar_kv_full(slot), ((2 * t) / C::kRing) & 1, abort_flag, p.timeout_ns);
        if (!ok) return;
        tc_fence_after();
        const uint64_t kd = smem_desc_sw128(s_kv(slot), 16, 1024);
        const uint64_t qd = smem_desc_sw128(s_q + (g % C::kQBufs) * C::kQBytes, 16, 1024);
        for (int k = 0; k < steps; ++k)
          mma_fp8_ss(tbase + (t & 1) * C::kNS, desc_add(kd, (k >> 2) * 16384 + (k & 3) * 32),
                     desc_add(qd, (k >> 2) * (C::kNS * 128) + (k & 3) * 32), id_s, k > 0);
        mma_commit(bar_s_full(t & 1));
        mma_commit(bar_kv_empty(slot));
      };
      for (int u = u0; u < u1 && ok; ++seg) {
        const Segment s(p, at, u, u1);
        if (s.blk1 <= s.blk0) break;
        ok = wait(bar_q_full(seg % C::kQBufs), (seg / C::kQBufs) & 1, abort_flag, p.timeout_ns);
        if (!ok) break;
        scores(tile, seg);
        for (int j = 0; j < s.tiles && ok; ++j, ++tile) {
          if (j + 1 < s.tiles) scores(tile + 1, seg);
          else mma_commit(bar_q_empty(seg % C::kQBufs));
          if (!ok) break;
          const int slot = (2 * tile + 1) % C::kRing;
          ok = wait(bar_kv_full(slot), ((2 * tile + 1) / C::kRing) & 1, abort_flag, p.timeout_ns) &&
               wait(bar_p_ready(tile & 1), (tile >> 1) & 1, abort_flag, p.timeout_ns);
          if (!ok) break;
          tc_fence_after();
          const uint64_t pd = smem_desc_sw128(s_p + (tile & 1) * C::kPBytes, 16, 1024);
#pragma unroll
          for (int mb = 0; mb < C::kChunks; ++mb) {
            if (128 * mb >= p.c.d) continue;
            const uint64_t vd = smem_desc_sw128(s_kv(slot) + mb * 16384, 16384, 1024);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_fp8_ss(tbase + C::kColO + mb * C::kNP, desc_add(vd, k * 4096), desc_add(pd, k * 32), id_o, j > 0 || k > 0);
          }
          mma_commit(bar_p_empty(tile & 1));
          mma_commit(bar_kv_empty(slot));
        }
        u = s.next;
      }
    }
    __syncwarp();
  } else if (warp == 6) {
    // ------------------------------------------------------------ queries
    bool ok = true;
    int seg = 0;
    for (int u = u0; u < u1 && ok; ++seg) {
      const Segment s(p, at, u, u1);
      if (s.blk1 <= s.blk0) break;
      const int buf = seg % C::kQBufs;
      const size_t qrow = (static_cast<size_t>(s.b) * p.Hq + static_cast<size_t>(s.h) * p.G) * p.Nq + s.chunk * R;
      const int rows = min(R, p.R - s.chunk * R);
      ok = wait(bar_q_empty(buf), ((seg / C::kQBufs) & 1) ^ 1, abort_flag, p.timeout_ns);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t dst = s_q + buf * C::kQBytes;
      for (int q0 = 0; q0 < R; q0 += 8) {
        uint2 v[C::kE][C::kChunks];                      // the rows' loads on their way together
#pragma unroll
        for (int e = 0; e < C::kE; ++e)
#pragma unroll
          for (int ch = 0; ch < C::kChunks; ++ch) {
            const int col = 128 * ch + 4 * lane;
            v[e][ch] = make_uint2(0, 0);
            if (q0 + e < rows && col < p.c.d) v[e][ch] = *reinterpret_cast<const uint2*>(p.q + (qrow + q0 + e) * p.c.d + col);
          }
        float amax[C::kE];
#pragma unroll
        for (int e = 0; e < C::kE; ++e) {
          amax[e] = 0.f;
#pragma unroll
          for (int ch = 0; ch < C::kChunks; ++ch) {
            const uint32_t w[2] = {v[e][ch].x, v[e][ch].y};
#pragma unroll
            for (int k = 0; k < 2; ++k)
              amax[e] = fmaxf(amax[e], fmaxf(fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xFFFF0000u))));
          }
        }
        // (non-negative floats order like their bits)
#pragma unroll
        for (int e = 0; e < C::kE; ++e) amax[e] = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax[e])));
#pragma unroll
        for (int e = 0; e < C::kE; ++e) {
          const int q = q0 + e;
          // exponent that brings the largest to [128, 256); bounded so that both powers are normal.
          // An infinity among them becomes NaN, as its logits are.
          const int e2 = amax[e] > 0.f ? max(-100, min(100, static_cast<int>(__float_as_uint(amax[e]) >> 23) - 127 - 7)) : 0;
          const float down = amax[e] < INFINITY ? __uint_as_float(static_cast<uint32_t>(127 - e2) << 23) : NAN;
          if (lane == 0) q_scale[buf * R + q] = __uint_as_float(static_cast<uint32_t>(127 + e2) << 23);
#pragma unroll
          for (int ch = 0; ch < C::kChunks; ++ch) {
            const uint32_t w[2] = {v[e][ch].x, v[e][ch].y};
            uint32_t hi = 0, lo = 0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float a = __uint_as_float(w[k] << 16) * down, b = __uint_as_float(w[k] & 0xFFFF0000u) * down;
              const uint32_t c0 = pack_e4m3x2(a, b);
              const float2 f = e4m3x2_to_float2(c0);
              hi |= c0 << (16 * k);
              lo |= pack_e4m3x2((a - f.x) * 16.f, (b - f.y) * 16.f) << (16 * k);
            }
            // row q (first terms) and row R + q (second) of the operand, bytes 4 lane .. + 3
            const uint32_t box = dst + ch * (C::kNS * 128);
            asm volatile("st.shared.b32 [%0], %1;" :: "r"(swz128(box, q, lane >> 2) + (lane & 3) * 4), "r"(hi) : "memory");
            asm volatile("st.shared.b32 [%0], %1;" :: "r"(swz128(box, R + q, lane >> 2) + (lane & 3) * 4), "r"(lo) : "memory");
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_q_full(buf));
      u = s.next;
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax
    const int row = threadIdx.x;                         // token of the tile; column of d in the epilogue
    const int half = row >> 6;
    const uint32_t lane_off = static_cast<uint32_t>(warp * 32) << 16;
    bool ok = true;
    int tile = 0, seg = 0;
    if (row < R) ref_l[row] = ref_o[row] = -INFINITY;
    named_bar_sync(1, 128);
    int u = u0;
    Segment s(p, at, u0, u1);
    for (; u < u1 && s.blk1 > s.blk0; ++seg) {
      const int row0 = s.chunk * R;
      const int all = p.causal ? max(0, s.len - p.Nq + 1) : s.len;     // keys below it are visible to every row
      float l[R];
#pragma unroll
      for (int q = 0; q < R; ++q) l[q] = 0.f;
      const float* const qs = q_scale + (seg % C::kQBufs) * R;
      // where there are registers to spare, the references and the queries' scales stay in them between
      // their changes (65.4 -> 64.7 us over 32 sequences; 16 rows of d 256 52 -> 46)
      constexpr bool kKeep = R * S <= 16;
      float ml[kKeep ? R : 1], mo[kKeep ? R : 1], sq[kKeep ? R : 1];
#pragma unroll
      for (int q = 0; q < (kKeep ? R : 1); ++q) {
        ml[q] = mo[q] = -INFINITY;
        sq[q] = 0.f;
      }
      auto top_l = [&](int q) { return kKeep ? ml[kKeep ? q : 0] : ref_l[q]; };
      auto top_o = [&](int q) { return kKeep ? mo[kKeep ? q : 0] : ref_o[q]; };
      auto scale_q = [&](int q) { return kKeep ? sq[kKeep ? q : 0] : qs[q]; };
      for (int j = 0; j < s.tiles; ++j, ++tile) {
        const int buf = tile & 1;
        // the queries' scales are there when their operand is
        if (ok && j == 0) ok = wait(bar_q_full(seg % C::kQBufs), (seg / C::kQBufs) & 1, abort_flag, p.timeout_ns);
        if (ok)
          ok = wait(bar_info(tile % kInfo), (tile / kInfo) & 1, abort_flag, p.timeout_ns) &&
               wait(bar_s_full(buf), (tile >> 1) & 1, abort_flag, p.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (kKeep && j == 0) {
#pragma unroll
          for (int q = 0; q < R; ++q) sq[kKeep ? q : 0] = qs[q];
        }
        const float ks = info[(tile % kInfo) * 8 + half * 4] * p.scale_log2;
        const float vs = info[(tile % kInfo) * 8 + half * 4 + 1];
        const int blk = s.blk0 + 2 * j + half;
        const int key = blk * kCacheBlock + (row & 63);
        // tokens past the length, of no block, or of another CTA's block are absent
        const bool there = blk < s.blk1 && key < s.len && info[(tile % kInfo) * 8 + half * 4 + 2] != 0.f;
        const float lvs = log2f(vs);
        float x[R];
        bool grow = !ok;
        if (ok) {
          tc_fence_after();
          uint32_t hi[16], lo[16];                       // both terms
          tmem_ld_x16(tbase + lane_off + buf * C::kNS, hi);
          if (R > 8) tmem_ld_x16(tbase + lane_off + buf * C::kNS + R, lo);
          tmem_wait_ld();
          reg_fence_x16(hi);
          if (R > 8) reg_fence_x16(lo);
#pragma unroll
          for (int q = 0; q < R; ++q)
            x[q] = fmaf(__uint_as_float(R > 8 ? lo[q] : hi[(R + q) % 16]), 0.0625f, __uint_as_float(hi[q])) * (ks * scale_q(q));
          tc_fence_before();
          if (!there || key >= all) {
            // row row0 + q is query (row0 + q) % Nq of its head, and sees the keys up to its own position
            int query = p.causal ? row0 % p.Nq : p.Nq - 1;
#pragma unroll
            for (int q = 0; q < R; ++q) {
              x[q] = there && key <= s.len - p.Nq + query ? x[q] : -INFINITY;
              if (p.causal && ++query == p.Nq) query = 0;
            }
          }
#pragma unroll
          for (int q = 0; q < R; ++q) grow |= x[q] > top_l(q) + kTrail || x[q] + lvs > top_o(q) + kTrail;
        }
        if (j == 0 || meet_or(grow)) {
          // the tile's maxima, as integers of the floats' order
#pragma unroll
          for (int q = 0; q < R; ++q) {
            auto most = [&](float v) {
              const uint32_t b = __float_as_uint(v);
              // (a NaN takes no part: it would raise the reference for good)
              const uint32_t key_of = v != v ? 0u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
              const uint32_t top = __reduce_max_sync(0xffffffffu, key_of);
              return top == 0u ? -INFINITY : __uint_as_float((top & 0x80000000u) ? top & 0x7FFFFFFFu : ~top);
            };
            const float a = most(x[q]);                  // (a warp's tokens are of one block: one V scale)
            if (lane == 0) {
              warp_l[warp * R + q] = a;
              warp_o[warp * R + q] = a + lvs;
            }
          }
          if (meet_or(!ok)) {                            // a wait ran out somewhere: all leave together
            ok = false;
            break;
          }
          if (row < R) {
            auto raise = [&](float* ref, const float* w, float* change) {
              const float old = ref[row];
              const float now = fmaxf(old, fmaxf(fmaxf(w[row], w[R + row]), fmaxf(w[2 * R + row], w[3 * R + row])));
              ref[row] = now;
              change[row] = now > old ? ex2_approx(old - now) : 1.f;
            };
            raise(ref_l, warp_l, change_l);
            raise(ref_o, warp_o, change_o);
          }
          named_bar_sync(1, 128);
#pragma unroll
          for (int q = 0; q < R; ++q) {
            l[q] *= change_l[q];
            if (kKeep) {
              ml[kKeep ? q : 0] = ref_l[q];
              mo[kKeep ? q : 0] = ref_o[q];
            }
          }
          if (j > 0) {
            // O <- O * change, once the P V before has completed
            ok = wait(bar_p_empty(buf ^ 1), ((tile - 1) >> 1) & 1, abort_flag, p.timeout_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (ok) {
              tc_fence_after();
#pragma unroll
              for (int mb = 0; mb < C::kChunks; ++mb)
#pragma unroll
                for (int c0 = 0; c0 < 3 * R; c0 += 8) {
                  uint32_t o[8];
                  const uint32_t col = tbase + lane_off + C::kColO + mb * C::kNP + c0;
                  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                               : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]), "=r"(o[7]) : "r"(col));
                  tmem_wait_ld();
                  asm volatile("" : "+r"(o[0]), "+r"(o[1]), "+r"(o[2]), "+r"(o[3]), "+r"(o[4]), "+r"(o[5]), "+r"(o[6]), "+r"(o[7]) :: "memory");
#pragma unroll
                  for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * change_o[(c0 + e) % R]);
                  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                               :: "r"(col), "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7]) : "memory");
                }
              tmem_wait_st();
              tc_fence_before();
            }
          }
        }
        if (p.scores != nullptr && blk < s.blk1) {
          // for the weights: this token's scores, -inf where hidden or absent
          float4* const keep =
              reinterpret_cast<float4*>(p.scores + (static_cast<size_t>(s.unit0 + blk) * kCacheBlock + (row & 63)) * p.score_row);
#pragma unroll
          for (int q = 0; q < R; q += 4)
            if (row0 + q < p.R) keep[q / 4] = make_float4(x[q], x[q + 1], x[q + 2], x[q + 3]);
        }
        // (the P V that read this buffer two tiles ago was issued ahead of this tile's S, so it has completed)
        const uint32_t dst = s_p + buf * C::kPBytes + (row & 15);
        const int unit = row >> 4;
#pragma unroll
        for (int q = 0; q < R; q += 2) {
          float y[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float a = top_l(q + e), c = top_o(q + e);
            l[q + e] += ex2_approx(x[q + e] - (a == -INFINITY ? 0.f : a));
            y[e] = ex2_approx(x[q + e] + (lvs - (c == -INFINITY ? 0.f : c) + kShift));
          }
          if (!there) y[0] = y[1] = 0.f;                 // (no block: no scale either)
          const uint32_t c0 = pack_e4m3x2(y[0], y[1]);
          const float2 f0 = e4m3x2_to_float2(c0);
          const float r0 = (y[0] - f0.x) * 32.f, r1 = (y[1] - f0.y) * 32.f;
          const uint32_t c1 = pack_e4m3x2(r0, r1);
          const float2 f1 = e4m3x2_to_float2(c1);
          const uint32_t c2 = pack_e4m3x2((r0 - f1.x) * 32.f, (r1 - f1.y) * 32.f);
          const uint32_t codes[3] = {c0, c1, c2};
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            // rows k R + q and k R + q + 1 of the operand, byte `row`
            store_byte(dst + (k * R + q) * 128 + ((unit ^ ((k * R + q) & 7)) << 4), codes[k]);
            store_byte(dst + (k * R + q + 1) * 128 + ((unit ^ ((k * R + q + 1) & 7)) << 4), codes[k] >> 8);
          }
        }
        if (!there) {
          // this token's V may be anything; P is 0, but 0 x NaN is not: clear it
          const int slot = (2 * tile + 1) % C::kRing;
          if (ok) ok = wait(bar_kv_full(slot), ((2 * tile + 1) / C::kRing) & 1, abort_flag, p.timeout_ns);
#pragma unroll
          for (int ch = 0; ch < C::kChunks; ++ch)
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (ok)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" :: "r"(s_kv(slot) + ch * 16384 + row * 128 + i * 16), "r"(0) : "memory");
        }
        fence_proxy_async_smem();
        if (ok) mbar_arrive(bar_p_ready(buf));
      }
      // ---------------------------------------------------------- the row group's result
      // (while the last P V runs) the sums over the tile's 128 tokens
#pragma unroll
      for (int q = 0; q < R; ++q) {
        float sum = l[q];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) warp_l[warp * R + q] = sum;
      }
      if (meet_or(!ok)) break;
      if (row == 0) mbar_arrive(bar_q_empty(seg % C::kQBufs));         // all have read the queries' scales
      const bool whole = s.blk0 == 0 && s.blk1 == s.nblk;
      const long long slot0 = (2LL * blockIdx.x + (u == u0 ? 0 : 1)) * R;
      const size_t qrow = (static_cast<size_t>(s.b) * p.Hq + static_cast<size_t>(s.h) * p.G) * p.Nq + row0;
      const int rows = min(R, p.R - row0);
      float* const factor = change_l;                    // of O, per row
      if (row < R) {
        const float sum = warp_l[row] + warp_l[R + row] + warp_l[2 * R + row] + warp_l[3 * R + row];
        const float ml = ref_l[row], mo = ref_o[row] - kShift;
        if (whole) {
          factor[row] = sum == 0.f ? kNoKey : ex2_approx(mo - ml) / sum;
          if (row < rows) p.lse[qrow + row] = sum == 0.f ? -INFINITY : (ml + log2f(sum)) * kLn2;
        } else {
          float* const s3 = p.part_s + (slot0 + row) * 3;
          s3[0] = ml;
          s3[1] = sum;
          s3[2] = mo;
        }
        ref_l[row] = ref_o[row] = -INFINITY;             // for the next row group
      }
      u = s.next;
      if (u < u1) s = Segment(p, at, u, u1);
      const int last = tile - 1;
      ok = wait(bar_p_empty(last & 1), (last >> 1) & 1, abort_flag, p.timeout_ns);
      if (meet_or(!ok)) break;
      tc_fence_after();
#pragma unroll
      for (int mb = 0; mb < C::kChunks; ++mb)
#pragma unroll
        for (int q0 = 0; q0 < R; q0 += 8) {
          uint32_t o[3][8];
#pragma unroll
          for (int k = 0; k < 3; ++k)
            asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                         : "=r"(o[k][0]), "=r"(o[k][1]), "=r"(o[k][2]), "=r"(o[k][3]), "=r"(o[k][4]), "=r"(o[k][5]), "=r"(o[k][6]), "=r"(o[k][7])
                         : "r"(tbase + lane_off + C::kColO + mb * C::kNP + k * R + q0));
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 3; ++k)
            asm volatile("" : "+r"(o[k][0]), "+r"(o[k][1]), "+r"(o[k][2]), "+r"(o[k][3]), "+r"(o[k][4]), "+r"(o[k][5]), "+r"(o[k][6]), "+r"(o[k][7]) :: "memory");
          const int col = 128 * mb + row;
          float v[C::kE];
#pragma unroll
          for (int e = 0; e < C::kE; ++e)
            v[e] = __uint_as_float(o[0][e]) + (__uint_as_float(o[1][e]) + __uint_as_float(o[2][e]) * 0.03125f) * 0.03125f;
          if (whole) {
            __nv_bfloat16* const dst = p.o + (qrow + q0) * p.c.d + col;
            if (col < p.c.d) {
#pragma unroll
              for (int e = 0; e < C::kE; ++e)
                if (q0 + e < rows) dst[e * p.c.d] = __float2bfloat16_rn(times_factor(v[e], factor[q0 + e]));
            }
          } else {
            float* const dst = p.part_o + (slot0 + q0) * D + col;
#pragma unroll
            for (int e = 0; e < C::kE; ++e) dst[e * D] = v[e];
          }
        }
      tc_fence_before();
    }
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    if (threadIdx.x == 0) atomicOr(p.status, kDevTimeout);
    abort_grace_period();
  }
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tbase, C::kTmem);
}

// ------------------------------------------------------------------ second kernel
// Joins the rows whose units went to several parts, and adds
// the weights: weight_j = decay weight_j + sum over the group's rows of
// 2^(s_rj - LSE_r), from the scores that the first kernel kept (the
// probabilities need the whole row's LSE; reading K again instead costs d
// bytes per token and head against 8 per row, mostly from L2).
constexpr int kFinishWarps = 4;
constexpr int kWeightCtas = 1216;        // 8 per SM
// Up to two rows per SM: four warps join a row, which has many parts then (128 rows of 19: 87.7 us
// for the call, 89.2 with one warp each); past that one warp (384 rows of two or three: 40.8 against 44.4).
constexpr int kJoinRows = 2 * kCache8Sms;

// Where a row's partial results lie.
struct RowParts {
  int c0, c1, first, cols, r;                            // parts c0 .. c1; in c0 it is that part's first row or not
  // `before`: units before the sequence (b, nblk); row r of its head h
  __device__ __forceinline__ RowParts(const Cache8Params& p, const Line& line, int before, int b, int nblk, int h, int row, int cols_)
      : cols(cols_), r(row % cols_) {
    const int ua = before + line.turn * b * p.c.Hkv * p.chunks + (h * p.chunks + row / cols_) * (nblk + line.turn);
    c0 = line.part_of(ua + line.turn);
    c1 = line.part_of(ua + line.turn + nblk - 1);
    first = line.begin(c0) >= ua ? 0 : 1;
  }
  __device__ __forceinline__ long long slot(int c) const { return (2LL * c + (c == c0 ? first : 0)) * cols + r; }
};

// kJoin: warps that join a row together, kFinishWarps or one each.
// Every CTA waits for the first kernel before it ends, also where nothing is left to join: what
// follows in the stream, or in a graph, is ordered behind this kernel alone, and would run beside the
// first one if this one could end before it.
template <int D, int kJoin>
__global__ void __launch_bounds__(kFinishWarps * 32, 8) cache8_finish_kernel(const Cache8Params p, int cols, int ctas, int shares) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int units = line_total(p, lane);                 // (lengths are the caller's: no need to wait for them)
  const Line line(p, units, ctas);
  const int per_block = p.c.Hkv * p.chunks;
  __shared__ float lse2[kCache8MaxRows];
  if (static_cast<int>(blockIdx.x) >= shares) {          // (the weights' CTAs first: they take longer)
    // ---- join: rows of the B * Hkv * R
    const int per_seq = p.c.Hkv * p.R;
    const int row = kJoin == 1 ? (static_cast<int>(blockIdx.x) - shares) * kFinishWarps + warp : static_cast<int>(blockIdx.x) - shares;
    const int b = row / per_seq, hr = row - b * per_seq;
    if (b >= p.B) {
      wait_before();
      return;
    }
    const int h = hr / p.R, r = hr - h * p.R;
    int before = 0;
    for (int i = lane; i < b; i += 32) before += line_blocks(p, i);
    before = __reduce_add_sync(0xffffffffu, before) * per_block;
    const int nblk = line_blocks(p, b);
    const RowParts rp(p, line, before, b, nblk, h, r, cols);
    wait_before();
    if (rp.c0 == rp.c1) return;                          // written whole
    // several parts a warp at a time, all their loads together
    constexpr int kPer = D / 128;                        // float4 per lane
    constexpr int kAtOnce = kJoin == 1 ? 3 : 8;
    float ml = -INFINITY, mo = -INFINITY, sum = 0.f;
    float4 a[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) a[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = rp.c0 + (kJoin == 1 ? 0 : warp); c <= rp.c1; c += kAtOnce * kJoin) {
      float s3[kAtOnce][3];
      float4 y[kAtOnce][kPer];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        const int ck = min(c + k * kJoin, rp.c1);
        const long long slot = rp.slot(ck);
        const bool mine = c + k * kJoin <= rp.c1;
#pragma unroll
        for (int e = 0; e < 3; ++e) s3[k][e] = mine ? p.part_s[slot * 3 + e] : e == 1 ? 0.f : -INFINITY;
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          y[k][i] = mine ? *reinterpret_cast<const float4*>(p.part_o + slot * D + 128 * i + 4 * lane)
                         : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float nl = ml, no = mo;
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        nl = fmaxf(nl, s3[k][0]);
        no = fmaxf(no, s3[k][2]);
      }
      sum = ml == -INFINITY ? sum : sum * ex2_approx(ml - nl);
      const float f0 = mo == -INFINITY ? 1.f : ex2_approx(mo - no);
      ml = nl;
      mo = no;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        a[i].x *= f0;
        a[i].y *= f0;
        a[i].z *= f0;
        a[i].w *= f0;
      }
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) {
        sum += s3[k][0] == -INFINITY ? s3[k][1] : s3[k][1] * ex2_approx(s3[k][0] - ml);
        const float f = s3[k][2] == -INFINITY ? 1.f : ex2_approx(s3[k][2] - mo);   // (no term yet: O is 0, or a NaN that stays)
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          a[i].x = fmaf(f, y[k][i].x, a[i].x);
          a[i].y = fmaf(f, y[k][i].y, a[i].y);
          a[i].z = fmaf(f, y[k][i].z, a[i].z);
          a[i].w = fmaf(f, y[k][i].w, a[i].w);
        }
      }
    }
    if constexpr (kJoin > 1) {
      __shared__ float4 sum_o[kFinishWarps][32 * kPer];
      __shared__ float sum_l[kFinishWarps], top_l[kFinishWarps], top_o[kFinishWarps];
#pragma unroll
      for (int i = 0; i < kPer; ++i) sum_o[warp][32 * i + lane] = a[i];
      if (lane == 0) {
        sum_l[warp] = sum;
        top_l[warp] = ml;
        top_o[warp] = mo;
      }
      __syncthreads();
      if (warp != 0) return;
      ml = fmaxf(fmaxf(top_l[0], top_l[1]), fmaxf(top_l[2], top_l[3]));
      mo = fmaxf(fmaxf(top_o[0], top_o[1]), fmaxf(top_o[2], top_o[3]));
      float fo[kFinishWarps];
      sum = 0.f;
#pragma unroll
      for (int w = 0; w < kFinishWarps; ++w) {
        sum += top_l[w] == -INFINITY ? sum_l[w] : sum_l[w] * ex2_approx(top_l[w] - ml);
        fo[w] = top_o[w] == -INFINITY ? 1.f : ex2_approx(top_o[w] - mo);
      }
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        a[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kFinishWarps; ++w) {
          const float4 y = sum_o[w][32 * i + lane];
          a[i].x = fmaf(fo[w], y.x, a[i].x);
          a[i].y = fmaf(fo[w], y.y, a[i].y);
          a[i].z = fmaf(fo[w], y.z, a[i].z);
          a[i].w = fmaf(fo[w], y.w, a[i].w);
        }
      }
    }
    const size_t at = (static_cast<size_t>(b) * p.Hq + static_cast<size_t>(h) * p.G) * p.Nq + r;
    const float f = sum == 0.f ? kNoKey : ex2_approx(mo - ml) / sum;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (128 * i + 4 * lane < p.c.d)
        *reinterpret_cast<uint2*>(p.o + at * p.c.d + 128 * i + 4 * lane) =
            make_uint2(pack_bf16x2(times_factor(a[i].x, f), times_factor(a[i].y, f)),
                       pack_bf16x2(times_factor(a[i].z, f), times_factor(a[i].w, f)));
    if (lane == 0) p.lse[at] = sum == 0.f ? -INFINITY : (ml + log2f(sum)) * kLn2;
    return;
  }
  // ---- weights: an equal share of the (sequence, KV head, block), two at a time,
  // one thread per token
  const int all = units / p.chunks;                      // (sequence, KV head, block)
  const int share = static_cast<int>(blockIdx.x);
  const int w0 = static_cast<int>(static_cast<long long>(all) * share / shares);
  const int w1 = static_cast<int>(static_cast<long long>(all) * (share + 1) / shares);
  if (w0 >= w1) {
    wait_before();
    return;
  }
  Place at;
  at.turn = 0;
  at.find(p, w0 * p.chunks, lane);                       // (sequences have `chunks` times as many units)
  const int half = threadIdx.x >> 6, slot = threadIdx.x & 63;
  wait_before();
  for (int u = w0; u < w1;) {
    // the blocks of one head from u on
    at.go(p, u * p.chunks);
    const int in_seq = u - at.before / p.chunks;
    const int h = in_seq / at.nblk, blk0 = in_seq - h * at.nblk;
    const int blk1 = min(at.nblk, blk0 + (w1 - u));
    __syncthreads();
    for (int r = warp; r < p.R; r += kFinishWarps) {
      // a row in several parts is being joined by another CTA: its LSE from the parts, one per lane
      const RowParts rp(p, line, at.before, at.b, at.nblk, h, r, cols);
      float v;
      if (p.whole || rp.c0 == rp.c1) {
        v = p.lse[(static_cast<size_t>(at.b) * p.Hq + static_cast<size_t>(h) * p.G) * p.Nq + r] * kLog2e;
      } else {
        float ml = -INFINITY, sum = 0.f;
        for (int c = rp.c0 + lane; c <= rp.c1; c += 32) {
          const float* const s3 = p.part_s + rp.slot(c) * 3;
          const float m = s3[0], s = s3[1], now = fmaxf(ml, m);
          sum = (ml == -INFINITY ? sum : sum * ex2_approx(ml - now)) + (m == -INFINITY ? s : s * ex2_approx(m - now));
          ml = now;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const float m = __shfl_xor_sync(0xffffffffu, ml, o), s = __shfl_xor_sync(0xffffffffu, sum, o), now = fmaxf(ml, m);
          sum = (ml == -INFINITY ? sum : sum * ex2_approx(ml - now)) + (m == -INFINITY ? s : s * ex2_approx(m - now));
          ml = now;
        }
        v = sum == 0.f ? -INFINITY : ml + log2f(sum);
      }
      if (lane == 0) lse2[r] = v == -INFINITY ? INFINITY : v;   // a row that sees no key adds nothing
    }
    __syncthreads();
    // four blocks a thread at a time, the tables' entries and the scores together; then the weights
    for (int blk = blk0 + half; blk < blk1; blk += 8) {
      int page[4];
      float sum[4];
      bool there[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int bk = blk + 2 * k;
        there[k] = bk < blk1 && bk * kCacheBlock + slot < at.len;
        page[k] = there[k] ? p.table[static_cast<long long>(at.b) * p.max_blocks + bk] : -1;
        sum[k] = 0.f;
      }
      for (int chunk = 0; chunk < p.chunks; ++chunk) {
        const int rows = min(cols, p.R - chunk * cols);
        const size_t unit = static_cast<size_t>(at.before + (h * p.chunks + chunk) * at.nblk + blk);
        const float4* const x = reinterpret_cast<const float4*>(p.scores + (unit * kCacheBlock + slot) * p.score_row);
        const int step = 2 * kCacheBlock * p.score_row / 4;   // float4 from block to block
        for (int q = 0; q < rows; q += 4) {
          const float* const l = lse2 + chunk * cols + q;
          float4 y[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (there[k]) y[k] = x[k * step + q / 4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (there[k]) {
              sum[k] += ex2_approx(y[k].x - l[0]);
              if (q + 1 < rows) sum[k] += ex2_approx(y[k].y - l[1]);
              if (q + 2 < rows) sum[k] += ex2_approx(y[k].z - l[2]);
              if (q + 3 < rows) sum[k] += ex2_approx(y[k].w - l[3]);
            }
        }
      }
      float old[4];
      float* dst[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        old[k] = 0.f;
        there[k] = there[k] && page[k] >= 0 && page[k] < p.c.num_blocks;
        dst[k] = p.c.weight + (static_cast<size_t>(page[k]) * p.c.Hkv + h) * kCacheBlock + slot;
        // (a decay of 0 drops what was there, a NaN too)
        if (there[k] && p.decay != 0.f) old[k] = *dst[k];
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (there[k]) *dst[k] = p.decay * old[k] + sum[k];
    }
    u += blk1 - blk0;
  }
}

// CTAs per SM: at d 64 the softmax, not the memory, paces two of four rows each (32 and 256
// sequences of up to 4096 tokens 32 and 194 us, with three 30 and 162; at d 128 62 and 63; eight rows
// have no registers for three: 17 against 21 us for 8 sequences).
int cache8_per_sm(int d, int cols) { return d > 128 && cols > 8 ? 1 : d <= 64 && cols == 4 ? 3 : 2; }

template <int D, int R, int S>
cudaError_t launch_fwd(const CUtensorMap& mk, const CUtensorMap& mv, const Cache8Params& p, int parts, cudaStream_t stream) {
  static PerDeviceOnce attr;
  const cudaError_t e = attr.run([] {
    return cudaFuncSetAttribute(cache8_fwd_kernel<D, R, S>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, R, S>::kSmem);
  });
  if (e != cudaSuccess) return e;
  return launch_early(cache8_fwd_kernel<D, R, S>, dim3(parts), dim3(kThreads), Cfg<D, R, S>::kSmem, stream, mk, mv, p);
}

template <int D>
cudaError_t launch_all(const CUtensorMap& mk, const CUtensorMap& mv, const Cache8Params& p, int parts, cudaStream_t stream) {
  const int cols = cache8_columns(p.R);
  cudaError_t e = cudaErrorInvalidValue;
  if (cols == 4 && cache8_per_sm(p.c.d, cols) == 3) {
    if constexpr (D == 128) e = launch_fwd<D, 4, 3>(mk, mv, p, parts, stream);
  } else if (cols == 4) {
    e = launch_fwd<D, 4, 2>(mk, mv, p, parts, stream);
  } else if (cols == 8) {
    e = launch_fwd<D, 8, 2>(mk, mv, p, parts, stream);
  } else {
    e = launch_fwd<D, 16, D == 256 ? 1 : 2>(mk, mv, p, parts, stream);
  }
  if (e != cudaSuccess) return e;
  const int rows = parts > 1 && !p.whole ? p.B * p.c.Hkv * p.R : 0;
  const bool single = rows > kJoinRows;
  const int join = single ? (rows + kFinishWarps - 1) / kFinishWarps : rows;
  const long long blocks = static_cast<long long>(p.B) * p.c.Hkv * p.max_blocks;
  const int weigh = p.add_weights ? static_cast<int>(blocks < kWeightCtas ? blocks : kWeightCtas) : 0;
  if (join + weigh == 0) return cudaSuccess;
  return launch_early(single ? cache8_finish_kernel<D, 1> : cache8_finish_kernel<D, kFinishWarps>, dim3(join + weigh),
                      dim3(kFinishWarps * 32), 0, stream, p, cols, parts, weigh);
}

}  // namespace

// CTAs that run at once
static int cache8_wave(int d, int cols) { return kCache8Sms * cache8_per_sm(d, cols); }

// Rows a CTA takes at once: as many as there are up to 16, past that 16 or 8, whichever leaves fewer
// empty. 16 sequences of up to 8000, d 128: 32 rows by 16 93 us, by 8 101, by 32 118 (its softmax has too few
// registers); 20 rows 90, 79, 113; 40 rows 130, 124, 190. K and V come from L2 again for the others.
int cache8_columns(int R) { return R <= 4 ? 4 : (R - 1) / 8 % 2 == 0 ? 8 : 16; }

// Short row groups: one CTA each, as they come, and no second launch (4 us less for the caller).
// GPU time in us, 64 heads on 8, against cut and joined. Up to 8 blocks: 8 groups of 4 and 8
// 6.7 and 8.7 against 8.7 and 8.8, 128 groups 8.3 and 10.3 against 14.1 and 14.3, 1024 30 and 40
// against 42 and 55; at d 256 384 groups 14.5 and 23 against 20 and 26.5. Up to 16 at d 128 with more
// groups than SMs: 240, 384 and 1024 groups 16, 29 and 61 against 21, 29 and 66 (8 groups 12.8
// against 9.8; d 256 45 against 41; 32 blocks 29, 51 and 105 against 33, 44 and 94). By the table's width,
// since the lengths are on the device: eight sequences of 300 tokens under a wider table lose those 4 us.
bool cache8_whole(int B, int Hkv, int d, int R, int max_blocks) {
  const int cols = cache8_columns(R), chunks = (R + cols - 1) / cols;
  const bool many = static_cast<long long>(B) * Hkv * chunks > kCache8Sms && d <= 128;
  return max_blocks <= (many ? 2 * kWholeBlocks : kWholeBlocks);
}

int cache8_parts(int B, int Hkv, int d, int R, int max_blocks) {
  const int cols = cache8_columns(R), chunks = (R + cols - 1) / cols;
  const long long groups = static_cast<long long>(B) * Hkv * chunks, units = groups * max_blocks;
  if (cache8_whole(B, Hkv, d, R, max_blocks)) return static_cast<int>(groups);
  const int most = cache8_wave(d, cols);
  return static_cast<int>(units < most ? units : most);
}

cudaError_t launch_cache8_fwd(const CUtensorMap& mk, const CUtensorMap& mv, Cache8Params p, cudaStream_t stream) {
  p.whole = cache8_whole(p.B, p.c.Hkv, p.c.d, p.R, p.max_blocks) ? 1 : 0;
  const int parts = cache8_parts(p.B, p.c.Hkv, p.c.d, p.R, p.max_blocks);
  return p.c.d <= 128 ? launch_all<128>(mk, mv, p, parts, stream) : launch_all<256>(mk, mv, p, parts, stream);
}

}  // namespace fa
