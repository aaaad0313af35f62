// Forward over packed sequences of different lengths, bf16, d <= 128: the tile
// algorithm of fa_fwd.cu (two 128-row query tiles per CTA in ping-pong on the
// tensor core, K and V through one ring that both read) in a persistent grid
// of one CTA per SM.
//
// Why persistent. Sequences of a few hundred rows make items of a few key tiles,
// and a CTA of its own for each spent 13,000 cycles around them: finding its
// sequence, TMEM and barriers, the first loads, the store. Here a scheduler
// warp finds the next items ahead of time, the producer loads their Q, K and
// V while the last ones are worked on, and the issuer puts the next item's
// first S right behind the last P V.
//
// Items. Two query tiles that read the same K and V: where a KV head has an even
// number of query heads, the same tile of two of them (both see the same key
// tiles, so neither group idles at the diagonal); otherwise two neighbouring
// tiles of one head. Item r of the line is (tile or tile pair, sequence) number
// r / inner in the order of the tile's index, largest first (causal: those
// with the most key tiles first), and head (pair) r % inner. CTA c takes item
// c of the first round of gridDim.x items, the c-th from the end of the second, and so
// on: costs fall along the line, so the two directions even out.
//
// What bounds it (64 heads on 8, d 128, causal, 16384 rows). A step of two tiles takes about
// 2700 cycles where the tensor core needs 2048: the issuing thread's pace, as in fa_fwd.cu. Around
// an item 2800 more: the diagonal tile's softmax (700 above the others'), its P V with nothing
// beside it, and O's way out (1900 to 3000, through 4 KB per warp, whose second half is read
// and packed while the TMA unit takes the first; 16-byte stores from registers take 10% longer,
// coalesced ones through the same 4 KB 30%). Sequences of 128, 512, 1024, 2048, 8192 rows: 130, 188,
// 264, 420, 1400 us, the last at 1.57 PFLOP/s; 24 of 32 to 1593 rows 297 us (0.91 PFLOP/s of what
// the causal rule needs, 1.15 with the diagonal tiles whole). Up to 128 rows the bytes of Q and O
// bound it (4.6 TB/s).
//
// Warps: 0-3 and 4-7 the two softmax groups (one thread per query row), 8 TMA
// producer, 9 tensor-core issuer, 10 ring watcher, 11 scheduler. Barriers and
// parities run on across items; the steps within an item are as in fa_fwd.cu, but
// O has staging of its own, 4 KB per softmax warp, so that the next item's Q
// can be loaded over this one's while O leaves.
#include "fa_common.cuh"
#include "fa_kernels.h"

namespace fa {
namespace {

template <int D>
struct Cfg {
  static constexpr int kNBox = D / 64;                     // 128-byte swizzled boxes per 128-row tile
  static constexpr int kTileBytes = kNBox * kBoxBytes;
  static constexpr int kStages = D == 64 ? 10 : 4;         // K / V ring slots, what shared memory holds
  static constexpr int kOutBytes = 8 * 4096;               // per softmax warp 32 rows x 64 columns of O
  static constexpr int kThreads = 384;
  // setmaxnreg: 256 x 184 + 128 x 120 of the 384 x 168 launched
  static constexpr uint32_t kRegsSoftmax = 184, kRegsOther = 120;
  static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= 384 * 168, "register split");
  static constexpr int kBarBytes = 512;
  static constexpr int kSmem = (2 + kStages) * kTileBytes + kOutBytes + kBarBytes + 1024;
  static_assert(kSmem <= 227 * 1024, "shared memory budget");
  static __device__ __forceinline__ uint32_t col_s(int i) { return 128u * i; }
  static __device__ __forceinline__ uint32_t col_o(int i) { return 256u + D * i; }
};
constexpr int kItems = 4;                                  // items the scheduler may be ahead
constexpr int kReaders = 11;                               // producer, issuer, watcher, 8 softmax warps

struct Item {
  int start, len;                                          // the sequence's first row and length
  int tile;                                                // tile (two heads) or tile pair (one head); -1: no more items
  int head;                                                // head pair or head
};

__device__ __forceinline__ void sequence(const FwdParams& p, int s, int& start, int& len) {
  start = max(0, min(p.cu[s], p.T));
  len = max(0, min(p.cu[s + 1], p.T) - start);
}

// Finds items in the line's order, by one warp: C(w) = sum_s max(0, n_s - w)
// counts the (sequence, tile) of index w or more; the r-th has the index w with
// C(w) > r >= C(w + 1). r only grows, so w only falls. The first 256
// sequences' counts stay in registers, 8 per lane; others are read again. Within an
// index the sequence only grows too, and each look-up goes on from where the one before
// ended: from the first sequence on every time, 16384 of four rows took 61 ms, now 4.9, and the time grew with the
// square of their number, up to look-ups that outlast the other warps' waits.
struct Finder {
  const FwdParams& p;
  const int unit, lane;
  int n[8];
  int w, above;                                            // index, C(w + 1)
  int upto;                                                // C(w)
  int at, before;                                          // the last look-up's 32 sequences; how many before them have more than w tiles
  __device__ __forceinline__ int tiles(int s) const {
    if (s >= p.S) return 0;
    int start, len;
    sequence(p, s, start, len);
    return (len + unit - 1) / unit;
  }
  __device__ __forceinline__ int count(int x) const {
    int c = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) c += max(0, n[i] - x);
    for (int s = 256 + lane; s < p.S; s += 32) c += max(0, tiles(s) - x);
    return __reduce_add_sync(0xffffffffu, c);
  }
  __device__ __forceinline__ Finder(const FwdParams& pp, int u, int l) : p(pp), unit(u), lane(l) {
    int top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      n[i] = tiles(32 * i + lane);
      top = max(top, n[i]);
    }
    for (int s = 256 + lane; s < p.S; s += 32) top = max(top, tiles(s));
    w = __reduce_max_sync(0xffffffffu, top);
    above = upto = 0;                                      // nothing has index w
    at = before = 0;
  }
  // r >= the r of earlier calls; false: there are not that many
  __device__ __forceinline__ bool find(int r, Item& it) {
    if (r >= upto) {
      // the largest x below w with C(x) > r, by halving
      int lo = 0, hi = w;
      if (w == 0 || count(0) <= r) return false;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (count(mid) > r) lo = mid;
        else hi = mid;
      }
      w = lo;
      above = count(lo + 1);
      upto = count(lo);
      at = before = 0;
    }
    int k = r - above - before;                            // of those from `at` on, the k-th sequence with more than w tiles
    for (int s0 = at; s0 < p.S; s0 += 32) {
      int np = 0;
      if (s0 < 256) {
#pragma unroll
        for (int i = 0; i < 8; ++i) np = s0 == 32 * i ? n[i] : np;
      } else {
        np = tiles(s0 + lane);
      }
      unsigned hit = __ballot_sync(0xffffffffu, np > w);
      const int c = __popc(hit);
      if (k < c) {
        at = s0;
        for (; k > 0; --k) hit &= hit - 1;
        const int s = s0 + __ffs(hit) - 1;
        sequence(p, s, it.start, it.len);
        it.tile = w;
        return true;
      }
      k -= c;
      before += c;
    }
    return false;
  }
};

template <int D>
__device__ __forceinline__ void issue_qk(uint32_t d_tmem, uint64_t qd, uint64_t kd, uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t off = (kk * 32 / 128) * kBoxBytes + (kk * 32) % 128;
    mma_bf16_ss(d_tmem, desc_add(qd, off), desc_add(kd, off), idesc, kk > 0);
  }
}
__device__ __forceinline__ void issue_pv(uint32_t d_tmem, uint32_t p_tmem, uint64_t vd, uint32_t idesc, bool acc) {
#pragma unroll
  for (int kk = 0; kk < kBN / 16; ++kk) mma_bf16_ts(d_tmem, p_tmem + kk * 8, desc_add(vd, kk * 16 * 128), idesc, acc || kk > 0);
}

// Bounded wait whose limit starts at its own first look at the timer: a
// persistent CTA has no one deadline, and no register holds it in between.
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

template <int D>
__global__ void __launch_bounds__(384, 1)
fwd_packed_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_o, const FwdParams p) {
  using C = Cfg<D>;
  constexpr int kSt = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  const uint32_t s_kv = base + 2 * C::kTileBytes;
  auto s_q = [&](int i) { return base + i * C::kTileBytes; };
  const uint32_t s_out = s_kv + kSt * C::kTileBytes;
  const uint32_t bars = s_out + C::kOutBytes;
  uint8_t* const gbars = gbase + (bars - base);
  auto bar_q_empty = [&](int i) { return bars + 8u * i; };
  auto bar_s_full = [&](int i) { return bars + 16u + 8u * i; };
  auto bar_p_ready = [&](int i) { return bars + 32u + 8u * i; };
  auto bar_o_final = [&](int i) { return bars + 48u + 8u * i; };
  const uint32_t bar_q1_full = bars + 64u;               // Q of group 1 (group 0's lands on K_0's barrier)
  auto bar_item_full = [&](int i) { return bars + 112u + 8u * i; };
  auto bar_item_empty = [&](int i) { return bars + 112u + 8u * (kItems + i); };
  auto bar_kv_full = [&](int s) { return bars + 176u + 8u * s; };
  auto bar_kv_empty = [&](int s) { return bars + 176u + 8u * (kSt + s); };
  static_assert(176 + 16 * kSt <= 352, "barrier area");
  const uint32_t bar_stall = bars + 352;                             // nothing arrives (timeout test)
  uint32_t* const tmem_slot = reinterpret_cast<uint32_t*>(gbars + 360);
  volatile int* const abort_flag = reinterpret_cast<volatile int*>(gbars + 364);
  unsigned long long* const clock_start = reinterpret_cast<unsigned long long*>(gbars + 368);   // [2]
  volatile int* const items = reinterpret_cast<volatile int*>(gbars + 384);                    // [kItems][4]

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const bool two_heads = p.num_pairs != 0;               // an item is one tile of two heads
  const int group = p.Hq / p.Hkv;

  if (threadIdx.x == 0) {
    clock_mark(clock_start);
    *abort_flag = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_q_empty(i), 1);
      mbar_init(bar_s_full(i), 1);
      mbar_init(bar_p_ready(i), 129);                    // + the ring watcher
      mbar_init(bar_o_final(i), 1);
    }
    for (int i = 0; i < kItems; ++i) {
      mbar_init(bar_item_full(i), 1);
      mbar_init(bar_item_empty(i), kReaders);
    }
    for (int s = 0; s < kSt; ++s) {
      mbar_init(bar_kv_full(s), 1);
      mbar_init(bar_kv_empty(s), 1);
    }
    mbar_init(bar_q1_full, 1);
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

  // What a role has to know of an item.
  struct Work {
    int row0, len, nk;                                   // the sequence's rows and key tiles
    int qt[2], head[2], nkv[2], nmax;                    // per group; nkv = 0: the group has no tile
    int kv_head;
  };
  // Takes the n-th item (waits for it); false: there is none, or a wait ran
  // out. All threads that call it read the item before `release` says so.
  auto take = [&](int n, Work& w) -> bool {
    const int slot = n % kItems;
    if (!wait(bar_item_full(slot), (n / kItems) & 1, abort_flag, p.timeout_ns)) return false;
    const int tile = items[4 * slot + 2];
    if (tile < 0) return false;
    w.row0 = items[4 * slot];
    w.len = items[4 * slot + 1];
    const int head = items[4 * slot + 3];
    w.nk = (w.len + kBN - 1) / kBN;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w.qt[i] = two_heads ? tile : 2 * tile + i;
      w.head[i] = two_heads ? 2 * head + i : head;
      w.nkv[i] = w.qt[i] >= w.nk ? 0 : p.causal ? w.qt[i] + 1 : w.nk;
    }
    w.nmax = max(w.nkv[0], w.nkv[1]);
    w.kv_head = w.head[0] / group;
    return true;
  };
  auto release = [&](int n) { mbar_arrive(bar_item_empty(n % kItems)); };

  if (warp == 8) {
    // ------------------------------------------------------------ producer
    setmaxnreg_dec<C::kRegsOther>();
    if (lane == 0) {
      tma_prefetch_map(&map_q);
      tma_prefetch_map(&map_k);
      tma_prefetch_map(&map_v);
      Work w;
      int c = 0, nq[2] = {0, 0};                         // loads of the ring; Q tiles of each group
      bool ok = true;
      for (int n = 0; ok && take(n, w); ++n) {
        release(n);
        // The Q tiles can be loaded only when the last item's last S is done, and
        // come from device memory: into L2 with them meanwhile.
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (w.nkv[i] > 0)
            for (int bx = 0; bx < C::kNBox; ++bx)
              tma_prefetch_l2_3d(&map_q, bx * 64, w.row0 + w.qt[i] * kBM, w.head[i]);
        for (int x = 0; x < 2 * w.nmax && ok; ++x, ++c) {
          const int slot = c % kSt;
          ok = wait(bar_kv_empty(slot), ((c / kSt) & 1) ^ 1, abort_flag, p.timeout_ns);
          if (!ok) break;
          // K_0's barrier stands for group 0's Q tile too (the group always has one):
          // one wait before the item's first S
          mbar_arrive_expect_tx(bar_kv_full(slot), (x > 0 ? 1 : 2) * C::kTileBytes);
          const CUtensorMap* m = (x & 1) ? &map_v : &map_k;
          for (int bx = 0; bx < C::kNBox; ++bx)
            tma_load_3d(s_kv + slot * C::kTileBytes + bx * kBoxBytes, m, bar_kv_full(slot), bx * 64,
                        w.row0 + (x >> 1) * kBN, w.kv_head);
          if (x > 0) continue;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (!ok || w.nkv[i] == 0) continue;
            ok = wait(bar_q_empty(i), (nq[i] & 1) ^ 1, abort_flag, p.timeout_ns);
            if (!ok) continue;
            ++nq[i];
            const uint32_t bar = i ? bar_q1_full : bar_kv_full(slot);
            if (i) mbar_arrive_expect_tx(bar, C::kTileBytes);
            for (int bx = 0; bx < C::kNBox; ++bx)
              tma_load_3d(s_q(i) + bx * kBoxBytes, &map_q, bar, bx * 64, w.row0 + w.qt[i] * kBM, w.head[i]);
          }
        }
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ tensor-core issuer
    setmaxnreg_dec<C::kRegsOther>();
    if (lane == 0) {
      // The issuing thread paces the kernel (about 48 cycles per product of 64),
      // so the steps between an item's first and last two run in a loop of
      // their own without a decision in it, and slots are stepped, not divided.
      const uint32_t idesc_qk = make_idesc(1, 128, 128, 0, 0);
      const uint32_t idesc_pv = make_idesc(1, 128, D, 0, 1);
      const uint64_t qd0 = smem_desc_sw128(s_q(0), 16, 1024), qd1 = smem_desc_sw128(s_q(1), 16, 1024);
      const uint64_t kd = smem_desc_sw128(s_kv, 16, 1024), vd = smem_desc_sw128(s_kv, kBoxBytes, 1024);
      constexpr uint32_t kSlotDesc = C::kTileBytes >> 4;
      int slot = 0, round = 0;                           // of the next load to be used, and its use of the slot
      auto step_slot = [&](int by) {
        slot += by;
        if (slot >= kSt) {
          slot -= kSt;
          round ^= 1;
        }
      };
      uint32_t np0 = 0, np1 = 0, nq1 = 0;                // parities: P-ready of each group, Q of group 1
      bool ok = !p.test_stall || wait(bar_stall, 0, abort_flag, p.timeout_ns);   // runs out by design
      auto scores0 = [&]() {
        issue_qk<D>(tbase + C::col_s(0), qd0, kd + slot * kSlotDesc, idesc_qk);
        mma_commit(bar_s_full(0));
      };
      auto scores1 = [&]() {
        issue_qk<D>(tbase + C::col_s(1), qd1, kd + slot * kSlotDesc, idesc_qk);
        mma_commit(bar_s_full(1));
      };
      // S_i(0) of an item whose group i has n_i key tiles; early: S_0(0) is out already
      auto first_scores = [&](int n0, int n1, bool early) {
        if (!early) {
          ok = wait(bar_kv_full(slot), round, abort_flag, p.timeout_ns);
          if (!ok) return;
          tc_fence_after();
          scores0();
        }
        if (n1 > 0) {
          ok = wait(bar_q1_full, nq1, abort_flag, p.timeout_ns);
          if (!ok) return;
          nq1 ^= 1;
          tc_fence_after();
          scores1();
        }
        step_slot(1);
      };
      Work nx;
      int n = 0;
      bool have = ok && take(0, nx);
      if (have) {
        release(0);
        first_scores(nx.nkv[0], nx.nkv[1], false);
      }
      while (have && ok) {
        const int nkv0 = nx.nkv[0], nkv1 = nx.nkv[1], nmax = nx.nmax;
        ++n;
        have = take(n, nx);                              // the next one, while the softmax is at this one's first tile
        if (have) release(n);
        // V_j and K_{j+1} are there when P-ready is (the watcher's arrival). P-ready
        // of j = 0 also says that the group has read the last item's O.
        auto edge_step = [&](int j) {
          const uint64_t v0 = vd + slot * kSlotDesc;
          step_slot(1);
          if (j < nkv0) {
            ok = wait(bar_p_ready(0), np0, abort_flag, p.timeout_ns);
            if (!ok) return;
            np0 ^= 1;
            tc_fence_after();
            issue_pv(tbase + C::col_o(0), tbase + C::col_s(0), v0, idesc_pv, j > 0);
            if (j + 1 < nkv0) {
              scores0();
            } else {
              mma_commit(bar_o_final(0));
            }
          }
          // The next item's S_0(0) already here, if its tiles are: group 0
          // is at it while group 1 finishes. (Not if the next item has no group 1:
          // then its first S would stand for this item's last P V towards the watcher.)
          bool early = false;
          if (j + 1 == nmax && have && nx.nkv[1] > 0 && mbar_try_wait(bar_kv_full(slot), round)) {
            early = true;
            tc_fence_after();
            scores0();
          }
          if (j < nkv1) {
            ok = wait(bar_p_ready(1), np1, abort_flag, p.timeout_ns);
            if (!ok) return;
            np1 ^= 1;
            tc_fence_after();
            issue_pv(tbase + C::col_o(1), tbase + C::col_s(1), v0, idesc_pv, j > 0);
            if (j + 1 < nkv1) {
              scores1();
            } else {
              mma_commit(bar_o_final(1));
            }
          }
          if (j + 1 < nmax) step_slot(1);
          else if (have) first_scores(nx.nkv[0], nx.nkv[1], early);
        };
        edge_step(0);
        int j = 1;
        const int inner = min(nkv0, nkv1) - 1;           // both groups have two more steps
        for (; j < inner && ok; ++j) {
          const uint64_t v0 = vd + slot * kSlotDesc;
          step_slot(1);
          ok = wait(bar_p_ready(0), np0, abort_flag, p.timeout_ns);
          if (!ok) break;
          tc_fence_after();
          issue_pv(tbase + C::col_o(0), tbase + C::col_s(0), v0, idesc_pv, true);
          scores0();
          ok = wait(bar_p_ready(1), np1, abort_flag, p.timeout_ns);
          if (!ok) break;
          tc_fence_after();
          issue_pv(tbase + C::col_o(1), tbase + C::col_s(1), v0, idesc_pv, true);
          scores1();
          step_slot(1);
          np0 ^= 1;
          np1 ^= 1;
        }
        for (; j < nmax && ok; ++j) edge_step(j);
      }
    }
    __syncwarp();
  } else if (warp == 10) {
    // ------------------------------------------------------------ ring watcher
    // As in fa_fwd.cu: one arrival on P-ready(i) when V_j and K_{j+1} have
    // landed, and K_j and the load before it back to the producer when the
    // last S of step j, issued behind all their readers, is done. It waits for
    // every load in order, so no parity is taken for that of two phases earlier.
    setmaxnreg_dec<C::kRegsOther>();
    Work w;
    int c0 = 0;                                          // load number of the item's K_0
    int np0 = 0, np1 = 0, ns0 = 0, ns1 = 0;              // P-ready phases handed, S phases of each group
    bool ok = true;
    for (int n = 0;; ++n) {
      // lane 0 waits; the others come along for the items and the ragged tiles
      ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0);
      bool have = ok && take(n, w);
      have = __all_sync(0xffffffffu, have);
      if (!have) break;
      if (lane == 0) release(n);
      const int L = w.nkv[1] == w.nmax ? 1 : 0;          // the group whose S is issued last in a step
      const int nsl = L ? ns1 : ns0;
      auto hand = [&](int i, int& np) {
        // arrive for a phase only once the one before it has completed
        if (np > 0) ok = wait(bar_p_ready(i), (np - 1) & 1, abort_flag, p.timeout_ns);
        if (ok) mbar_arrive(bar_p_ready(i));
        ++np;
      };
      if (lane == 0) ok = wait(bar_kv_full(c0 % kSt), (c0 / kSt) & 1, abort_flag, p.timeout_ns);
      for (int j = 0; j < w.nmax; ++j) {
        const int cv = c0 + 2 * j + 1;
        if (lane == 0 && ok) ok = wait(bar_kv_full(cv % kSt), (cv / kSt) & 1, abort_flag, p.timeout_ns);
        if (j == w.nk - 1 && w.len % kBN != 0) {
          // The rows of V behind the sequence's end are another sequence's and
          // may hold anything; P is 0 there, but 0 x inf is not. The whole warp
          // clears them before the product may read the tile.
          ok = __shfl_sync(0xffffffffu, static_cast<int>(ok), 0);
          if (ok) {
            const int from = w.len % kBN;
            const uint32_t dst = s_kv + (cv % kSt) * C::kTileBytes + from * 128;
            const int units = (kBN - from) * 8;          // 16 bytes each, in every box
#pragma unroll
            for (int bx = 0; bx < C::kNBox; ++bx)
              for (int i = lane; i < units; i += 32)
                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" :: "r"(dst + bx * kBoxBytes + i * 16), "r"(0)
                             : "memory");
            fence_proxy_async_smem();
          }
          __syncwarp();
        }
        if (lane == 0 && ok) {
          if (j + 1 < w.nmax) ok = wait(bar_kv_full((cv + 1) % kSt), ((cv + 1) / kSt) & 1, abort_flag, p.timeout_ns);
          if (ok && L == 1 && j < w.nkv[0]) hand(0, np0);
          if (ok) ok = wait(bar_s_full(L), (nsl + j) & 1, abort_flag, p.timeout_ns);
          if (ok) {
            mbar_arrive(bar_kv_empty((cv - 1) % kSt));
            if (cv > 1) mbar_arrive(bar_kv_empty((cv - 2) % kSt));
          }
          if (ok && j + 1 == w.nmax) {                   // every S of the item is done: its Q tiles too
            if (w.nkv[0] > 0) mbar_arrive(bar_q_empty(0));
            if (w.nkv[1] > 0) mbar_arrive(bar_q_empty(1));
          }
          if (ok && L == 1) hand(1, np1);
          else if (ok) hand(0, np0);
        }
      }
      c0 += 2 * w.nmax;
      ns0 += w.nkv[0];
      ns1 += w.nkv[1];
    }
    __syncwarp();
  } else if (warp == 11) {
    // ------------------------------------------------------------ scheduler
    setmaxnreg_dec<C::kRegsOther>();
    Finder finder(p, two_heads ? kBM : 2 * kBM, lane);
    const int inner = two_heads ? p.Hq / 2 : p.Hq;
    bool more = true;
    for (int n = 0; more; ++n) {
      const long long at = static_cast<long long>(n) * gridDim.x + ((n & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      const long long r = at / inner;
      Item it{0, 0, -1, static_cast<int>(at - r * inner)};
      more = r < 0x7FFFFFFF && finder.find(static_cast<int>(r), it);
      if (!more) it.tile = -1;
      bool ok = true;
      if (n >= kItems) ok = wait(bar_item_empty(n % kItems), ((n / kItems) & 1) ^ 1, abort_flag, p.timeout_ns);
      if (!__all_sync(0xffffffffu, ok)) break;
      if (lane == 0) {
        volatile int* const dst = items + 4 * (n % kItems);
        dst[0] = it.start;
        dst[1] = it.len;
        dst[2] = it.tile;
        dst[3] = it.head;
        mbar_arrive(bar_item_full(n % kItems));
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ softmax groups
    setmaxnreg_inc<C::kRegsSoftmax>();
    const int g = warp >> 2;
    const int quarter = warp & 3;                        // TMEM lane quarter this warp may access
    const int row = quarter * 32 + lane;                 // query row within the tile
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t t_s = tbase + lane_off + C::col_s(g);
    const uint32_t t_o = tbase + lane_off + C::col_o(g);
    const float sl2 = p.scale_log2;
    const uint32_t stage = s_out + warp * 4096;
    uint32_t ns = 0, no = 0;                             // parities: S, O final
    // The group's next item with a tile for it, from n on: its key tiles and the
    // keys this row sees (causal), or that there are. -1: no more.
    int n = 0, n_kv, seen;
    auto next = [&]() {
      for (;; ++n) {
        Work w;
        const bool have = take(n, w);
        n_kv = -1;
        if (!__all_sync(0xffffffffu, have)) return;
        n_kv = g ? w.nkv[1] : w.nkv[0];
        seen = p.causal ? min(w.len, (g ? w.qt[1] : w.qt[0]) * kBM + row + 1) : w.len;
        if (n_kv > 0) return;
        if (lane == 0) release(n);
      }
    };
    next();
    while (n_kv > 0) {
      float m = -INFINITY;                               // running max, log2 units of scale*s
      float l = 0.f;                                     // running sum relative to m
      bool ok = true;
      for (int j = 0; j < n_kv; ++j) {
        ok = wait(bar_s_full(g), ns, abort_flag, p.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ns ^= 1;
        tc_fence_after();
        uint32_t sr[4][32];
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) tmem_ld_32x32b_x32(t_s + q4 * 32, sr[q4]);
        tmem_wait_ld();
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) reg_fence_x32(sr[q4]);
        float s[128];
#pragma unroll
        for (int x = 0; x < 128; ++x) s[x] = __uint_as_float(sr[x >> 5][x & 31]);
        const int lim = seen - j * kBN;
        if (lim < kBN) {
#pragma unroll
          for (int x = 0; x < 128; ++x) s[x] = (x < lim) ? s[x] : -INFINITY;
        }
        float mk[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float* v = s + 32 * k;
          float a = fmax3(v[0], v[1], v[2]);
#pragma unroll
          for (int e = 3; e < 31; e += 2) a = fmax3(a, v[e], v[e + 1]);
          mk[k] = fmaxf(a, v[31]);
        }
        const float mx = fmax3(mk[0], mk[1], fmaxf(mk[2], mk[3])) * sl2;
        const bool grow = mx > m + 8.0f;                 // also true on the first tile (m = -inf)
        const float m_new = grow ? mx : m;
        const float alpha = grow ? ex2_approx(m - m_new) : 1.0f;
        m = m_new;
        const float neg_m = (m == -INFINITY) ? 0.f : -m;   // a row behind the sequence's end may hold NaN only
        float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
        for (int h2 = 0; h2 < 2; ++h2) {
          uint32_t pr[32];
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            float x0, x1;
            fma2_bc(x0, x1, s[h2 * 64 + 2 * x], s[h2 * 64 + 2 * x + 1], sl2, neg_m);
            const float p0 = ex2_approx(x0);
            const float p1 = ex2_approx(x1);
            add2_acc(sum0, sum1, p0, p1);
            // P in bf16, as in fa_fwd.cu: the product wants it in V's type, and each term is within 2^-8 of
            // itself, as O is. Two bf16 terms would double the P V products, half of all. l sums P unrounded.
            pr[x] = pack_bf16x2(p0, p1);
          }
          tmem_st_32x32b_x32(t_s + h2 * 32, pr);
        }
        l = l * alpha + (sum0 + sum1);
        // O <- alpha O; the P V before it is done: it was issued before the S just waited for
        if (j > 0 && __any_sync(0xffffffffu, grow)) {
#pragma unroll
          for (int x0 = 0; x0 < D; x0 += 32) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(t_o + x0, o);
            tmem_wait_ld();
            reg_fence_x32(o);
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
            tmem_st_32x32b_x32(t_o + x0, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar_p_ready(g));
      }
      // ---------------------------------------------------------- epilogue
      // what it needs before O is final
      const float inv_l = l > 0.f ? 1.0f / l : 0.f;
      volatile int* const it = items + 4 * (n % kItems);   // once more: the loop above holds no register for it
      const int head = two_heads ? 2 * it[3] + g : it[3];
      const int first = (two_heads ? it[2] : 2 * it[2] + g) * kBM + quarter * 32;   // this warp's rows in the sequence
      const int valid = min(32, it[1] - first);            // of them inside it, may be <= 0
      const int at = it[0] + first;
      __syncwarp();
      if (lane == 0) release(n);
      if (ok && lane < valid)                              // (a NaN among the logits stays one)
        p.lse[static_cast<long long>(head) * p.T + at + lane] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      ++n;
      next();                                              // while the last P V runs
      if (ok) ok = wait(bar_o_final(g), no, abort_flag, p.timeout_ns);
      if (!__all_sync(0xffffffffu, ok)) break;
      no ^= 1;
      tc_fence_after();
#pragma unroll
      for (int x0 = 0; x0 < D; x0 += 64) {
        // (the second half is read and packed while the first one leaves)
        uint32_t o[2][32], r[32];
#pragma unroll
        for (int x = 0; x < 2; ++x) tmem_ld_32x32b_x32(t_o + x0 + 32 * x, o[x]);
        tmem_wait_ld();
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          reg_fence_x32(o[x]);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            r[16 * x + e] = pack_bf16x2(__uint_as_float(o[x][2 * e]) * inv_l, __uint_as_float(o[x][2 * e + 1]) * inv_l);
        }
        if (lane == 0) tma_store_wait_read0();           // the warp's last store has left its buffer
        __syncwarp();
#pragma unroll
        for (int u = 0; u < 8; ++u)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" :: "r"(swz128(stage, lane, u)), "r"(r[4 * u]), "r"(r[4 * u + 1]),
                       "r"(r[4 * u + 2]), "r"(r[4 * u + 3]) : "memory");
        if (valid == 32) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&map_o, stage, x0, at, head);
            tma_store_commit();
          }
        } else {
          // the sequence ends among the warp's rows: the rows behind are another's
          __syncwarp();
          for (int i = lane; i < valid * 8; i += 32) {
            const int rr = i >> 3, u = i & 7;
            if (x0 + 8 * u < p.head_dim) {
              uint4 y;
              asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(y.x), "=r"(y.y), "=r"(y.z), "=r"(y.w)
                           : "r"(swz128(stage, rr, u)) : "memory");
              *reinterpret_cast<uint4*>(p.o + head * p.o_sh + (at + rr) * p.o_st + x0 + 8 * u) = y;
            }
          }
        }
      }
    }
    if (lane == 0) tma_store_wait_all0();
    __syncwarp();
  }

  // ---------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    if (threadIdx.x == 0) atomicOr(p.status, kDevTimeout);
    abort_grace_period();
  }
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tbase, 512);
  if (threadIdx.x == 0) clock_record(p.clock_acc, clock_start);
}

template <int D>
cudaError_t launch(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mo,
                   const FwdParams& p, int grid,
                   cudaStream_t stream) {
  using C = Cfg<D>;
  static PerDeviceOnce attr;
  const cudaError_t e = attr.run(
      [] { return cudaFuncSetAttribute(fwd_packed_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem); });
  if (e != cudaSuccess) return e;
  fwd_packed_kernel<D><<<grid, C::kThreads, C::kSmem, stream>>>(mq, mk, mv, mo, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fwd_packed(int d, const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                              const CUtensorMap& mo, FwdParams p, int num_sms, cudaStream_t stream) {
  const bool two_heads = (p.Hq / p.Hkv) % 2 == 0;
  p.num_pairs = two_heads ? 1 : 0;
  const int unit = two_heads ? kBM : 2 * kBM;
  // at most (n + unit - 1) / unit items per sequence and head (pair)
  const long long most = (p.T + static_cast<long long>(unit - 1) * p.S) / unit * (two_heads ? p.Hq / 2 : p.Hq);
  const int grid = static_cast<int>(most < num_sms ? most : num_sms);
  return d <= 64 ? launch<64>(mq, mk, mv, mo, p, grid, stream) : launch<128>(mq, mk, mv, mo, p, grid, stream);
}

}  // namespace fa
