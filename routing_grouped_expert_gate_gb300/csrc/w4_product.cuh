// The product kernel of the experts with 4-bit weights (w4.cu says how the
// codes are laid out), instantiated for one group size per file.
#pragma once
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "glu_act.cuh"
#include "internal.h"
#include "tc_ptx.cuh"
#include "w4.h"

namespace moe {

namespace {

// d = a b
__device__ __forceinline__ void mma_new(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// c += a b
__device__ __forceinline__ void mma_add(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Bits 4i..4i+3 of both halves of w as a pair of bf16 u - 8, exactly: 128 + u
// by bits, less 136. (x & mask) | magic is one instruction when only one of the
// two constants is an immediate, so the mask comes in a register. Taking 136
// sum_k x[k] off a group's sum of (128 + u) x instead leaves the rounding of 136
// |x| in it, whatever the weight, and is no faster: one token through 2 of 8
// experts of 4096 x 14336 50.8 us (50.0 so), 12 tokens through 8 of 64 of 2048 x
// 1408 66.4 us (64.7).
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int i, uint32_t mask) {
  uint32_t t;
  asm("lop3.b32 %0, %1, %2, 0x43004300, 0xEA;" : "=r"(t) : "r"(w >> (4 * i)), "r"(mask));
  const uint32_t k136 = 0x43084308u;
  const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&t),
                                   *reinterpret_cast<const __nv_bfloat162*>(&k136));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// the scales of one row's slab as they lie: four, two or one bf16
template <int GS> struct Scales;
template <> struct Scales<32> {
  uint2 v;
  __device__ __forceinline__ void load(const bf16* p) { v = __ldg(reinterpret_cast<const uint2*>(p)); }
  __device__ __forceinline__ void store(char* p) const { *reinterpret_cast<uint2*>(p) = v; }
  __device__ __forceinline__ void take(const char* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ float get(int g) const {
    const uint32_t w = g < 2 ? v.x : v.y;
    return __uint_as_float((g & 1) ? (w & 0xffff0000u) : (w << 16));
  }
};
template <> struct Scales<64> {
  uint32_t v;
  __device__ __forceinline__ void load(const bf16* p) { v = __ldg(reinterpret_cast<const uint32_t*>(p)); }
  __device__ __forceinline__ void store(char* p) const { *reinterpret_cast<uint32_t*>(p) = v; }
  __device__ __forceinline__ void take(const char* p) { v = *reinterpret_cast<const uint32_t*>(p); }
  __device__ __forceinline__ float get(int g) const {
    return __uint_as_float((g & 1) ? (v & 0xffff0000u) : (v << 16));
  }
};
template <> struct Scales<128> {
  unsigned short v;
  __device__ __forceinline__ void load(const bf16* p) {
    v = __ldg(reinterpret_cast<const unsigned short*>(p));
  }
  __device__ __forceinline__ void store(char* p) const { *reinterpret_cast<unsigned short*>(p) = v; }
  __device__ __forceinline__ void take(const char* p) {
    v = *reinterpret_cast<const unsigned short*>(p);
  }
  __device__ __forceinline__ float get(int) const { return __uint_as_float((uint32_t)v << 16); }
};

__device__ __forceinline__ uint32_t word_of(uint4 v, int j) {
  return j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
}

// ---- the sums' exchange between the blocks of a cluster
__device__ __forceinline__ void arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(tc::su32(b)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool wait_cluster(uint64_t* b, uint32_t parity, const W4Args& a) {
  const uint64_t t0 = global_timer_ns();
  while (!try_wait_cluster(b, parity)) {
    if (global_timer_ns() - t0 > a.timeout_ns) {
      record_error(a.status, MOE_ERR_TIMEOUT, 40);
      return false;
    }
  }
  return true;
}
// Row of eight that the lanes of a fragment's row (or column) g hold. A quarter
// warp's 16-byte loads cover two of them, four pieces each; in the 128-byte
// swizzle a row's pieces 0..3 lie in the half that bit 2 of the row says, so
// the two rows differ in that bit and no bank is asked twice.
__device__ __forceinline__ int row_of(int g) { return (g >> 1) | ((g & 1) << 2); }
__device__ __forceinline__ int place_of(int row) { return ((row & 3) << 1) | (row >> 2); }

constexpr int kMaxStages = 8;

// How the blocks share the tasks.
// In turn: whole tasks one after another, or the slabs of each by a cluster of
// blocks whose sums meet in its shared memory.
// Late (one token tile, clusters): and a task's outputs are finished one task
// late, with one more warp that tells the other blocks of a block's sums (one
// token, 2 of 8 wide experts: 50 us, 85 with whole tasks in turn; in blocks of
// their own it only costs: 12 tokens on 64 experts 66 us, 65 in turn).
// Dealt (more token tiles): the steps of all tasks, in a row, in even parts by
// their time, so that a task may begin in one block and end in another; their
// sums meet in global memory. That fills all blocks, whatever the number of
// tasks, for about 4 us in each launch (64 tokens, 2 of 8 wide experts, 128 tasks
// in the second product: 218 us, 235 in turn).
enum class Sharing { kInTurn, kLate, kDealt };

// Sixteen A tiles a task. One token tile: two of them and every other slab for
// a warp, so that what a warp does once per slab (activations, their sums, the
// wait) serves two tiles. More token tiles: one A tile and all slabs, for the
// accumulators' sake.
template <int NTMAX, Sharing HOW> struct Shape {
  static constexpr bool kLate = HOW == Sharing::kLate, kDealt = HOW == Sharing::kDealt;
  // that multiply, and three that load
  static constexpr int kWarps = 16;
  static constexpr int kWays = NTMAX == 1 ? 2 : 1, kMt = kWays;
  static constexpr int kThreads = (kWarps + 3 + (kLate ? 1 : 0)) * 32;
  static constexpr int kTiles = kWarps / kWays * kMt;
  static constexpr int kBoxRows = kTiles * 8;        // weight rows of a box of codes
  static constexpr int kBoxBytes = kBoxRows * 128;   // two slabs (128 bytes) per row
  static constexpr int kCodeBytes = 2 * kBoxBytes;   // codes of a stage
  static constexpr int kPart = kTiles * NTMAX * 128;  // floats of a task's sums
  static_assert(kTiles == kW4Tiles, "");
};

// Time of a step by its token tiles, in some unit (64 tokens, 2 of 8 wide
// experts: 219 us with this 2, 222 with 3, 230 with 5; 221 with 1).
__device__ __forceinline__ uint32_t step_weight(int rows) { return 2 + (rows + 7) / 8; }
// the division of small numbers takes a fraction of the other's time
__device__ __forceinline__ uint64_t quotient(uint64_t a, uint64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}

struct W4Shared {
  int pre[kMaxE + 1];        // units before each expert
  uint32_t prew[kMaxE + 1];  // and their steps' weights
  int row0[kMaxE], cnt[kMaxE];
  int warp_tot[kMaxE / 32];
  uint32_t warp_totw[kMaxE / 32];
  int abort;
  uint64_t full[kMaxStages], empty[kMaxStages];
  // A cluster's sums of a task are all written, all read. Late: the block's sums
  // of a task are written (a barrier for every other task), and so are those of
  // all the cluster's blocks.
  uint64_t ready, free, done[2], all[2];
};

// Where a block is in its tasks: the expert, its unit and the first tile.
struct W4At {
  int g, unit, tile0;
};

template <bool FIRST, int NTMAX, int P, int GS, Sharing HOW>
struct W4 {
  using S = Shape<NTMAX, HOW>;
  using Out = typename std::conditional<P == 3, float, bf16>::type;
  static constexpr int kMt = S::kMt;
  // activations of a stage: per plane a box of four pieces of 64 k (128 bytes,
  // 128-byte swizzle) of all a unit's rows (of eight for a unit with no more)
  static constexpr int kBoxX = NTMAX * 1024, kPlaneX = 4 * kBoxX, kX = P * kPlaneX;
  // and its rows' scales: two slabs' next to each other
  static constexpr int kRec = 2 * (kSlab / GS) * 2, kScaleRows = 2 * S::kBoxRows;
  static constexpr int kStage = S::kCodeBytes + kX + 4096;
  static_assert(kRec * kScaleRows <= 4096, "");

  const W4Args& a;
  W4Shared& sh;
  char* ring;
  float* red;  // the block's sums (task() says of what)
  int kbeg, kend;  // the slabs of a task that are this block's
  int nc;          // from a task to the next: clusters, or 1
  uint32_t rank;
  int per;         // tasks of a unit
  // the first task and slab, and how many steps from there
  using Count = typename std::conditional<S::kDealt, int64_t, int>::type;
  int t0, s0;
  Count steps;

  __device__ __forceinline__ W4At locate(int task) const {
    const int u = task / per;
    int lo = 0, hi = a.G - 1;  // the expert of this unit: the last with pre[g] <= u
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sh.pre[mid] <= u) lo = mid;
      else hi = mid - 1;
    }
    return W4At{lo, u - sh.pre[lo], (task - u * per) * S::kTiles};
  }
  // the task nc behind it (short of the end: `task` exists)
  __device__ __forceinline__ void advance(W4At& p, int task) const {
    p.tile0 += nc * S::kTiles;
    if (p.tile0 < a.n_tiles) return;
    p = locate(task);
  }

  // Dealt out: block b begins where b / nblk of the weight of all steps, `total`,
  // lies before.
  int pairs;         // steps of a task
  uint64_t in_unit;  // steps of a unit
  uint64_t total;
  uint32_t nblk;     // blocks with work
  __device__ __forceinline__ int64_t first_step(uint32_t b) const {
    if (b >= nblk) return sh.pre[a.G] * (int64_t)in_unit;
    const uint64_t x = quotient(total * b, nblk);
    int lo = 0, hi = a.G - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (sh.prew[mid] * in_unit <= x) lo = mid;
      else hi = mid - 1;
    }
    const uint64_t full = step_weight(8 * NTMAX) * in_unit;
    const uint64_t y = x - sh.prew[lo] * in_unit;
    const W4At p{lo, min((int)quotient(y, full), sh.pre[lo + 1] - sh.pre[lo] - 1), 0};
    return (sh.pre[lo] + p.unit) * (int64_t)in_unit +
           (int64_t)quotient(y - p.unit * full, step_weight(rows_of(p)));
  }
  // The block whose step s of task p is: the last b with first_step(b) <= s,
  // which is to say total b / nblk < the weight up to the end of that step.
  __device__ __forceinline__ uint32_t block_of(const W4At& p, int s) const {
    const uint64_t w = (sh.prew[p.g] + p.unit * step_weight(8 * NTMAX)) * in_unit +
                       ((uint64_t)(p.tile0 / S::kTiles) * pairs + s + 1) * step_weight(rows_of(p));
    return (uint32_t)quotient(w * nblk + total - 1, total) - 1;
  }
  __device__ void deal() {
    kbeg = 0;
    kend = a.S;
    nc = 1;
    pairs = (a.S + 1) / 2;
    in_unit = (uint64_t)per * pairs;
    total = sh.prew[a.G] * in_unit;
    // As many blocks as leave each one step at least, whatever the steps' weights
    // (total / nblk is at least a full unit's step). The count of those that share a
    // task relies on it: no block between the first and the last may be without a step.
    nblk = (uint32_t)min((uint64_t)gridDim.x, quotient(total, 2 * step_weight(8 * NTMAX)) + 1);
    const bool any = total > 0 && blockIdx.x < nblk;
    const int64_t at = any ? first_step(blockIdx.x) : 0;
    steps = any ? first_step(blockIdx.x + 1) - at : 0;
    t0 = (int)quotient(at, pairs);
    s0 = 2 * (int)(at - (int64_t)t0 * pairs);
  }
  __device__ __forceinline__ int rows_of(const W4At& p) const {
    return min(sh.cnt[p.g] - p.unit * 8 * NTMAX, 8 * NTMAX);
  }

  // ---------------------------------------------------------- the loading warp
  __device__ __forceinline__ void load_codes(const CUtensorMap* codes, const W4At& p, int s, int st) {
    const int y = FIRST ? p.g * 2 * a.F + p.tile0 * 8 : p.g * a.d + p.tile0 * 16;
    char* to = ring + st * kStage;
    tc::mbar_expect_tx(&sh.full[st], S::kCodeBytes + P * 4 * (rows_of(p) <= 8 ? 1024 : kBoxX));
    tc::tma_load_2d(to, codes, &sh.full[st], s * (kSlab / 4), y);
    tc::tma_load_2d(to + S::kBoxBytes, codes, &sh.full[st], s * (kSlab / 4),
                    y + (FIRST ? a.F : S::kBoxRows));
  }
  __device__ __forceinline__ void load_x(const CUtensorMap* xmap, const CUtensorMap* xmap8,
                                         const W4At& p, int s, int st) {
    const int r = sh.row0[p.g] + p.unit * 8 * NTMAX;
    const CUtensorMap* map = rows_of(p) <= 8 ? xmap8 : xmap;
    char* to = ring + st * kStage + S::kCodeBytes;
#pragma unroll
    for (int q = 0; q < P; ++q)
      tc::tma_load_3d_s(tc::su32(to + q * kPlaneX), map, tc::su32(&sh.full[st]), 0,
                        q * a.n_rows + r, s * (kSlab / 64));
  }
  // The place in the block's steps: slab s of task t.
  struct Walk {
    Count left;  // steps, this one among them
    Count n;     // steps before it
    int t, s;
    W4At p;
  };
  __device__ __forceinline__ Walk walk() const {
    return Walk{steps, 0, t0, s0, steps > 0 ? locate(t0) : W4At{0, 0, 0}};
  }
  // `by` steps on, up to the next task; whether it begins another one
  __device__ __forceinline__ bool step(Walk& w, int by = 1) const {
    w.n += by;
    w.left -= by;
    w.s += 2 * by;
    if (w.s < kend) return false;
    w.s = kbeg;
    w.t += nc;
    if (w.left > 0) advance(w.p, w.t);
    return true;
  }

  // one thread: codes and activations
  __device__ void load_tiles(const CUtensorMap* codes, const CUtensorMap* xmap,
                             const CUtensorMap* xmap8) {
    Walk w = walk();
    // codes of the first stages; the activations may still be on their way
    Walk first = w;
    for (; w.n < a.stages && w.left > 0; step(w)) load_codes(codes, w.p, w.s, w.n);
    pdl_wait();
    asm volatile("fence.proxy.async;" ::: "memory");
    for (; first.n < w.n; step(first)) load_x(xmap, xmap8, first.p, first.s, first.n);
    int st = 0, ph = 0;
    for (; w.left > 0; step(w)) {
      if (!tc::mbar_wait(&sh.empty[st], ph, sh.abort, a, 43)) break;
      load_codes(codes, w.p, w.s, st);
      load_x(xmap, xmap8, w.p, w.s, st);
      if (++st == a.stages) {
        st = 0;
        ph ^= 1;
      }
    }
    // its copies land before the block ends, also where a wait gave up
    const uint64_t from = global_timer_ns();
    for (Count i = max((Count)0, w.n - a.stages); i < w.n; ++i)
      while (!tc::mbar_try_wait(&sh.full[i % a.stages], (i / a.stages) & 1) &&
             global_timer_ns() - from < a.timeout_ns) {
      }
  }

  // Two warps, a stage each in turn: scales. They are too few per row and stage
  // for TMA's 16-byte pieces; the lanes, two to a row for the stage's two slabs,
  // have a stage's in registers before it has room. (Asking a task's scales into
  // L2 beforehand, by bulk or plain prefetches, measured slower: 74 us against
  // 67 for 12 tokens on 64 experts.)
  __device__ void load_scales(int turn) {
    constexpr int kMine = kScaleRows / 16;
    const bf16* from[kMine];
    Scales<GS> next[kMine];
    const int slab = lane & 1;
    Walk w = walk();
    auto rows = [&]() {
      const int64_t N = FIRST ? 2 * a.F : a.d;
      const int last = (FIRST ? a.F : a.d) - 1;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int r = i * 16 + (lane >> 1);
        // rows past the end take the last one's scales; their results are dropped
        const int row = FIRST ? min(w.p.tile0 * 8 + r % S::kBoxRows, last) + (r / S::kBoxRows) * a.F
                              : min(w.p.tile0 * 16 + r, last);
        from[i] = a.s + ((w.p.g * N + row) * a.S + slab) * (kSlab / GS);
      }
    };
    auto fetch = [&]() {
      if (w.s + slab < kend) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) next[i].load(from[i] + w.s * (kSlab / GS));
      }
    };
    if (turn == 1 && w.left > 0) step(w);
    if (w.left <= 0) return;
    rows();
    fetch();
    int st = turn, ph = 1;  // the first round finds every stage free
    while (true) {
      if (!tc::mbar_wait(&sh.empty[st], ph, sh.abort, a, 44)) return;
      char* to = ring + st * kStage + S::kCodeBytes + kX + lane * (kRec / 2);
#pragma unroll
      for (int i = 0; i < kMine; ++i) next[i].store(to + i * 16 * kRec);
      tc::mbar_arrive(&sh.full[st]);
      bool another = step(w);
      if (w.left > 0 && step(w)) another = true;
      if (w.left <= 0) return;
      if (another) rows();
      fetch();
      if ((st += 2) >= a.stages) {
        st -= a.stages;
        ph ^= 1;
      }
    }
  }

  // ---------------------------------------------------------- the multiplying warps
  int lane, warp, tig, st, ph;
  int row8;  // this lane's row of eight, of weights and of tokens
  int flip;  // from a 16-byte piece to the one four behind it, in swizzled places
  uint32_t mask;
  bool ok;

  // Slab s from the codes of this lane's rows at q, their scales at r and the
  // activations at x; CHECKED where it may reach past K (the padding's scales
  // may hold anything).
  template <int NT, bool CHECKED>
  __device__ __forceinline__ void slab(int s, const char* q, const char* r, const char* x,
                                       float (&acc)[kMt][NT][4]) {
    uint4 w[kMt][2];
    Scales<GS> c[kMt][2];
#pragma unroll
    for (int m = 0; m < kMt; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        w[m][h] = *reinterpret_cast<const uint4*>(
            q + (FIRST ? m * 1024 + h * S::kBoxBytes : (2 * m + h) * 1024));
        c[m][h].take(r + (FIRST ? m * 8 + h * S::kBoxRows : (2 * m + h) * 8) * kRec);
      }
#pragma unroll
    for (int g = 0; g < kSlab / GS; ++g) {
      if (CHECKED && s * kSlab + g * GS >= a.K) return;
      constexpr int J = GS / 32;  // 32-k blocks of a group
      // k 32 j + 8 tig of the slab: piece 4 (j & 1) + tig of a row in the slab's
      // box j / 2, at its place xor the row mod 8
      constexpr int kBox = NT == 1 ? 1024 : kBoxX;
      float part[kMt][NT][4];
#pragma unroll
      for (int jj = 0; jj < J; ++jj) {
        const int j = g * J + jj;
        const char* xj = x + (j >> 1) * kBox + ((j & 1) ? flip : 0);
        uint32_t a0[kMt][4], a1[kMt][4];
#pragma unroll
        for (int m = 0; m < kMt; ++m)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              a0[m][2 * i + h] = code_pair(word_of(w[m][h], j), i, mask);
              a1[m][2 * i + h] = code_pair(word_of(w[m][h], j), 2 + i, mask);
            }
#pragma unroll
        for (int p = P - 1; p >= 0; --p) {  // the smallest plane first
          uint4 b[NT];
#pragma unroll
          for (int n = 0; n < NT; ++n)
            b[n] = *reinterpret_cast<const uint4*>(xj + p * kPlaneX + n * 1024);
          const bool begins = jj == 0 && p == P - 1;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < kMt; ++m) {
              if (begins) mma_new(part[m][n], a0[m], b[n].x, b[n].y);
              else mma_add(part[m][n], a0[m], b[n].x, b[n].y);
            }
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < kMt; ++m) mma_add(part[m][n], a1[m], b[n].z, b[n].w);
        }
      }
#pragma unroll
      for (int m = 0; m < kMt; ++m) {
        const float s0 = c[m][0].get(g), s1 = c[m][1].get(g);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          acc[m][n][0] = fmaf(part[m][n][0], s0, acc[m][n][0]);
          acc[m][n][1] = fmaf(part[m][n][1], s0, acc[m][n][1]);
          acc[m][n][2] = fmaf(part[m][n][2], s1, acc[m][n][2]);
          acc[m][n][3] = fmaf(part[m][n][3], s1, acc[m][n][3]);
        }
      }
    }
  }

  __device__ __forceinline__ void put(int t, int row, int64_t r, float lo, float hi) const {
    if (FIRST) {  // h in planes: the second product reads it as bf16
      const float h = glu_fwd(lo, hi, a.act);
      bf16* o = static_cast<bf16*>(a.out) + r * a.ldh + t * 8 + row;
      if (P == 1) {
        *o = from_f32<bf16>(h);
      } else {
        float p0, p1, p2;
        planes3(h, p0, p1, p2);
        const int64_t plane = (int64_t)a.n_rows * a.ldh;
        o[0] = from_f32<bf16>(p0);
        o[plane] = from_f32<bf16>(p1);
        o[2 * plane] = from_f32<bf16>(p2);
      }
    } else {
      Out* o = static_cast<Out*>(a.out) + r * a.d + t * 16 + row;
      *o = from_f32<Out>(lo);
      if (t * 16 + 8 + row < a.d) o[8] = from_f32<Out>(hi);
    }
  }

  // Late: outputs of task n (the last_ ones) from the sums of both
  // ways and of all the cluster's blocks, in the order of their ranks; each block takes
  // its share of them.
  int last_row0, last_rows, last_tile0;
  __device__ __forceinline__ void finish(int n) {
    uint64_t* bar = &sh.all[n & 1];
    if (ok) ok = wait_cluster(bar, (n >> 1) & 1, a);
    const uint32_t base = tc::su32(red + (n & 1) * 2 * S::kTiles * 128);
    const int count = S::kTiles * 8 * last_rows;
    for (int i = rank * (S::kWarps * 32) + threadIdx.x; i < count; i += a.split * (S::kWarps * 32)) {
      const int row = i & 7, tt = (i >> 3) / last_rows, tok = (i >> 3) - tt * last_rows;
      if (last_tile0 + tt >= a.n_tiles) continue;
      const int col = place_of(tok);
      const int at = (tt * 4 + (col & 1)) * 32 + place_of(row) * 4 + (col >> 1);
      constexpr int kWay = S::kTiles * 128;  // from the first way's sums to the second's
      float lo = 0.f, hi = 0.f;
      for (int p = 0; p < a.split; ++p) {
        const uint32_t there = tc::mapa_shared(base + at * 4, p);
        lo += __uint_as_float(tc::ld_shared_cluster_u32(there)) +
              __uint_as_float(tc::ld_shared_cluster_u32(there + kWay * 4));
        hi += __uint_as_float(tc::ld_shared_cluster_u32(there + 256)) +
              __uint_as_float(tc::ld_shared_cluster_u32(there + 256 + kWay * 4));
      }
      put(last_tile0 + tt, row, last_row0 + tok, lo, hi);
    }
    __syncwarp();
  }
  // Late: a warp of its own tells the cluster's blocks when this
  // block's sums are in place (the release to the cluster takes a while).
  __device__ void announce() {
    for (int n = 0, left = (int)steps; left > 0; ++n, left -= (kend - kbeg + 1) / 2) {
      if (!tc::mbar_wait(&sh.done[n & 1], (n >> 1) & 1, sh.abort, a, 46)) return;
      if (lane < a.split) arrive_remote(tc::mapa_shared(tc::su32(&sh.all[n & 1]), lane));
      __syncwarp();
    }
  }

  // The task at p, the block's n_task-th: its slabs [from, to), or all that are
  // the block's. next() may move on to the task after it.
  template <int NT, typename Next>
  __device__ __forceinline__ void task(const W4At p, int rows, int from, int to, int n_task, Next next) {
    const int row0 = sh.row0[p.g] + p.unit * 8 * NTMAX, tile0 = p.tile0;
    if (!S::kDealt) {
      from = kbeg;
      to = kend;
    }
    float acc[kMt][NT][4];
#pragma unroll
    for (int m = 0; m < kMt; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
    const int place = row8 * 128 + ((tig ^ row8) * 16);
    const int tile = warp % (S::kWarps / S::kWays) * kMt, way = warp / (S::kWarps / S::kWays);
    // A rows: eight of the gate's box and eight of the up box, or sixteen in turn
    const int codes = tile * (FIRST ? 1024 : 2048) + place;
    const int rec = S::kCodeBytes + kX + (tile * (FIRST ? 8 : 16) + row8) * kRec;
    constexpr int kSlabX = 2 * (NT == 1 ? 1024 : kBoxX);  // from a slab's activations to the next
    for (int s = from; s < to; s += 2) {
      if (ok) ok = tc::mbar_wait(&sh.full[st], ph, sh.abort, a, FIRST ? 41 : 42);
      const char* at = ring + st * kStage;
      const bool whole = (s + 2) * kSlab <= a.K;
#pragma unroll
      for (int i = 0; i < 2 / S::kWays; ++i) {
        const int h = S::kWays == 2 ? way : i;
        if (s + h < to) {
          const char *q = at + codes + h * flip, *r = at + rec + h * (kRec / 2);
          const char* x = at + S::kCodeBytes + place + h * kSlabX;
          if (whole) slab<NT, false>(s + h, q, r, x, acc);
          else slab<NT, true>(s + h, q, r, x, acc);
        }
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sh.empty[st]);
      if (++st == a.stages) {
        st = 0;
        ph ^= 1;
      }
    }
    next();
    if (S::kWays == 2 && !S::kLate) {
      // the second slabs' sums join the first's; two buffers, so that the pair
      // of warps meets once a task
      float* to = red + ((n_task & 1) * S::kTiles + tile) * 128 + lane;
      if (way == 1) {
#pragma unroll
        for (int i = 0; i < kMt * 4; ++i) to[i * 32] = acc[i >> 2][0][i & 3];
      }
      asm volatile("bar.sync %0, 64;" ::"r"(tile / kMt + 1) : "memory");
      if (way == 1) return;
#pragma unroll
      for (int i = 0; i < kMt * 4; ++i) acc[i >> 2][0][i & 3] += to[i * 32];
    } else if (S::kLate) {
      // The sums of both ways and all blocks meet in shared memory, one task
      // late: what the task before left there is finished first, so that nobody
      // waits for the slowest warp or the other blocks. That every block's sums
      // of it were in place says that all had read the task's before it, whose
      // buffer is written now.
      if (n_task > 0) finish(n_task - 1);
      float* to = red + (((n_task & 1) * 2 + way) * S::kTiles + tile) * 128 + lane;
#pragma unroll
      for (int m = 0; m < kMt; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) to[(m * 4 + i) * 32] = acc[m][0][i];
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&sh.done[n_task & 1]);
      last_row0 = row0;
      last_rows = rows;
      last_tile0 = tile0;
      return;
    }
    if (NTMAX > 1 && !S::kDealt && a.split > 1) {
      // The cluster's blocks hold sums over their own slabs: each adds up its
      // share of the outputs over all of them, in the order of their ranks.
      if (n_task > 0 && ok) ok = wait_cluster(&sh.free, (n_task - 1) & 1, a);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[((tile * NT + n) * 4 + i) * 32 + lane] = acc[0][n][i];
      __syncwarp();
      if (lane < a.split) arrive_remote(tc::mapa_shared(tc::su32(&sh.ready), lane));
      if (ok) ok = wait_cluster(&sh.ready, n_task & 1, a);
      const uint32_t base = tc::su32(red);
      for (int i = rank * (S::kWarps * 32) + threadIdx.x; i < S::kTiles * NT * 64;
           i += a.split * (S::kWarps * 32)) {
        const int row = i & 7, tok = (i >> 3) % (8 * NT), tt = (i >> 3) / (8 * NT);
        if (tok >= rows || tile0 + tt >= a.n_tiles) continue;
        const int col = place_of(tok & 7);
        const int at = ((tt * NT + (tok >> 3)) * 4 + (col & 1)) * 32 + place_of(row) * 4 + (col >> 1);
        float lo = 0.f, hi = 0.f;
        for (int p = 0; p < a.split; ++p) {
          const uint32_t there = tc::mapa_shared(base + at * 4, p);
          lo += __uint_as_float(tc::ld_shared_cluster_u32(there));
          hi += __uint_as_float(tc::ld_shared_cluster_u32(there + 256));
        }
        put(tile0 + tt, row, row0 + tok, lo, hi);
      }
      __syncwarp();
      if (lane < a.split) arrive_remote(tc::mapa_shared(tc::su32(&sh.free), lane));
      return;
    }
    if (S::kDealt && (from > 0 || to < a.S)) {
      // Several blocks have steps of this task, block_of its first to its last.
      // Each leaves its sums in its slot (one for a task begun before it, one
      // for a task that goes on behind it); whoever comes last adds them all up,
      // in the blocks' order. Nobody waits, and each warp does this by itself.
      const uint32_t lo = block_of(p, 0), hi = block_of(p, pairs - 1);
      float* slot = a.part + ((int64_t)blockIdx.x * 2 + (from == 0)) * S::kPart;
      const int mine = tile * NTMAX * 128 + lane;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) __stcg(slot + mine + (n * 4 + i) * 32, acc[0][n][i]);
      // Lane 0's fences stand between the warp's barriers and its ticket, so that
      // the ticket releases what all lanes stored and a ticket that is the last
      // one acquires it for all lanes.
      __syncwarp();
      uint32_t before = 0;
      if (lane == 0) {
        __threadfence();
        before = atomicAdd(a.came + lo * S::kTiles + tile, 1u);
        __threadfence();
      }
      before = __shfl_sync(0xffffffffu, before, 0);
      __syncwarp();
      if (before != hi - lo) return;
      for (uint32_t b = lo; b <= hi; ++b) {
        const float* q = a.part + ((int64_t)b * 2 + (b == lo)) * S::kPart + mine;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float v = __ldcg(q + (n * 4 + i) * 32);
            acc[0][n][i] = b == lo ? v : acc[0][n][i] + v;
          }
      }
    }
#pragma unroll
    for (int m = 0; m < kMt; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int tok = n * 8 + row_of(2 * tig + e), t = tile0 + tile + m;
          if (tok < rows && t < a.n_tiles)
            put(t, row8, row0 + tok, acc[m][n][e], acc[m][n][2 + e]);
        }
  }
};

// Codes and activations come through one ring of TMA stages (two slabs of 256
// weight rows and of the unit's rows) that one thread keeps ahead of the
// multiplying warps, across tasks, as two warps do with the scales: HBM is busy
// while sums leave.
template <bool FIRST, int NTMAX, int P, int GS, Sharing HOW>
__global__ void __launch_bounds__(Shape<NTMAX, HOW>::kThreads, 1)
    w4_product(const __grid_constant__ CUtensorMap codes, const __grid_constant__ CUtensorMap xmap,
             const __grid_constant__ CUtensorMap xmap8, const W4Args a) {
  using K = W4<FIRST, NTMAX, P, GS, HOW>;
  using S = Shape<NTMAX, HOW>;
  __shared__ W4Shared sh;
  extern __shared__ char dyn_raw[];
  char* dyn = dyn_raw + ((1024u - (tc::su32(dyn_raw) & 1023u)) & 1023u);
  // The kernel before this one (the rows' copy, or the first product) has let
  // it start early, after everything before that was complete: the offsets and
  // the weights may be read at once, the activations after pdl_wait.
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  bool bad = false;
  if (threadIdx.x < kMaxE) {
    const int g = threadIdx.x;
    int lo = 0, n = 0;
    if (g < a.G) {
      lo = a.offsets != nullptr ? a.offsets[g] : 0;
      const int hi = a.offsets != nullptr ? a.offsets[g + 1] : a.n_rows;
      bad = lo < 0 || hi < lo || hi > a.n_rows;
      if (bad) {
        if (blockIdx.x == 0) record_error(a.status, MOE_ERR_DEVICE_INDEX, g);
      } else {
        n = hi - lo;
      }
    }
    int sum = (n + 8 * NTMAX - 1) / (8 * NTMAX);
    uint32_t sumw = 0;
    if (S::kDealt && sum > 0)
      sumw = (sum - 1) * step_weight(8 * NTMAX) + step_weight(n - (sum - 1) * 8 * NTMAX);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
      if (S::kDealt) {
        const uint32_t vw = __shfl_up_sync(0xffffffffu, sumw, o);
        if (lane >= o) sumw += vw;
      }
    }
    if (lane == 31) {
      sh.warp_tot[warp] = sum;
      sh.warp_totw[warp] = sumw;
    }
    sh.pre[g + 1] = sum;
    sh.prew[g + 1] = sumw;
    sh.row0[g] = lo;
    sh.cnt[g] = n;
  } else if (threadIdx.x == kMaxE) {
    sh.pre[0] = 0;
    sh.prew[0] = 0;
    sh.abort = 0;
    for (int i = 0; i < kMaxStages; ++i) {
      tc::mbar_init(&sh.full[i], 1 + 32);  // the copies' start and each lane's scales
      tc::mbar_init(&sh.empty[i], S::kWarps);
    }
    const int blocks = max(a.split, 1);  // of a cluster
    tc::mbar_init(&sh.ready, S::kWarps * blocks);
    tc::mbar_init(&sh.free, S::kWarps * blocks);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sh.done[i], S::kWarps);
      tc::mbar_init(&sh.all[i], blocks);
    }
    tc::fence_barrier_init();
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x < kMaxE && !bad) {
    int add = 0;
    uint32_t addw = 0;
    for (int w = 0; w < warp; ++w) {
      add += sh.warp_tot[w];
      addw += sh.warp_totw[w];
    }
    sh.pre[threadIdx.x + 1] += add;
    sh.prew[threadIdx.x + 1] += addw;
  }
  if (bad && threadIdx.x == 0) {
    // rows that an expert before has are skipped too: no more rows than the call's
    int end = 0;
    for (int g = 0; g < a.G; ++g) {
      if (sh.row0[g] < end) sh.cnt[g] = 0;
      const int n = sh.cnt[g], units = (n + 8 * NTMAX - 1) / (8 * NTMAX);
      if (n > 0) end = sh.row0[g] + n;
      sh.pre[g + 1] = sh.pre[g] + units;
      sh.prew[g + 1] = sh.prew[g];
      if (S::kDealt && n > 0)
        sh.prew[g + 1] += (units - 1) * step_weight(8 * NTMAX) + step_weight(n - (units - 1) * 8 * NTMAX);
    }
  }
  if (a.split > 1) tc::cluster_barrier();  // the barriers of all blocks are set up
  else __syncthreads();

  K k{a, sh};
  k.ring = dyn;
  k.red = reinterpret_cast<float*>(dyn + a.stages * K::kStage);
  k.per = (a.n_tiles + S::kTiles - 1) / S::kTiles;
  k.rank = 0;
  if constexpr (S::kDealt) {
    k.deal();
  } else {
    if (a.split > 1) k.rank = tc::cluster_ctarank();
    // an even number of slabs for each block but the last
    const int pairs = (a.S + 1) / 2;
    k.kbeg = (int)((int64_t)pairs * k.rank / a.split) * 2;
    k.kend = min((int)((int64_t)pairs * (k.rank + 1) / a.split) * 2, a.S);
    k.nc = gridDim.x / a.split;
    k.t0 = blockIdx.x / a.split;
    k.s0 = k.kbeg;
    const int tasks = sh.pre[a.G] * k.per;
    const int own = k.t0 < tasks ? (tasks - 1 - k.t0) / k.nc + 1 : 0;
    k.steps = (typename K::Count)own * ((k.kend - k.kbeg + 1) / 2);
  }
  k.lane = lane;
  if (warp == S::kWarps) {
    if (lane == 0) k.load_tiles(&codes, &xmap, &xmap8);
    __syncwarp();
  } else if (warp == S::kWarps + 1 || warp == S::kWarps + 2) {
    k.load_scales(warp - S::kWarps - 1);
    __syncwarp();
  } else if (S::kLate && warp == S::kWarps + 3) {
    k.announce();
    __syncwarp();
  } else {
    k.warp = warp;
    k.row8 = row_of(lane >> 2);
    k.tig = lane & 3;
    k.mask = a.mask;
    k.flip = (k.row8 & 4) ? -64 : 64;
    k.st = k.ph = 0;
    k.ok = true;
    typename K::Walk w = k.walk();
    // outputs are written after this: the kernel before may still read there
    pdl_wait();
    if (FIRST) pdl_launch_dependents();
    int n = 0;
    auto task = [&](int rows, int from, int to, auto next) {
      if (NTMAX == 1 || rows <= 8) k.template task<1>(w.p, rows, from, to, n, next);
      else if (NTMAX == 2 || rows <= 16)
        k.template task<NTMAX < 2 ? 1 : 2>(w.p, rows, from, to, n, next);
      else if (rows <= 24) k.template task<NTMAX < 4 ? 1 : 3>(w.p, rows, from, to, n, next);
      else k.template task<NTMAX < 4 ? 1 : 4>(w.p, rows, from, to, n, next);
    };
    if constexpr (!S::kDealt) {
      const int tasks = sh.pre[a.G] * k.per;
      for (int t = k.t0; t < tasks; ++n, t += k.nc)
        task(k.rows_of(w.p), 0, 0, [&]() {
          if (t + k.nc < tasks) k.advance(w.p, t + k.nc);
        });
    } else {
      for (; w.left > 0; ++n) {
        const int go = (int)min(w.left, (typename K::Count)((a.S - w.s + 1) / 2));
        task(k.rows_of(w.p), w.s, min(w.s + 2 * go, a.S), []() {});
        k.step(w, go);
      }
    }
    if (S::kLate && n > 0) k.finish(n - 1);
    __syncwarp();
  }
  if (a.split > 1) tc::cluster_barrier();  // no block leaves while another reads its sums
}

constexpr int kMostShared = 222 * 1024;

template <bool FIRST, int NTMAX, int P, int GS, Sharing HOW>
cudaError_t allow_shared() {
  static std::atomic<uint64_t> attr_set_mask{0};  // bit: device
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = 1ull << (dev & 63);
  if (attr_set_mask.load() & bit) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(w4_product<FIRST, NTMAX, P, GS, HOW>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
  if (e == cudaSuccess) attr_set_mask.fetch_or(bit);
  return e;
}

cudaLaunchConfig_t config(int blocks, int threads, size_t shared, cudaStream_t stream,
                          cudaLaunchAttribute (&attr)[2], int split) {
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  return cfg;
}

// Clusters of `split` blocks that are on the GPU at once: fewer than its SMs
// would give (of 152: 36 of four, 15 of eight), and the rest would come behind
// all of them.
template <bool FIRST, int NTMAX, int P, int GS>
int places(const Ctx& c, int split) {
  static std::atomic<int> known[64][9];  // one more than the number; 0: not asked yet
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  const int got = known[dev & 63][split].load();
  if (got != 0) return got - 1;
  constexpr Sharing kHow = NTMAX == 1 ? Sharing::kLate : Sharing::kInTurn;
  if (allow_shared<FIRST, NTMAX, P, GS, kHow>() != cudaSuccess) return 0;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = config(c.sm_count / split * split, Shape<NTMAX, kHow>::kThreads,
                                        kMostShared, c.stream, attr, split);
  if (cudaOccupancyMaxActiveClusters(&n, w4_product<FIRST, NTMAX, P, GS, kHow>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  known[dev & 63][split].store(n + 1);
  return n;
}

// How the blocks share the tasks. Whole tasks in turn (split 1); or clusters of
// `split` blocks share each one's slabs; or, with more than one token tile, all
// steps dealt out (split 0). The way with the least slabs per place (cluster that
// fits on the GPU), a task's start and end counted as four, the meeting of shared
// tasks in global memory as eight, and the earlier way when the next gains under
// 5%. How many rows each expert has is not known here: they count as even.
template <bool FIRST, int NTMAX, int P, int GS>
void plan(const Ctx& c, W4Args& a) {
  constexpr int kRows = 8 * NTMAX;
  const int64_t per = (a.n_tiles + kW4Tiles - 1) / kW4Tiles;
  const int64_t active = std::min<int64_t>(a.n_rows, a.G), each = (a.n_rows + active - 1) / active;
  const int64_t tasks = active * ((each + kRows - 1) / kRows) * per;
  const int64_t most = std::min<int64_t>(a.n_rows, a.G + a.n_rows / kRows) * per;
  a.split = 1;
  a.blocks = (int)std::min<int64_t>(c.sm_count, most);
  int64_t best = (tasks + c.sm_count - 1) / c.sm_count * (a.S + 4);
  for (int s = 2; s <= 8 && a.S >= 4 * s; s *= 2) {
    const int64_t fit = places<FIRST, NTMAX, P, GS>(c, s);
    if (fit == 0) continue;
    const int64_t cost = (tasks + fit - 1) / fit * ((a.S + s - 1) / s + 4);
    if (cost * 20 < best * 19) {
      best = cost;
      a.split = s;
      a.blocks = (int)std::min(fit, most) * s;
    }
  }
  if (NTMAX > 1) {
    const int64_t sms = std::min(c.sm_count, kW4MostBlocks);
    const int64_t cost = (tasks * (a.S + 4) + sms - 1) / sms + 8;
    if (cost * 20 < best * 19) {
      a.split = 0;
      a.blocks = (int)sms;
    }
  }
}

template <bool FIRST, int NTMAX, int P, int GS, Sharing HOW>
cudaError_t product(const Ctx& c, W4Args a) {
  using K = W4<FIRST, NTMAX, P, GS, HOW>;
  using S = Shape<NTMAX, HOW>;
  const cudaError_t e = allow_shared<FIRST, NTMAX, P, GS, HOW>();
  if (e != cudaSuccess) return e;
  CUtensorMap codes, xmap, xmap8;
  if (!tc::make_map_bf16(&codes, a.q, (int64_t)a.G * (FIRST ? 2 * (int64_t)a.F : a.d),
                         (int64_t)a.S * (kSlab / 4), S::kBoxRows) ||
      !tc::make_map_bf16_chunks(&xmap8, a.x, (int64_t)P * a.n_rows, a.ldx, 8, 4))
    return cudaErrorInvalidValue;
  xmap = xmap8;
  if (NTMAX > 1 &&
      !tc::make_map_bf16_chunks(&xmap, a.x, (int64_t)P * a.n_rows, a.ldx, 8 * NTMAX, 4))
    return cudaErrorInvalidValue;
  const int red = (S::kLate ? 4 : S::kWays == 2 ? 2 : a.split > 1 ? 1 : 0) * S::kPart * (int)sizeof(float);
  a.stages = std::min(kMaxStages, (kMostShared - 1024 - red) / K::kStage);
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = config(a.blocks, S::kThreads, 1024 + red + a.stages * K::kStage,
                                        c.stream, attr, a.split);
  note_launches(1);
  return cudaLaunchKernelEx(&cfg, w4_product<FIRST, NTMAX, P, GS, HOW>, (const CUtensorMap)codes,
                            (const CUtensorMap)xmap, (const CUtensorMap)xmap8, (const W4Args)a);
}

template <bool FIRST, int NTMAX, int P, int GS>
cudaError_t product_of(const Ctx& c, const W4Args& a) {
  W4Args b = a;
  plan<FIRST, NTMAX, P, GS>(c, b);
  constexpr Sharing kOther = NTMAX == 1 ? Sharing::kLate : Sharing::kDealt;
  if (NTMAX == 1 ? b.split > 1 : b.split == 0) return product<FIRST, NTMAX, P, GS, kOther>(c, b);
  return product<FIRST, NTMAX, P, GS, Sharing::kInTurn>(c, b);
}

template <int NTMAX, int P, int GS>
cudaError_t both(const Ctx& c, const W4Args& g1, const W4Args& g2) {
  const cudaError_t e = product_of<true, NTMAX, P, GS>(c, g1);
  return e != cudaSuccess ? e : product_of<false, NTMAX, P, GS>(c, g2);
}

// Both products of rows in one bf16 plane, or three (fp32).
template <int GS>
cudaError_t w4_both(const Ctx& c, int planes, const W4Args& g1, const W4Args& g2) {
  const bool few = w4_few(g1.n_rows, g1.G);
  if (planes == 1) return few ? both<1, 1, GS>(c, g1, g2) : both<4, 1, GS>(c, g1, g2);
  return few ? both<1, 3, GS>(c, g1, g2) : both<2, 3, GS>(c, g1, g2);
}

}  // namespace

}  // namespace moe
