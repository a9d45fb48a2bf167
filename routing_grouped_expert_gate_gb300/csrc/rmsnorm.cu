// Residual add + RMSNorm and its backward: the step between one block's output
// and the layer's input.
//
//   s = x + r,  rstd = 1 / sqrt(mean_j s_j^2 + eps),  y_j = s_j rstd w_j
//   dx_j = rstd (a_j - xh_j mean_i(a_i xh_i)) + d_sum_j,  a = dy w, xh = s rstd
//   dw_j = sum_t dy_tj xh_tj
//
// Both are bound by HBM: every element is read once and stays in registers
// between the row's sum and its use. Two chunks of eight elements a thread (one
// block a row, several blocks an SM) against one: 8192 x 7168 bf16 with the
// 8-bit output 79 us, 6.7 TB/s, against 92. A warp a row up to 512 columns
// (16000 x 512: 13.4 us, 14.1 with a block), a block above (16000 x 1000 fp32:
// 43 us, 52 with a warp).
#include <algorithm>
#include <atomic>

#include "common.cuh"
#include "internal.h"
#include "mx8.cuh"
#include "tc_ptx.cuh"

namespace moe {

namespace {

// Eight elements as loaded. Plain loads, not the read-only path: an output may
// be the very buffer that an input is in.
template <typename T> struct Row8;
template <> struct Row8<bf16> {
  uint4 a;
  __device__ __forceinline__ void load(const bf16* p) { a = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void read(const bf16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
template <> struct Row8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p + 4));
  }
  __device__ __forceinline__ void read(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

// The sum of one value per thread over the `warps` warps that share a row, in
// a fixed order; `red` holds one float per warp of the block. Every thread of
// the block calls it.
template <bool WARP_ROW>
__device__ __forceinline__ float row_sum(float v, float* red, int warps) {
  v = warp_sum(v);
  if (WARP_ROW) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  return warp_sum(lane < warps ? red[lane] : 0.f);
}

struct NormFwd {
  const void *x, *res;
  const float* w;
  void *sum, *y;
  uint8_t *y8, *y8_scale;
  float* rstd;
  float eps;
  int64_t T;
  int d;
};

// One row per block (WARP_ROW: per warp), C chunks of eight elements per
// thread, thread i holding chunks i, i + n, ... of the n threads of a row: a
// warp's loads and stores are 512 (bf16) or 1024 (fp32) consecutive bytes, and
// a block of the 8-bit format is a quad of lanes.
template <typename T, int C, bool WARP_ROW>
__global__ void __launch_bounds__(1024) rmsnorm_fwd(const NormFwd a) {
  __shared__ float red[32];
  pdl_wait();
  const int n = WARP_ROW ? 32 : blockDim.x;
  const int i0 = WARP_ROW ? (threadIdx.x & 31) : threadIdx.x;
  const int64_t row = WARP_ROW ? (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)
                               : (int64_t)blockIdx.x;
  if (WARP_ROW && row >= a.T) return;  // a whole warp
  const int n8 = a.d >> 3;
  const int64_t at = row * a.d;
  Row8<T> rx[C], rr[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = i0 + c * n;
    if (i < n8) {
      rx[c].load(static_cast<const T*>(a.x) + at + i * 8);
      if (a.res != nullptr) rr[c].load(static_cast<const T*>(a.res) + at + i * 8);
      else rr[c].zero();
    } else {
      rx[c].zero();
      rr[c].zero();
    }
  }
  float s[C][8];
  float ss = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    float v[8];
    rx[c].get(s[c]);
    rr[c].get(v);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s[c][e] += v[e];
      ss = fmaf(s[c][e], s[c][e], ss);
    }
    const int i = i0 + c * n;
    // the stream's own copy is rounded; the norm is of the unrounded sum
    if (a.sum != nullptr && i < n8) store8(static_cast<T*>(a.sum) + at + i * 8, s[c]);
  }
  ss = row_sum<WARP_ROW>(ss, red, blockDim.x >> 5);
  const float rstd = 1.f / sqrtf(ss / (float)a.d + a.eps);
  if (a.rstd != nullptr && i0 == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = i0 + c * n;
    float w[8];
    if (i < n8) {
      load8(a.w + i * 8, w);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = 0.f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) s[c][e] = s[c][e] * rstd * w[e];
    if (a.y != nullptr && i < n8) store8(static_cast<T*>(a.y) + at + i * 8, s[c]);
    if (a.y8 != nullptr) {
      // lanes past the row count as zeros (0 * an infinite rstd would be NaN)
      const uint32_t byte = mx8_scale_byte(quad_max(i < n8 ? abs_bits_max8(s[c]) : 0u));
      if (i < n8) {
        *reinterpret_cast<uint2*>(a.y8 + at + i * 8) = mx8_pack8(s[c], mx8_up(byte));
        if ((i & 3) == 0) a.y8_scale[row * ((a.d + 31) >> 5) + (i >> 2)] = (uint8_t)byte;
      }
    }
  }
}

struct NormBwd {
  const void *dy, *d_sum, *sum;
  const float *w, *rstd;
  void* dx;
  float* part;  // [blocks][d] partial sums of dw
  float inv_d;
  int64_t T;
  int d;
};

// Blocks take rows blockIdx.x, + gridDim.x, ... (WARP_ROW: warps do); a thread
// keeps the same columns for all of them, so dw's sums stay in registers and
// leave once per block. A row's loads are issued before the previous row's sum.
// Above 8192 columns a block of 1024 threads has 64 registers a thread for all of
// that, and some spill: 4096 x 12288 bf16 143 us, 2.8 TB/s, fp32 272 us, 3.0 TB/s.
template <typename T, int C, bool WARP_ROW, int THREADS>
__global__ void __launch_bounds__(THREADS) rmsnorm_bwd(const NormBwd a) {
  __shared__ float red[2][32];
  pdl_wait();
  const int n = WARP_ROW ? 32 : blockDim.x;
  const int i0 = WARP_ROW ? (threadIdx.x & 31) : threadIdx.x;
  const int per = WARP_ROW ? (blockDim.x >> 5) : 1;
  const int64_t step = (int64_t)gridDim.x * per;
  int64_t row = (int64_t)blockIdx.x * per + (WARP_ROW ? (threadIdx.x >> 5) : 0);
  const int n8 = a.d >> 3;
  float w[C][8], dw[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = i0 + c * n;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[c][e] = dw[c][e] = 0.f;
    if (i < n8) load8(a.w + i * 8, w[c]);
  }
  Row8<T> dy[C], sm[C], ds[C];
  float rstd = 0.f;
  auto fetch = [&](int64_t r) {
    const int64_t at = r * a.d;
    rstd = r < a.T ? __ldcs(a.rstd + r) : 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = i0 + c * n;
      if (i < n8 && r < a.T) {
        dy[c].load(static_cast<const T*>(a.dy) + at + i * 8);
        sm[c].load(static_cast<const T*>(a.sum) + at + i * 8);
        if (a.d_sum != nullptr) ds[c].load(static_cast<const T*>(a.d_sum) + at + i * 8);
        else ds[c].zero();
      } else {
        dy[c].zero();
        sm[c].zero();
        ds[c].zero();
      }
    }
  };
  fetch(row);
  for (int par = 0; row < a.T; row += step, par ^= 1) {
    // a * xh summed over the row; g = dy w and xh kept for the second use
    float g[C][8], xh[C][8], dot = 0.f;
    const float rs = rstd;
    Row8<T> keep[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      dy[c].get(g[c]);
      sm[c].get(xh[c]);
      keep[c] = ds[c];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xh[c][e] *= rs;
        dw[c][e] = fmaf(g[c][e], xh[c][e], dw[c][e]);
        g[c][e] *= w[c][e];
        dot = fmaf(g[c][e], xh[c][e], dot);
      }
    }
    fetch(row + step);
    const float m = row_sum<WARP_ROW>(dot, red[par], blockDim.x >> 5) * a.inv_d;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = i0 + c * n;
      if (i >= n8) continue;
      float k[8];
      keep[c].get(k);
#pragma unroll
      for (int e = 0; e < 8; ++e) k[e] += rs * (g[c][e] - xh[c][e] * m);
      store8(static_cast<T*>(a.dx) + row * a.d + i * 8, k);
    }
  }
  if (!WARP_ROW) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = i0 + c * n;
      if (i < n8) store8(a.part + (int64_t)blockIdx.x * a.d + i * 8, dw[c]);
    }
  } else {
    // the block's warps one after another into shared memory
    extern __shared__ float acc[];
    for (int k = 0; k < per; ++k) {
      if ((threadIdx.x >> 5) == k) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const int i = i0 + c * n;
          if (i < n8) {
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[i * 8 + e] = dw[c][e] + (k > 0 ? acc[i * 8 + e] : 0.f);
          }
        }
      }
      __syncthreads();
    }
    for (int j = threadIdx.x; j < a.d; j += blockDim.x)
      a.part[(int64_t)blockIdx.x * a.d + j] = acc[j];
  }
}

// The same, from 520 to 8192 columns, with the rows in a ring of shared memory
// that bulk copies fill some rows ahead: the registers hold only the rows at
// hand, and what a block has in flight does not depend on them. The row sum's
// barrier is also what says that a stage's rows have been read, so the next
// copies start right behind it.
constexpr int kRingBytes = 200 * 1024;  // of the blocks on an SM together
constexpr int kMaxRing = 8;

struct NormRing {
  NormBwd b;
  int stages, row_bytes;
  int* status;
  uint64_t timeout_ns;
};

// The sum over the block's warps from one float each in shared memory, in a
// fixed order; `warps` is rounded up to whole float4 and the rest is zero.
__device__ __forceinline__ float sum_of(const float* red, int warps) {
  float v = 0.f;
  for (int i = 0; i < warps; i += 4) {
    const float4 q = *reinterpret_cast<const float4*>(red + i);
    v += (q.x + q.y) + (q.z + q.w);
  }
  return v;
}

// R rows at a time share one barrier, and few blocks leave few partial sums. Where
// R rows a block would leave SMs without one, fewer: 300 x 4096 bf16 6.0 us with
// two rows, 6.7 with three; 16 x 4096 4.1 with one, 5.1 with three. A block holds
// no more stages than it has rounds, so that the column sums' blocks find room
// next to few rows' (300 x 2048 fp32 5.4 us, 6.0 with all stages).
// 16000 x 1000 bf16: 25 us with three rows and three blocks an SM, 27 with two
// and six, 36 with one (and 47 with a warp a row and no ring); 4096 x 4096 bf16
// 25.5 us with three and one block, 27.7 with two and two, 30 with one; fp32 45
// with two and one block, 52 with two and two blocks, 56 with three; 8192 x 2048
// bf16 26.0 with three and two blocks, 26.7 with two and three, fp32 43.5 with
// three and one block, 47.7; 8192 x 7168 bf16, one row at a time, 72 us, 6.5 TB/s
// (79 with two). Blocks take rows R b .. R b + R - 1, b = blockIdx.x, + gridDim.x, ...
template <typename T, int C, int R, int THREADS, int BLOCKS>
__global__ void __launch_bounds__(THREADS, BLOCKS) rmsnorm_bwd_ring(const NormRing r) {
  const NormBwd& a = r.b;
  __shared__ __align__(16) float red[2][R][32];
  __shared__ uint64_t full[kMaxRing];
  __shared__ int abort_flag;
  extern __shared__ __align__(128) char ring[];
  for (int i = threadIdx.x; i < 2 * R * 32; i += blockDim.x) (&red[0][0][0])[i] = 0.f;
  if (threadIdx.x == 0) {
    abort_flag = 0;
    for (int i = 0; i < r.stages; ++i) tc::mbar_init(&full[i], 1);
    tc::fence_barrier_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_launch_dependents();  // the sum of the blocks' parts, as soon as there is room
  const int ins = a.d_sum != nullptr ? 3 : 2, in_bytes = R * r.row_bytes;
  const int64_t pitch = (int64_t)gridDim.x * R;
  int64_t ahead = (int64_t)blockIdx.x * R;  // the next rows to load
  int n_loads = 0, load_at = 0;
  auto load = [&]() {  // thread 0
    if (ahead < a.T) {
      char* to = ring + load_at * ins * in_bytes;
      uint64_t* bar = &full[load_at];
      const int64_t at = ahead * r.row_bytes;
      const uint32_t bytes = (uint32_t)min((int64_t)R, a.T - ahead) * r.row_bytes;
      tc::mbar_expect_tx(bar, ins * bytes);
      tc::bulk_load_1d(to, static_cast<const char*>(a.dy) + at, bytes, bar);
      tc::bulk_load_1d(to + in_bytes, static_cast<const char*>(a.sum) + at, bytes, bar);
      if (ins == 3)
        tc::bulk_load_1d(to + 2 * in_bytes, static_cast<const char*>(a.d_sum) + at, bytes, bar);
      ahead += pitch;
      ++n_loads;
      if (++load_at == r.stages) load_at = 0;
    }
  };
  if (threadIdx.x == 0)
    for (int i = 0; i < r.stages; ++i) load();
  const int n = blockDim.x, n8 = a.d >> 3, warps = n >> 5;
  float w[C][8], dw[C][8];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = threadIdx.x + c * n;
#pragma unroll
    for (int e = 0; e < 8; ++e) w[c][e] = dw[c][e] = 0.f;
    if (i < n8) load8(a.w + i * 8, w[c]);
  }
  int st = 0, ph = 0, par = 0;
  bool ok = true;
  float rstd[R];
  auto next_rstd = [&](int64_t row) {
#pragma unroll
    for (int q = 0; q < R; ++q) rstd[q] = row + q < a.T ? __ldcs(a.rstd + row + q) : 0.f;
  };
  next_rstd((int64_t)blockIdx.x * R);
  for (int64_t row = (int64_t)blockIdx.x * R; row < a.T; row += pitch, par ^= 1) {
    float rs[R];
#pragma unroll
    for (int q = 0; q < R; ++q) rs[q] = rstd[q];
    next_rstd(row + pitch);
    if (ok) ok = tc::mbar_wait(&full[st], ph, abort_flag, r, 50);
    const char* from = ring + st * ins * in_bytes;
    float g[R][C][8], xh[R][C][8], dot[R];
    Row8<T> keep[R][C];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      dot[q] = 0.f;
      const bool have = R == 1 || row + q < a.T;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int i = threadIdx.x + c * n;
        if (i < n8 && have) {
          const char* at = from + q * r.row_bytes + i * 8 * sizeof(T);
          load8(reinterpret_cast<const T*>(at), g[q][c]);
          load8(reinterpret_cast<const T*>(at + in_bytes), xh[q][c]);
          if (ins == 3) keep[q][c].read(reinterpret_cast<const T*>(at + 2 * in_bytes));
          else keep[q][c].zero();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            xh[q][c][e] *= rs[q];
            dw[c][e] = fmaf(g[q][c][e], xh[q][c][e], dw[c][e]);
            g[q][c][e] *= w[c][e];
            dot[q] = fmaf(g[q][c][e], xh[q][c][e], dot[q]);
          }
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int q = 0; q < R; ++q) dot[q] += __shfl_xor_sync(0xffffffffu, dot[q], o);
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int q = 0; q < R; ++q) red[par][q][threadIdx.x >> 5] = dot[q];
    }
    __syncthreads();
    if (threadIdx.x == 0) load();  // every thread has read this stage
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const float m = sum_of(red[par][q], warps) * a.inv_d;
      const bool have = R == 1 || row + q < a.T;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int i = threadIdx.x + c * n;
        if (i < n8 && have) {
          float k[8];
          keep[q][c].get(k);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            k[e] = fmaf(rs[q], fmaf(-xh[q][c][e], m, g[q][c][e]), k[e]);
          store8(static_cast<T*>(a.dx) + (row + q) * a.d + i * 8, k);
        }
      }
    }
    if (++st == r.stages) {
      st = 0;
      ph ^= 1;
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = threadIdx.x + c * n;
    if (i < n8) store8(a.part + (int64_t)blockIdx.x * a.d + i * 8, dw[c]);
  }
  if (threadIdx.x == 0 && !ok) {
    // a wait gave up: the copies in flight land before the block ends
    const uint64_t from = global_timer_ns();
    for (int i = 0; i < r.stages; ++i) {
      const int k = (n_loads + r.stages - 1 - i) / r.stages;
      while (k > 0 && !tc::mbar_try_wait(&full[i], (k - 1) & 1) &&
             global_timer_ns() - from < r.timeout_ns) {
      }
    }
  }
}

// dw[j] = sum over the blocks' partials, in a fixed order: 32 strided sums per
// column, then those in turn.
__global__ void __launch_bounds__(1024) rmsnorm_dw(const float* part, int blocks, int d, float* dw) {
  __shared__ float acc[32][33];
  pdl_wait();
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5, j = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (j < d) {
    for (int b0 = g; b0 < blocks; b0 += 8 * 32) {  // eight loads, then their sum
      float q[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        q[u] = b0 + u * 32 < blocks ? part[(int64_t)(b0 + u * 32) * d + j] : 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) v += q[u];
    }
  }
  acc[g][lane] = v;
  __syncthreads();
  v = warp_sum(acc[lane][g]);  // column g's 32 sums
  const int col = blockIdx.x * 32 + g;
  if (lane == 0 && col < d) dw[col] = v;
}

__global__ void __launch_bounds__(256) rmsnorm_zero(float* dw, int d) {
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j < d) dw[j] = 0.f;
}

constexpr int kMostSms = 256;  // the workspace is sized without a device
int device_sms(const Ctx& c) { return std::min(c.sm_count, kMostSms); }

// threads of a row-per-block kernel with C chunks of 8 per thread
int row_threads(int d, int C) {
  const int n = (d / 8 + C - 1) / C;
  return (n + 31) / 32 * 32;
}

constexpr int kWarpRowD = 512;  // up to here a warp holds a row (two chunks a lane)
constexpr int kWarpsPerBlock = 8;

// The backward's shape for a size: rows at a time, chunks of eight elements and
// threads of a block, blocks on an SM.
struct BwdShape {
  int rows, chunks, threads, per_sm;
};
BwdShape bwd_shape(int64_t T, int d, int act_dtype, int sms) {
  if (d <= kWarpRowD) return {kWarpsPerBlock, d <= 256 ? 1 : 2, 32 * kWarpsPerBlock, 4};
  if (d > 8192) return {1, 2, row_threads(d, 2), 1};
  const int es = act_dtype == MOE_BF16 ? 2 : 4;
  BwdShape s = d <= 1024   ? BwdShape{3, 1, 0, 3}
               : d <= 2048 ? BwdShape{3, 1, 0, es == 2 ? 2 : 1}
               : d <= 4096 ? BwdShape{es == 2 ? 3 : 2, 1, 0, 1}
                           : BwdShape{1, 2, 0, 1};
  // no more rows at a time than give every SM a block
  s.rows = (int)std::max<int64_t>(1, std::min<int64_t>(s.rows, (T + sms - 1) / sms));
  // A block of 512 threads leaves the column sums' blocks no registers. With one
  // round a block it pays to start them early: half as many threads (200 x 4096
  // bf16 5.6 us, 6.2 with 512; fp32 gains nothing).
  if (es == 2 && d > 2048 && T <= 2 * (int64_t)sms) s.chunks = 2;
  s.threads = row_threads(d, s.chunks);
  // two stages of three inputs for each block, or fewer blocks
  s.per_sm = std::max(1, std::min(s.per_sm, kRingBytes / (6 * s.rows * d * es)));
  return s;
}

int bwd_blocks(const moe_cfg& cfg, int sms) {
  const BwdShape s = bwd_shape(cfg.T, cfg.d, cfg.act_dtype, sms);
  return (int)std::min<int64_t>((cfg.T + s.rows - 1) / s.rows, (int64_t)s.per_sm * sms);
}

template <typename T>
cudaError_t fwd(const Ctx& c, const NormFwd& a) {
  note_launches(1);
  if (a.d <= kWarpRowD) {
    const int64_t blocks = (a.T + kWarpsPerBlock - 1) / kWarpsPerBlock;
    const dim3 g((unsigned)blocks), b(32 * kWarpsPerBlock);
    if (a.d <= 256) return launch_dependent(rmsnorm_fwd<T, 1, true>, g, b, 0, c.stream, a);
    return launch_dependent(rmsnorm_fwd<T, 2, true>, g, b, 0, c.stream, a);
  }
  const dim3 g((unsigned)a.T);
  return launch_dependent(rmsnorm_fwd<T, 2, false>, g, dim3(row_threads(a.d, 2)), 0, c.stream, a);
}

template <typename T, int C, int R, int THREADS, int BLOCKS>
cudaError_t launch_ring(const Ctx& c, const NormBwd& a, const BwdShape& s, int blocks) {
  auto kern = rmsnorm_bwd_ring<T, C, R, THREADS, BLOCKS>;
  static std::atomic<uint64_t> attr_set_mask{0};  // bit: device
  int dev = 0;
  cudaGetDevice(&dev);
  const uint64_t bit = 1ull << (dev & 63);
  if (!(attr_set_mask.load() & bit)) {
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (e != cudaSuccess) return e;
    attr_set_mask.fetch_or(bit);
  }
  const int row_bytes = a.d * (int)sizeof(T), stage = (a.d_sum != nullptr ? 3 : 2) * R * row_bytes;
  const int64_t rounds = (a.T + (int64_t)R * blocks - 1) / ((int64_t)R * blocks);
  const int stages = (int)std::min<int64_t>(rounds, std::min(kMaxRing, kRingBytes / s.per_sm / stage));
  const NormRing r{a, stages, row_bytes, c.status, c.timeout_ns};
  return launch_dependent(kern, dim3(blocks), dim3(s.threads), (size_t)r.stages * stage, c.stream, r);
}

// up to R rows at a time
template <typename T, int C, int R, int THREADS, int BLOCKS>
cudaError_t launch_rows(const Ctx& c, const NormBwd& a, const BwdShape& s, int blocks) {
  if (s.rows == 1) return launch_ring<T, C, 1, THREADS, BLOCKS>(c, a, s, blocks);
  if (R == 2 || s.rows == 2) return launch_ring<T, C, 2, THREADS, BLOCKS>(c, a, s, blocks);
  return launch_ring<T, C, R, THREADS, BLOCKS>(c, a, s, blocks);
}

template <typename T>
cudaError_t bwd(const Ctx& c, const NormBwd& a, int blocks) {
  constexpr bool kHalf = sizeof(T) == 2;
  const BwdShape s = bwd_shape(a.T, a.d, kHalf ? MOE_BF16 : MOE_F32, device_sms(c));
  if (a.d <= kWarpRowD) {
    const dim3 g(blocks), b(s.threads);
    const size_t sm = (size_t)a.d * sizeof(float);
    if (a.d <= 256) return launch_dependent(rmsnorm_bwd<T, 1, true, 256>, g, b, sm, c.stream, a);
    return launch_dependent(rmsnorm_bwd<T, 2, true, 256>, g, b, sm, c.stream, a);
  }
  if (a.d <= 1024) return launch_rows<T, 1, 3, 128, 3>(c, a, s, blocks);
  if (a.d <= 2048) return launch_rows<T, 1, 3, 256, kHalf ? 2 : 1>(c, a, s, blocks);
  if constexpr (kHalf)
    if (a.d <= 4096 && s.chunks == 2) return launch_rows<T, 2, 2, 256, 2>(c, a, s, blocks);
  if (a.d <= 4096) return launch_rows<T, 1, kHalf ? 3 : 2, 512, 1>(c, a, s, blocks);
  if (a.d <= 8192) return launch_ring<T, 2, 1, 512, 1>(c, a, s, blocks);
  return launch_dependent(rmsnorm_bwd<T, 2, false, 1024>, dim3(blocks), dim3(s.threads), 0,
                          c.stream, a);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const Ctx& c, const moe_cfg& cfg, const void* x, const void* res,
                               const float* w, float eps, void* sum, void* y, uint8_t* y8,
                               uint8_t* y8_scale, float* rstd) {
  NormFwd a{x, res, w, sum, y, y8, y8_scale, rstd, eps, cfg.T, cfg.d};
  return cfg.act_dtype == MOE_BF16 ? fwd<bf16>(c, a) : fwd<float>(c, a);
}

size_t rmsnorm_bwd_ws_bytes(const moe_cfg& cfg) {
  return (size_t)bwd_blocks(cfg, kMostSms) * cfg.d * sizeof(float);
}

cudaError_t launch_add_rmsnorm_bwd(const Ctx& c, const moe_cfg& cfg, const void* dy,
                                   const void* d_sum, const void* sum, const float* w,
                                   const float* rstd, void* dx, float* dw, void* ws) {
  if (cfg.T == 0) {
    rmsnorm_zero<<<(cfg.d + 255) / 256, 256, 0, c.stream>>>(dw, cfg.d);
    note_launches(1);
    return cudaGetLastError();
  }
  const int blocks = bwd_blocks(cfg, device_sms(c));
  NormBwd a{dy, d_sum, sum, w, rstd, dx, static_cast<float*>(ws), 1.f / (float)cfg.d, cfg.T, cfg.d};
  cudaError_t e = cfg.act_dtype == MOE_BF16 ? bwd<bf16>(c, a, blocks) : bwd<float>(c, a, blocks);
  if (e != cudaSuccess) return e;
  e = launch_dependent(rmsnorm_dw, dim3((cfg.d + 31) / 32), dim3(1024), 0, c.stream,
                       (const float*)ws, blocks, cfg.d, dw);
  note_launches(2);
  return e;
}

}  // namespace moe
