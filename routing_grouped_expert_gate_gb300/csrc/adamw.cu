// One AdamW step over many tensors in one pass: a launch for each kTable tensors
// with 32-bit states and one for each kTable with 8-bit states.
//
//   g' = g * grad_scale,  m = b1 m + (1 - b1) g',  v = b2 v + (1 - b2) g'^2
//   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Bound by HBM: each element's parameter, gradient and states are read once and
// written once (28 bytes for a bf16 parameter with an fp32 master copy and fp32
// states, 16.1 with 8-bit states): 562 M parameters take 2.36 ms, 6.7 TB/s, with
// 32-bit states, 604 M with 8-bit ones 1.69 ms, 5.8 TB/s; 94 small tensors 9 us
// on the GPU. All arithmetic is fp32, whatever the storage types; m and v take one
// rounding per product and sum, the parameter's update may use fused ones. The
// 8-bit states hold m and sqrt(v) (the root halves v's range of exponents, which
// e4m3 needs) in blocks of 32 with a power-of-two scale; a root that is not zero
// is kept at least as the format's smallest step, so that no later step divides by
// eps alone.
#include <math.h>

#include "common.cuh"
#include "internal.h"
#include "mx8.cuh"

namespace moe {

namespace {

constexpr int kTable = 96;      // tensors per launch (their table travels as a kernel parameter)
template <bool BITS8> constexpr int kThreads = BITS8 ? 128 : 256;
template <bool BITS8> constexpr int kChunk = kThreads<BITS8> * 8;  // elements: eight per thread

struct Entry {
  void* p;
  const void* g;
  float* master;
  void *m, *v;
  uint8_t *m_scale, *v_scale;
  int64_t n;
  float decay;  // 1 - lr * weight_decay, or weight_decay when lr_scale is given
  int kind;     // bit 0: p bf16, 1: g bf16, 2: master
};

struct Table {
  Entry e[kTable];
  int64_t first[kTable + 1];  // first chunk of each tensor
  int count;
  int last;  // this launch ends the step
  float beta1, beta2, one_minus_b1, one_minus_b2, eps;
  double lr, log_b1, log_b2;
  int64_t* step;
  const float *grad_scale, *lr_scale;
};

struct Hyper {
  float rate, root, lr, gs;  // lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
};

template <typename T>
__device__ __forceinline__ void get8(const T* p, int64_t at, int cnt, float (&v)[8]) {
  if (cnt == 8) {
    load8(p + at, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < cnt ? to_f32<T>(p[at + i]) : 0.f;
  }
}

template <typename T>
__device__ __forceinline__ void put8(T* p, int64_t at, int cnt, const float (&v)[8]) {
  if (cnt == 8) {
    store8(p + at, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < cnt) p[at + i] = from_f32<T>(v[i]);
  }
}

__device__ __forceinline__ uint2 get8b(const uint8_t* p, int64_t at, int cnt) {
  if (cnt == 8) return *reinterpret_cast<const uint2*>(p + at);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < cnt) w[i >> 2] |= (uint32_t)p[at + i] << (8 * (i & 3));
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void put8b(uint8_t* p, int64_t at, int cnt, uint2 q) {
  if (cnt == 8) {
    *reinterpret_cast<uint2*>(p + at) = q;
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < cnt) p[at + i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
}

// eight elements of one tensor per thread, at element `at` (cnt of them exist)
template <typename P, typename G, bool MASTER, bool BITS8>
__device__ __forceinline__ void update8(const Entry& e, const Table& t, const Hyper& h, int64_t at,
                                        int cnt) {
  float g[8], p[8], m[8], v[8];
  get8(static_cast<const G*>(e.g), at, cnt, g);
  if (MASTER) get8(e.master, at, cnt, p);
  else get8(static_cast<const P*>(e.p), at, cnt, p);
  if (BITS8) {
    const uint2 qm = get8b(static_cast<const uint8_t*>(e.m), at, cnt);
    const uint2 qv = get8b(static_cast<const uint8_t*>(e.v), at, cnt);
    const float sm = cnt > 0 ? mx8_scale(e.m_scale[at >> 5]) : 0.f;
    const float sv = cnt > 0 ? mx8_scale(e.v_scale[at >> 5]) : 0.f;
    mx8_unpack8(qm, sm, m);
    mx8_unpack8(qv, sv, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fmul_rn(v[i], v[i]);
  } else {
    get8(static_cast<const float*>(e.m), at, cnt, m);
    get8(static_cast<const float*>(e.v), at, cnt, v);
  }
  const float decay = t.lr_scale != nullptr ? 1.f - h.lr * e.decay : e.decay;
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float gi = __fmul_rn(g[i], h.gs);
    m[i] = __fadd_rn(__fmul_rn(m[i], t.beta1), __fmul_rn(gi, t.one_minus_b1));
    v[i] = __fadd_rn(__fmul_rn(v[i], t.beta2), __fmul_rn(__fmul_rn(gi, gi), t.one_minus_b2));
    r[i] = __fsqrt_rn(v[i]);
    // 8-bit states leave less time for arithmetic: the fast quotient there, off by
    // 2^-22 of a step whose m and v were kept to 2^-4 (604 M parameters 1685 us,
    // 1737 with the rounded quotient). The states do not see it.
    const float den = fmaf(r[i], h.root, t.eps);
    p[i] = p[i] * decay - (BITS8 ? __fdividef(m[i], den) : m[i] / den) * h.rate;
  }
  put8(static_cast<P*>(e.p), at, cnt, p);
  if (MASTER) put8(e.master, at, cnt, p);
  if (BITS8) {
#pragma unroll
    for (int i = 0; i < 8; ++i)  // elements past the end must not enter the block's maximum
      if (i >= cnt) m[i] = r[i] = 0.f;
    const uint32_t bm = mx8_scale_byte(quad_max(abs_bits_max8(m)));
    const uint32_t bv = mx8_scale_byte(quad_max(abs_bits_max8(r)));
    put8b(static_cast<uint8_t*>(e.m), at, cnt, mx8_pack8(m, mx8_up(bm)));
    // at least the smallest step, 2^-9, unless it is zero: what lies below
    // would round to that step or to nothing
    const float up = mx8_up(bv);
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = fmaxf(r[i] * up, r[i] > 0.f ? 0x1p-9f : 0.f);
    put8b(static_cast<uint8_t*>(e.v), at, cnt, mx8_pack8(r, 1.f));
    if (cnt > 0 && (at & 31) == 0) {
      e.m_scale[at >> 5] = (uint8_t)bm;
      e.v_scale[at >> 5] = (uint8_t)bv;
    }
  } else {
    put8(static_cast<float*>(e.m), at, cnt, m);
    put8(static_cast<float*>(e.v), at, cnt, v);
  }
}

// Blocks on an SM. 32-bit states have enough bytes in flight with three of 256
// threads, and more only spread the accesses over more DRAM pages (562 M bf16
// parameters with master copies: 2363 us with three, 2570 with four, 2593 with
// five). 8-bit states want ten of 128 (604 M: 1690 us, 1731 with nine, 1839 with
// eleven; of 256 threads 1718 with five, 1818 with six, 1854 with four).
template <bool BITS8> constexpr int kBlocks = BITS8 ? 10 : 3;

template <bool BITS8>
__global__ void __launch_bounds__(kThreads<BITS8>, kBlocks<BITS8>)
    adamw_kernel(const __grid_constant__ Table t) {
  __shared__ Hyper sh;
  __shared__ int64_t s_step;
  if (threadIdx.x == 0) {
    const int64_t k = t.step[0] + 1;
    const double lr = t.lr_scale != nullptr ? t.lr * (double)t.lr_scale[0] : t.lr;
    // 1 - b^t = -expm1(t log b), without the cancellation of 1 - pow; only the
    // exponent needs 64 bits
    sh.rate = (float)lr / -expm1f((float)((double)k * t.log_b1));
    sh.root = 1.f / sqrtf(-expm1f((float)((double)k * t.log_b2)));
    sh.lr = (float)lr;
    sh.gs = t.grad_scale != nullptr ? t.grad_scale[0] : 1.f;
    s_step = k;
  }
  __syncthreads();
  const Hyper h = sh;
  const int64_t chunks = t.first[t.count];
  int j = 0;
  for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
    // the tensor of chunk c: the last whose first chunk is not past it
    int lo = j, hi = t.count - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (t.first[mid] <= c) lo = mid;
      else hi = mid - 1;
    }
    j = lo;
    const Entry& e = t.e[j];
    const int64_t at = (c - t.first[j]) * kChunk<BITS8> + threadIdx.x * 8;
    const int64_t left = e.n - at;
    const int cnt = left >= 8 ? 8 : (left > 0 ? (int)left : 0);
    switch (e.kind) {
      case 0: update8<float, float, false, BITS8>(e, t, h, at, cnt); break;
      case 1: update8<bf16, float, false, BITS8>(e, t, h, at, cnt); break;
      case 2: update8<float, bf16, false, BITS8>(e, t, h, at, cnt); break;
      case 3: update8<bf16, bf16, false, BITS8>(e, t, h, at, cnt); break;
      case 5: update8<bf16, float, true, BITS8>(e, t, h, at, cnt); break;
      default: update8<bf16, bf16, true, BITS8>(e, t, h, at, cnt); break;
    }
  }
  if (t.last == 0) return;
  // the block that finishes last counts the step: by then every block has read
  // it. The second word is the ticket, 0 between calls.
  if (threadIdx.x == 0) {
    unsigned long long* ticket = reinterpret_cast<unsigned long long*>(t.step + 1);
    __threadfence();
    if (atomicAdd(ticket, 1ull) == gridDim.x - 1) {
      *ticket = 0;
      t.step[0] = s_step;
    }
  }
}

}  // namespace

cudaError_t launch_adamw(const Ctx& c, const moe_adamw_tensor* tensors, int n, double lr,
                         double beta1, double beta2, double eps, int64_t* step,
                         const float* grad_scale, const float* lr_scale) {
  Table t{};
  t.lr = lr;
  t.beta1 = (float)beta1;
  t.beta2 = (float)beta2;
  t.one_minus_b1 = (float)(1.0 - beta1);
  t.one_minus_b2 = (float)(1.0 - beta2);
  t.eps = (float)eps;
  t.log_b1 = log(beta1);  // -inf for 0: expm1 gives -1
  t.log_b2 = log(beta2);
  t.step = step;
  t.grad_scale = grad_scale;
  t.lr_scale = lr_scale;
  // the tensors with 32-bit states first, then those with 8-bit ones, each in
  // tables of up to kTable
  int left[2] = {0, 0};
  for (int i = 0; i < n; ++i)
    if (tensors[i].n > 0) ++left[tensors[i].state_bits == 8];
  int i = 0;
  bool bits8 = left[0] == 0;
  do {
    t.count = 0;
    t.first[0] = 0;
    const int chunk = bits8 ? kChunk<true> : kChunk<false>;
    for (; i < n && t.count < kTable; ++i) {
      const moe_adamw_tensor& s = tensors[i];
      if (s.n == 0 || (s.state_bits == 8) != bits8) continue;
      Entry& e = t.e[t.count];
      e.p = s.p;
      e.g = s.g;
      e.master = s.master;
      e.m = s.m;
      e.v = s.v;
      e.m_scale = s.m_scale;
      e.v_scale = s.v_scale;
      e.n = s.n;
      e.decay = lr_scale != nullptr ? s.weight_decay : (float)(1.0 - lr * s.weight_decay);
      e.kind = (s.p_dtype == MOE_BF16 ? 1 : 0) | (s.g_dtype == MOE_BF16 ? 2 : 0) |
               (s.master != nullptr ? 4 : 0);
      ++t.count;
      t.first[t.count] = t.first[t.count - 1] + (s.n + chunk - 1) / chunk;
    }
    left[bits8] -= t.count;
    t.last = left[0] + left[1] == 0;
    const int64_t chunks = t.first[t.count];
    const int64_t most = (int64_t)c.sm_count * (bits8 ? kBlocks<true> : kBlocks<false>);
    const int grid = (int)(chunks < 1 ? 1 : (chunks < most ? chunks : most));
    if (bits8) adamw_kernel<true><<<grid, kThreads<true>, 0, c.stream>>>(t);
    else adamw_kernel<false><<<grid, kThreads<false>, 0, c.stream>>>(t);
    note_launches(1);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (!bits8 && left[0] == 0) {
      bits8 = true;
      i = 0;
    }
  } while (!t.last);
  return cudaSuccess;
}

}  // namespace moe
