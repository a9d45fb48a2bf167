// Expert products with 4-bit weights, for few rows per expert (decoding).
//
//   w[n, k] = (u[n, k] - 8) * s[n, k / group],  u in 0..15, s bf16
//   h[r] = act(x[r] W1g^T, x[r] W1u^T),  out[r] = h[r] W2^T
//
// The bytes to move are the active experts' codes and scales, once (0.52 to
// 0.56 per weight). The weights are the A operand (16 weight rows by 16 k) of
// mma.sync m16n8k16 and eight tokens its N, so a pass over the weights serves
// eight tokens for the price of one. tcgen05 would want the decoded weights in
// shared or tensor memory first, four times the codes' bytes, and its
// accumulators back after every scale group.
//
// What it spends its time on beside the loads is the decoding: eleven
// instructions per eight codes, (word >> 4 i) & 0x000f000f | 0x43004300 being a
// pair of bf16 128 + u and a packed subtraction of 136 making it u - 8, exactly.
// The products of a scale group are summed in fp32 by the tensor cores, then
// multiplied by the group's scale and added in fp32: the weights themselves are
// never rounded.
//
// The code layout makes a lane's 16-byte load hold its operands of four
// consecutive 32-k blocks: within 128 k, the word at position 4 t + j holds k
// = 32 j + 8 t + (0, 2, 4, 6, 1, 3, 5, 7). Lane quad t of a block then owns k
// 8 t .. 8 t + 7, and the matching activations are 16 consecutive bytes.
//
// Measured (GB300, all launches of a call): one token through 2 of 8 experts of
// 4096 x 14336, groups of 128: 50 us, 3.6 TB/s (82 us with codes straight to
// registers and one slab ahead); 12 tokens, 8 of 64 experts of 2048 x 1408 each,
// groups of 32: 65 us, 3.8 TB/s; 64 tokens, 2 of 8 wide experts, groups of 64:
// 218 us, 3.4 TB/s. With the arithmetic left out the same loads take 37, 47 and
// 132 us; with the codes' loads left out the arithmetic takes 45, 57 and 209 us.
// fp32 rows (three planes, three times the products): one token, 2 of 8 wide
// experts, groups of 128: 65 us; 24 tokens, groups of 64: 266 us.
#include "common.cuh"
#include "internal.h"
#include "mx8.cuh"
#include "w4.h"

namespace moe {

namespace {

// ------------------------------------------------------------ quantise

// Eight consecutive k per thread; a group's 4, 8 or 16 threads are neighbours.
// Each weight is read once and each code written once, by one short thread per
// eight weights, eight exact divisions in it: 8 x 28672 x 4096 bf16 in groups of
// 128 1250 us, 1.9 TB/s, fp32 1229 us, 3.5 TB/s. It runs once for a layer's weights.
template <typename T>
__global__ void __launch_bounds__(256) w4_quantize_kernel(const T* w, int64_t rows, int K,
                                                          int group, uint8_t* q, bf16* scales) {
  pdl_wait();
  const int S = slabs_of(K), words = S * 16;
  const int64_t n = rows * words;  // words of 32 bits; a multiple of 16
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = i / words;
  const int wk = (int)(i - row * words), k = wk * 8;
  const bool in = i < n && k < K;
  float v[8];
  if (in) {
    load8(w + row * K + k, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
  }
  uint32_t a = abs_bits_max8(v);
  for (int o = 1; o < group / 8; o <<= 1) a = max(a, __shfl_xor_sync(0xffffffffu, a, o));
  if (i >= n) return;
  const bool bad = a >= 0x7f800000u;
  const bf16 s = from_f32<bf16>(bad ? __uint_as_float(0x7fffffffu)
                                    : __fdiv_rn(__uint_as_float(a), 7.f));
  const float sf = to_f32<bf16>(s);
  uint32_t out = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // bf16(amax / 7) may round down, so a code may reach 7 from above
    const float r = (sf > 0.f) ? rintf(__fdiv_rn(v[e], sf)) : 0.f;
    const uint32_t u = (uint32_t)((int)fminf(fmaxf(r, -8.f), 7.f) + 8);
    out |= u << (4 * ((e >> 1) + 4 * (e & 1)));
  }
  if (bad) out = 0x88888888u;
  const int in_slab = wk & 15;  // = 4 j + t, stored at 4 t + j
  const int at = (wk & ~15) + (in_slab & 3) * 4 + (in_slab >> 2);
  reinterpret_cast<uint32_t*>(q)[row * words + at] = out;
  if ((wk & (group / 8 - 1)) == 0) scales[row * (S * kSlab / group) + k / group] = s;
}

// Eight consecutive k per thread: 8 x 28672 x 4096 in groups of 128 to bf16 619 us,
// 3.8 TB/s, to fp32 748 us, 5.7 TB/s.
template <typename T>
__global__ void __launch_bounds__(256) w4_dequantize_kernel(const uint8_t* q, const bf16* scales,
                                                            int64_t rows, int K, int group, T* w) {
  pdl_wait();
  const int S = slabs_of(K), words = K >> 3;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= rows * words) return;
  const int64_t row = i / words;
  const int wk = (int)(i - row * words), in_slab = wk & 15;
  const int at = (wk & ~15) + (in_slab & 3) * 4 + (in_slab >> 2);
  const uint32_t c = reinterpret_cast<const uint32_t*>(q)[row * (S * 16) + at];
  const float s = to_f32<bf16>(scales[row * (S * kSlab / group) + wk * 8 / group]);
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e)
    v[e] = (float)((int)((c >> (4 * ((e >> 1) + 4 * (e & 1)))) & 15u) - 8) * s;
  store8(w + row * K + wk * 8, v);
}

// ------------------------------------------------------------ rows

// Row r of the call, x[src[r]] (zeros where src leaves x), next to row r - 1 as
// bf16: the act dtype's values, the 8-bit format's (exact), or three planes of
// fp32; eight elements per thread, zeros in the pitch's rest. Also zeros in the
// rest of h's pitch, which the first product does not write, and in the
// products' tickets.
template <int XK>
__global__ void __launch_bounds__(256) w4_rows(const void* x, const uint8_t* scale,
                                               const int32_t* src, int64_t x_rows, int64_t n_rows,
                                               int d, bf16* out, int F, bf16* h, uint32_t* came) {
  pdl_wait();
  // the product may start: it reads weights and offsets, complete by now
  pdl_launch_dependents();
  constexpr int P = XK == kRowsF32 ? 3 : 1;
  const int d8 = d >> 3, p8 = w4_pitch(d) >> 3;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, n8 = n_rows * p8;
  if (blockIdx.x == 0 && came != nullptr)
    for (int k = threadIdx.x; k < 2 * kW4Came; k += 256) came[k] = 0;
  if (i >= n8) {
    const int F8 = F >> 3, h8 = w4_pitch(F) >> 3, rest = h8 - F8;
    const int64_t k = i - n8;
    if (k < n_rows * P * rest)
      reinterpret_cast<uint4*>(h)[k / rest * h8 + F8 + k % rest] = make_uint4(0, 0, 0, 0);
    return;
  }
  const int64_t r = i / p8;
  const int c = (int)(i - r * p8);
  const int64_t row = src != nullptr ? (int64_t)src[r] : r;
  const bool in = row >= 0 && row < x_rows && c < d8;
  const int64_t at = row * d8 + c;
  if constexpr (XK == kRowsBf16) {
    reinterpret_cast<uint4*>(out)[i] =
        in ? static_cast<const uint4*>(x)[at] : make_uint4(0, 0, 0, 0);
  } else if constexpr (XK == kRows8) {
    float v[8] = {};
    if (in)
      mx8_unpack8(static_cast<const uint2*>(x)[at],
                  mx8_scale(scale[row * ((d8 + 3) >> 2) + (c >> 2)]), v);
    store8(out + i * 8, v);
  } else {
    float v[8] = {}, p[3][8];
    if (in) load8(static_cast<const float*>(x) + at * 8, v);
#pragma unroll
    for (int e = 0; e < 8; ++e) planes3(v[e], p[0][e], p[1][e], p[2][e]);
#pragma unroll
    for (int k = 0; k < 3; ++k) store8(out + (k * n8 + i) * 8, p[k]);
  }
}

}  // namespace

int w4_padded_k(int K) { return slabs_of(K) * kSlab; }

cudaError_t launch_w4_quantize(const Ctx& c, int64_t rows, int K, int group, int dt, const void* w,
                               uint8_t* q, void* scales) {
  const int64_t words = rows * (int64_t)(w4_padded_k(K) / 8);
  const dim3 g((unsigned)((words + 255) / 256));
  note_launches(1);
  if (dt == kBF16)
    return launch_dependent(w4_quantize_kernel<bf16>, g, dim3(256), 0, c.stream, (const bf16*)w,
                            rows, K, group, q, (bf16*)scales);
  return launch_dependent(w4_quantize_kernel<float>, g, dim3(256), 0, c.stream, (const float*)w,
                          rows, K, group, q, (bf16*)scales);
}

cudaError_t launch_w4_dequantize(const Ctx& c, int64_t rows, int K, int group, int dt,
                                 const uint8_t* q, const void* scales, void* w) {
  const int64_t words = rows * (int64_t)(K / 8);
  const dim3 g((unsigned)((words + 255) / 256));
  note_launches(1);
  if (dt == kBF16)
    return launch_dependent(w4_dequantize_kernel<bf16>, g, dim3(256), 0, c.stream, q,
                            (const bf16*)scales, rows, K, group, (bf16*)w);
  return launch_dependent(w4_dequantize_kernel<float>, g, dim3(256), 0, c.stream, q,
                          (const bf16*)scales, rows, K, group, (float*)w);
}

static size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// h and the rows next to each other, fp32 as three bf16 planes; then, for calls
// that may have more than one token tile, the two products' tickets and the
// blocks' partial sums
size_t w4_ws_bytes(int dt, int64_t n_rows, int d, int F) {
  const int planes = dt == kF32 ? 3 : 1;
  const size_t e = planes * sizeof(bf16);
  const size_t rows = up256((size_t)n_rows * w4_pitch(F) * e) + up256((size_t)n_rows * w4_pitch(d) * e);
  if (w4_few(n_rows, 1)) return rows;
  return rows + 2 * kW4Came * sizeof(uint32_t) + w4_part_floats(planes) * sizeof(float);
}

cudaError_t launch_w4_grouped_swiglu(const Ctx& c, int dt, int G, int64_t n_rows, int F, int d,
                                     int group, const int32_t* offsets, const void* x,
                                     const uint8_t* x_scale, int64_t x_rows, const int32_t* src,
                                     const uint8_t* w1_q, const void* w1_s, const uint8_t* w2_q,
                                     const void* w2_s, void* out, void* ws) {
  const int planes = dt == kF32 ? 3 : 1;
  bf16* h = static_cast<bf16*>(ws);
  bf16* rows = reinterpret_cast<bf16*>(static_cast<char*>(ws) +
                                       up256((size_t)n_rows * w4_pitch(F) * planes * sizeof(bf16)));
  uint32_t* came = nullptr;
  if (!w4_few(n_rows, G))
    came = reinterpret_cast<uint32_t*>(
        reinterpret_cast<char*>(rows) + up256((size_t)n_rows * w4_pitch(d) * planes * sizeof(bf16)));
  // Also where bf16 rows lie in order already: the products start on this
  // kernel's signal, with every launch before it complete, and load weights
  // while it runs.
  const int64_t n8 = n_rows * (w4_pitch(d) / 8) + n_rows * planes * ((w4_pitch(F) - F) / 8);
  auto kern = dt == kF32 ? w4_rows<kRowsF32> : x_scale != nullptr ? w4_rows<kRows8> : w4_rows<kRowsBf16>;
  const cudaError_t e = launch_dependent(kern, dim3((unsigned)((n8 + 255) / 256)), dim3(256), 0,
                                         c.stream, x, x_scale, src, x_rows, n_rows, d, rows, F, h, came);
  note_launches(1);
  if (e != cudaSuccess) return e;
  W4Args a{};
  a.G = G;
  a.n_rows = (int)n_rows;
  a.F = F;
  a.d = d;
  a.offsets = offsets;
  a.act = c.act;
  a.status = c.status;
  a.timeout_ns = c.timeout_ns;
  a.mask = 0x000f000fu;
  if (came != nullptr) a.part = reinterpret_cast<float*>(came + 2 * kW4Came);
  W4Args g1 = a, g2 = a;
  g1.K = d;
  g1.S = slabs_of(d);
  g1.n_tiles = F / 8;
  g1.x = rows;
  g1.ldx = w4_pitch(d);
  g1.ldh = w4_pitch(F);
  g1.q = w1_q;
  g1.s = static_cast<const bf16*>(w1_s);
  g1.out = h;
  g1.came = came;
  g2.K = F;
  g2.S = slabs_of(F);
  g2.n_tiles = (d + 15) / 16;
  g2.x = h;
  g2.ldx = w4_pitch(F);
  g2.q = w2_q;
  g2.s = static_cast<const bf16*>(w2_s);
  g2.out = out;
  if (came != nullptr) g2.came = came + kW4Came;
  if (group == 32) return w4_products<32>(c, planes, g1, g2);
  return group == 64 ? w4_products<64>(c, planes, g1, g2) : w4_products<128>(c, planes, g1, g2);
}

}  // namespace moe
