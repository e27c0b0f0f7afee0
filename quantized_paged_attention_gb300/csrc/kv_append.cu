// kv_append_fp8: new keys and values quantised to e4m3 and put into the pages.
//
// A unit is the head vector of one (row, K or V, head): head_dim / 16 threads
// take 16 elements each (32 bytes in, 16 bytes out). The call moves
// 4 + 2 bytes per element pair and is bound by them.
//
// Rounding. The code is the nearest e4m3 value of the exact quotient x / s.
// A float32 quotient rounded again can land on the wrong side of a midpoint
// between two codes, so the midpoint is compared without a quotient: with
// floor cell [f, f + u) of |x / s| and midpoint m = f + u/2 (at most 5
// significant bits), the sign of fma(-m, |s|, |x|) is the exact sign of
// |x| - m |s|: above 0 the code is the upper one, below 0 the lower one, and 0
// is a tie that goes to the even code. The cell comes from the rounded
// quotient; where that rounds up onto a cell's border f the comparison still
// gives f. The common case needs none of this: x times 1/s taken a little too
// small and a little too large rounds (in hardware) to the same code unless a
// midpoint lies between the two, and only then the comparison runs.
#include "qpa.h"
#include "common.cuh"
#include "qpa_internal.h"

namespace qpa {

namespace {

constexpr int kThreads = 256;

// The code of x / s by the exact comparison (any s; s = 0 and NaN follow IEEE
// division).
__device__ __noinline__ uint32_t e4m3_exact(float x, float s) {
  const uint32_t sign = ((__float_as_uint(x) ^ __float_as_uint(s)) >> 24) & 0x80u;
  float ax = fabsf(x), as = fabsf(s);
  const float q = __fdiv_rn(ax, as);
  if (q != q) return 0x7fu;
  if (q >= 464.f) return 0x7eu | sign;          // 448 and its upper neighbour's midpoint: saturates
  // below the smallest normal 2^-6 the codes are 2^-9 apart, as they are in [2^-6, 2^-5)
  const float base = q < 0.015625f ? 0.015625f : 0.f;
  const uint32_t t = __float_as_uint(q + base);
  const float m = __uint_as_float((t & 0xfff00000u) | 0x00080000u) - base;
  if (as < 1.f) {                               // keeps the products of tiny scales out of the subnormals (exact)
    ax *= 18446744073709551616.f;
    as *= 18446744073709551616.f;
  }
  const float r = fmaf(-m, as, ax);
  uint32_t c = t >> 20;                         // exponent and 3 mantissa bits
  c += (r > 0.f || (r == 0.f && (c & 1u))) ? 1u : 0u;
  c -= (120u << 3) + (base != 0.f ? 8u : 0u);
  return min(c, 0x7eu) | sign;
}

struct Scale {
  float s, lo, hi;    // the scale; 1/s rounded down and up past every error of x * (1/s)
  bool fast;
};

__device__ __forceinline__ Scale make_scale(float s) {
  Scale c;
  c.s = s;
  const float a = fabsf(s);
  c.fast = a > 7.8886e-31f && a < 1.2676e30f;   // 2^-100 .. 2^100: neither 1/s nor x/s near 448 leaves the normals
  const float inv = __frcp_rn(s);
  // a power of two: its reciprocal and the quotient are exact, nothing is ambiguous
  const bool pow2 = (__float_as_uint(s) & 0x007fffffu) == 0u;
  // |fl(x fl(1/s)) / (x/s) - 1| < 2^-22.9; the factors move it by 2^-21
  c.lo = pow2 ? inv : inv * (1.f - 4.76837158e-7f);
  c.hi = pow2 ? inv : inv * (1.f + 4.76837158e-7f);
  return c;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 4 codes of the bf16 pairs a, b
__device__ __forceinline__ uint32_t quant4(uint32_t a, uint32_t b, const Scale& c) {
  const float x0 = bf_lo(a), x1 = bf_hi(a), x2 = bf_lo(b), x3 = bf_hi(b);
  const uint32_t lo = prmt(f32x2_to_e4m3x2(x0 * c.lo, x1 * c.lo), f32x2_to_e4m3x2(x2 * c.lo, x3 * c.lo), 0x5410u);
  const uint32_t hi = prmt(f32x2_to_e4m3x2(x0 * c.hi, x1 * c.hi), f32x2_to_e4m3x2(x2 * c.hi, x3 * c.hi), 0x5410u);
  if (lo == hi && c.fast) return lo;
  return e4m3_exact(x0, c.s) | (e4m3_exact(x1, c.s) << 8) | (e4m3_exact(x2, c.s) << 16) | (e4m3_exact(x3, c.s) << 24);
}

template <int HD, bool PT>
__global__ void __launch_bounds__(kThreads) append_kernel(const AppendLaunch p, const int log2_bs) {
  constexpr int TPR = HD / 16;                 // threads per head vector
  const long long gt = (long long)blockIdx.x * kThreads + threadIdx.x;
  const int part = (int)(gt % TPR);
  const long long step = (long long)gridDim.x * kThreads / TPR;
  const int Hk = p.num_kv_heads, bs = p.block_size;
  const long long units = (long long)p.num_tokens * 2 * Hk, slots = (long long)p.num_blocks * bs;
  Scale fixed_k, fixed_v;
  if constexpr (!PT) {
    fixed_k = make_scale(__ldg(p.k_scale));
    fixed_v = make_scale(__ldg(p.v_scale));
  }
  // whole warps stay in the loop (the row maximum is a shuffle); lanes past the end idle
  const long long rounds = (units + step - 1) / step;
  for (long long i = 0; i < rounds; ++i) {
    const long long u = gt / TPR + i * step;
    const bool in = u < units;
    // unit = (row, K or V, head)
    const long long uu = in ? u : 0;
    const long long t = div_nonneg(uu, 2 * Hk);
    const int rem = (int)(uu - t * 2 * Hk), kv = rem >= Hk, h = rem - kv * Hk;
    const long long slot = in ? __ldg(p.slots + t) : -1;
    const bool live = slot >= 0 && slot < slots;
    if (slot >= slots) atomicExch(&g_kernel_error, (int)KERR_BAD_BLOCK);
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (live) {
      const uint16_t* src = static_cast<const uint16_t*>(kv ? p.v : p.k) +
                            t * (kv ? p.v_stride_tok : p.k_stride_tok) + h * (kv ? p.v_stride_head : p.k_stride_head);
      const uint4* s4 = reinterpret_cast<const uint4*>(src) + 2 * part;
      a = __ldg(s4);
      b = __ldg(s4 + 1);
    }
    Scale c = kv ? fixed_v : fixed_k;
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if constexpr (PT) {
      float m = 0.f;                           // fmaxf ignores NaN
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fmaxf(fabsf(bf_lo(w[j])), fabsf(bf_hi(w[j]))));
#pragma unroll
      for (int o = TPR / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      const float s = fmaxf(__fdiv_rn(fminf(m, 3.38953139e38f), 448.f), 1.17549435e-38f);
      c = make_scale(s);
    }
    if (!live) continue;
    uint4 o;
    o.x = quant4(w[0], w[1], c);
    o.y = quant4(w[2], w[3], c);
    o.z = quant4(w[4], w[5], c);
    o.w = quant4(w[6], w[7], c);
    const long long blk = slot >> log2_bs;
    const int off = (int)(slot & (bs - 1));
    uint8_t* dst = p.kv + (((blk * 2 + kv) * Hk + h) * bs + off) * HD;
    reinterpret_cast<uint4*>(dst)[part] = o;
    if (PT && part == 0) (kv ? p.v_scale : p.k_scale)[(blk * Hk + h) * bs + off] = c.s;
  }
}

}  // namespace

cudaError_t launch_append(const AppendLaunch& a, cudaStream_t stream) {
  int log2_bs = 0;
  while ((1 << log2_bs) < a.block_size) ++log2_bs;
  const long long units = (long long)a.num_tokens * 2 * a.num_kv_heads;
  const long long want = (units * (a.head_dim / 16) + kThreads - 1) / kThreads;
  const int grid = (int)std::min(want, (long long)a.num_sms * 8);
  auto launch = [&](auto kernel) { kernel<<<grid, kThreads, 0, stream>>>(a, log2_bs); };
  if (a.head_dim == 64) a.per_token ? launch(append_kernel<64, true>) : launch(append_kernel<64, false>);
  else a.per_token ? launch(append_kernel<128, true>) : launch(append_kernel<128, false>);
  return cudaGetLastError();
}

}  // namespace qpa
