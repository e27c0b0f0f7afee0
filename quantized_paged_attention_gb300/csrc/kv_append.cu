// kv_append_fp8: new keys and values quantised to e4m3 and put into the pages.
//
// A unit is the head vector of one (row, K or V, head): head_dim / 16 threads
// take 16 elements each (32 bytes in, 16 bytes out). The call moves
// 4 + 2 bytes per element pair: 16384 tokens x 8 heads x 128 in 22 us, 4.5 TB/s,
// bound half by them and half by the conversions (ALU 55 % busy).
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

// The code of x / s by the exact comparison, for any s (s = 0 and NaN follow
// IEEE division); scales outside [2^-100, 2^100] come here.
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
  float s, inv, lo, hi;   // the scale; 1/s, and 1/s moved down and up past every error of x * (1/s)
  bool fast;
};

__device__ __forceinline__ Scale make_scale(float s) {
  Scale c;
  c.s = s;
  const float a = fabsf(s);
  c.fast = a > 7.8886e-31f && a < 1.2676e30f;   // 2^-100 .. 2^100: neither 1/s nor x/s near 448 leaves the normals
  const float inv = __frcp_rn(s);
  c.inv = inv;
  // a power of two: its reciprocal and the quotient are exact, nothing is ambiguous
  const bool pow2 = (__float_as_uint(s) & 0x007fffffu) == 0u;
  // |fl(x fl(1/s)) / (x/s) - 1| < 2^-22.9; the factors move it by 2^-21
  c.lo = pow2 ? inv : inv * (1.f - 4.76837158e-7f);
  c.hi = pow2 ? inv : inv * (1.f + 4.76837158e-7f);
  return c;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// A value that rounds (in hardware) to the code of x / s: the midpoint of the
// cell that holds |x / s|, moved towards the quotient's side of it, or not at a
// tie. The cell comes from x * (1/s): off by an ulp it can be the neighbour's
// only where the quotient is next to the border between them, and either cell's
// comparison gives that border.
__device__ __forceinline__ float side_of_midpoint(float x, const Scale& c) {
  const float a = fabsf(x * c.inv);
  const float q = a > 480.f ? 480.f : a;             // (NaN stays)
  const float base = q < 0.015625f ? 0.015625f : 0.f;   // subnormal codes: as e4m3_exact
  const float m = __uint_as_float((__float_as_uint(q + base) & 0xfff00000u) | 0x00080000u) - base;
  const float r = fmaf(-m, fabsf(c.s), fabsf(x));
  const float v = r > 0.f ? m * 1.0009765625f : r < 0.f ? m * 0.9990234375f : r == 0.f ? m : r;
  return __uint_as_float((__float_as_uint(v) & 0x7fffffffu) | ((__float_as_uint(x) ^ __float_as_uint(c.s)) & 0x80000000u));
}

// 4 codes of the bf16 pairs a, b
__device__ __forceinline__ uint32_t quant4(uint32_t a, uint32_t b, const Scale& c) {
  const float x0 = bf_lo(a), x1 = bf_hi(a), x2 = bf_lo(b), x3 = bf_hi(b);
  const uint32_t lo = prmt(f32x2_to_e4m3x2(x0 * c.lo, x1 * c.lo), f32x2_to_e4m3x2(x2 * c.lo, x3 * c.lo), 0x5410u);
  const uint32_t hi = prmt(f32x2_to_e4m3x2(x0 * c.hi, x1 * c.hi), f32x2_to_e4m3x2(x2 * c.hi, x3 * c.hi), 0x5410u);
  if (lo == hi && c.fast) return lo;
  // (with per-token scales a vector whose largest element has a multiple of 7 as
  // significand, 448 being 7 * 64, meets a tie in every 16th element)
  if (c.fast)
    return prmt(f32x2_to_e4m3x2(side_of_midpoint(x0, c), side_of_midpoint(x1, c)),
                f32x2_to_e4m3x2(side_of_midpoint(x2, c), side_of_midpoint(x3, c)), 0x5410u);
  return e4m3_exact(x0, c.s) | (e4m3_exact(x1, c.s) << 8) | (e4m3_exact(x2, c.s) << 16) | (e4m3_exact(x3, c.s) << 24);
}

// A token's 2 Hk head vectors take 2 Hk TPR threads (in rounds, if more than the
// block has); a block holds as many tokens side by side as fit. A thread keeps
// its place (K or V, head, 16 dims) and steps through the tokens, UN of them at
// once so that their slots and then their 32 bytes are in flight together. Two
// tokens and 4 blocks per SM, one wave: 16384 tokens x 8 heads x 128 23.5 us (39
// with per-token scales); 4 tokens and 2 blocks 24.5 (43), 6 blocks 31 (43).
template <int HD, bool PT>
__global__ void __launch_bounds__(kThreads, 4) append_kernel(const AppendLaunch p, const int log2_bs, const int side) {
  constexpr int TPR = HD / 16;                 // threads per head vector
  constexpr int UN = 2;
  const int Hk = p.num_kv_heads, bs = p.block_size;
  const int tpt = 2 * Hk * TPR;                // threads per token
  const long long slots = (long long)p.num_blocks * bs;
  const int mine = threadIdx.x / tpt;          // token of the block's side-by-side ones
  const int round = kThreads / TPR * TPR;      // threads of a round (tpt > kThreads: one token)
  Scale fixed_k, fixed_v;
  if constexpr (!PT) {
    fixed_k = make_scale(__ldg(p.k_scale));
    fixed_v = make_scale(__ldg(p.v_scale));
  }
  const int step = gridDim.x * side;
  for (int i0 = 0; i0 < tpt; i0 += round) {
    const int i = side > 1 ? threadIdx.x - mine * tpt : i0 + threadIdx.x;
    const bool place = side > 1 ? mine < side : i < tpt;
    const int part = i % TPR, vec = i / TPR, kv = vec >= Hk, h = vec - kv * Hk;
    const uint16_t* src = static_cast<const uint16_t*>(kv ? p.v : p.k) + h * (kv ? p.v_stride_head : p.k_stride_head);
    const long long stride = kv ? p.v_stride_tok : p.k_stride_tok;
    const Scale fixed = kv ? fixed_v : fixed_k;
    // whole warps stay in the loop (the row maximum is a shuffle)
    for (long long t0 = (long long)blockIdx.x * side; t0 < p.num_tokens; t0 += (long long)UN * step) {
      long long slot[UN];
      uint4 a[UN], b[UN];
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const long long t = t0 + (long long)u * step + (side > 1 ? mine : 0);
        slot[u] = place && t < p.num_tokens ? __ldg(p.slots + t) : -1;
      }
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const long long t = t0 + (long long)u * step + (side > 1 ? mine : 0);
        if (slot[u] >= slots) {
          atomicExch(&g_kernel_error, (int)KERR_BAD_BLOCK);
          slot[u] = -1;
        }
        a[u] = b[u] = make_uint4(0, 0, 0, 0);
        if (slot[u] >= 0) {
          const uint4* s4 = reinterpret_cast<const uint4*>(src + t * stride) + 2 * part;
          a[u] = __ldcs(s4);
          b[u] = __ldcs(s4 + 1);
        }
      }
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const uint32_t w[8] = {a[u].x, a[u].y, a[u].z, a[u].w, b[u].x, b[u].y, b[u].z, b[u].w};
        Scale c = fixed;
        if constexpr (PT) {
          float m = 0.f;                       // fmaxf ignores NaN
#pragma unroll
          for (int j = 0; j < 8; ++j) m = fmaxf(m, fmaxf(fabsf(bf_lo(w[j])), fabsf(bf_hi(w[j]))));
#pragma unroll
          for (int o = TPR / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          c = make_scale(fmaxf(__fdiv_rn(fminf(m, 3.38953139e38f), 448.f), 1.17549435e-38f));
        }
        if (slot[u] < 0) continue;
        uint4 o;
        o.x = quant4(w[0], w[1], c);
        o.y = quant4(w[2], w[3], c);
        o.z = quant4(w[4], w[5], c);
        o.w = quant4(w[6], w[7], c);
        const long long blk = slot[u] >> log2_bs;
        const int off = (int)(slot[u] & (bs - 1));
        reinterpret_cast<uint4*>(p.kv + (((blk * 2 + kv) * Hk + h) * bs + off) * HD)[part] = o;
        if (PT && part == 0) (kv ? p.v_scale : p.k_scale)[(blk * Hk + h) * bs + off] = c.s;
      }
    }
    if (side > 1) break;
  }
}

}  // namespace

cudaError_t launch_append(const AppendLaunch& a, cudaStream_t stream) {
  int log2_bs = 0;
  while ((1 << log2_bs) < a.block_size) ++log2_bs;
  const int tpt = 2 * a.num_kv_heads * (a.head_dim / 16);
  const int side = std::max(1, kThreads / tpt);
  const long long want = ((long long)a.num_tokens + side - 1) / side;
  const int grid = (int)std::min(want, (long long)a.num_sms * 4);
  auto launch = [&](auto kernel) { kernel<<<grid, kThreads, 0, stream>>>(a, log2_bs, side); };
  if (a.head_dim == 64) a.per_token ? launch(append_kernel<64, true>) : launch(append_kernel<64, false>);
  else a.per_token ? launch(append_kernel<128, true>) : launch(append_kernel<128, false>);
  return cudaGetLastError();
}

}  // namespace qpa
