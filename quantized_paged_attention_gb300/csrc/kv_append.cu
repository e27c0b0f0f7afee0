// kv_append_fp8: new keys and values quantised to e4m3 and put into the pages.
//
// A unit is the head vector of one (row, K or V, head): head_dim / 16 threads
// take 16 elements each (32 bytes in, 16 bytes out). Bound: 4 bytes in and 2 out
// per element pair. Measured (GB300), 16384 tokens x 8 heads x 128: 22 us a call on
// fresh inputs, 4.5 TB/s, 17 on the same ones (21 with per-token scales), 18.5 under
// ncu; 5003 tokens x 8 heads x 64 with per-token scales 4.4 us in a graph of 20, 8
// under ncu.
//
// Rounding. The code is the nearest e4m3 value of the exact quotient x / s, a tie
// going to the even code. Midpoints between codes have a significand m of 5 bits
// at most, x has 8. With q = x hi + x lo, hi + lo = 1/s to 2^-40, rounded once (an
// fma takes x hi exactly), a quotient that is a midpoint comes out as that
// midpoint, and one that is 2^-18 of it away or
// more stays on its side. One in between, x = m s (1 - d) with 0 < |d| < 2^-18,
// could end on the wrong side. But all of them have the same d for a given s:
// s (1 - d) = x / m, and two such quotients of 8 and 5 bits are equal or 2^-13
// apart. So hi is moved by 2^-20 towards d's side, once per scale, and the
// conversion needs no test: two packed multiplies and one conversion per pair.
//  * Per tensor, the 16 odd m are tried by 16 lanes: the bf16 nearest to m s
//    tells whether there is such a quotient, and the sign of d.
//  * Per token, s = amax / 448 rounded: if there is one, then d is that rounding,
//    with the sign of 448 s - amax.
// (Converting with 1/s moved down and up, and comparing m s with x where the codes
// differed, took 39 us for 16384 tokens x 8 heads x 128 with per-token scales,
// whose ties are frequent: 448 = 7 * 64, and one significand in 7 divides by 7.)
#include "qpa.h"
#include "common.cuh"
#include "qpa_internal.h"

namespace qpa {

namespace {

constexpr int kThreads = 256;

// The code of x / s by the exact comparison, for any s (s = 0 and NaN follow
// IEEE division); scales per tensor outside (2^-100, 2^100) come here.
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
  float s, hi, lo;         // the scale; hi + lo = 1/s, hi moved past near midpoints
  bool fast;
};

// `side`: the sign of d above, so that x / s lies below (> 0) or above (< 0) its
// near midpoints, or 0: no such quotient, or exact ones
__device__ __forceinline__ Scale make_scale(float s, float side) {
  Scale c;
  c.s = s;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));     // within 2^-23
  const float h = r * (1.f - 2.38418579e-7f);               // 2^-22: below 1/s, so that lo has the sign of hi
  c.lo = fmaf(-s, h, 1.f) * h;                              // (and is not 0: infinity times it stays infinite)
  c.hi = h * (side > 0.f ? 1.f - 9.53674316e-7f : side < 0.f ? 1.f + 9.53674316e-7f : 1.f);
  c.fast = fabsf(s) > 7.8886e-31f && fabsf(s) < 1.2676e30f;   // 2^-100 .. 2^100: nothing above leaves the normals
  return c;
}

// The side of a scale's near midpoints, in every lane of a warp.
__device__ __forceinline__ float side_of(float s, int lane) {
  const float as = fabsf(s), m = (float)(2 * (lane & 15) + 1), v = m * as;
  const float x = __bfloat162float(__float2bfloat16_rn(v));
  const float d = fabsf(v - x) <= v * 3.81469727e-6f ? fmaf(m, as, -x) : 0.f;   // 2^-18 (rounding of v: 2^-24)
  const unsigned below = __ballot_sync(0xffffffffu, d > 0.f), above = __ballot_sync(0xffffffffu, d < 0.f);
  return below ? 1.f : above ? -1.f : 0.f;
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// (a, b) * hi + (a, b) * lo
__device__ __forceinline__ uint32_t quant2(float a, float b, const Scale& c) {
  asm("{ .reg .b64 x, y, z; mov.b64 x, {%0, %1}; mov.b64 y, {%2, %2}; mov.b64 z, {%3, %3}; "
      "mul.rn.f32x2 z, x, z; fma.rn.f32x2 x, x, y, z; mov.b64 {%0, %1}, x; }" : "+f"(a), "+f"(b) : "f"(c.hi), "f"(c.lo));
  return f32x2_to_e4m3x2(a, b);
}

// 4 codes of the bf16 pairs a, b
template <bool FAST>
__device__ __forceinline__ uint32_t quant4(uint32_t a, uint32_t b, const Scale& c) {
  const float x0 = bf_lo(a), x1 = bf_hi(a), x2 = bf_lo(b), x3 = bf_hi(b);
  if (FAST || c.fast) return prmt(quant2(x0, x1, c), quant2(x2, x3, c), 0x5410u);
  return e4m3_exact(x0, c.s) | (e4m3_exact(x1, c.s) << 8) | (e4m3_exact(x2, c.s) << 16) | (e4m3_exact(x3, c.s) << 24);
}

// max(m, |w|) of bf16 pairs, a NaN ignored
__device__ __forceinline__ void amax2(uint32_t& m, uint32_t w) {
  asm("{ .reg .b32 t; abs.bf16x2 t, %1; max.bf16x2 %0, %0, t; }" : "+r"(m) : "r"(w));
}

// amax / 448 rounded to nearest, at least 2^-126 (infinity as the largest bf16)
__device__ __forceinline__ Scale token_scale(float m) {
  m = fminf(m, 3.38953139e38f);
  // 1/448 as two floats; the quotient of 8 bits by 7 is no closer than 1/14 of a
  // unit to where the rounding would turn, and this sum is within 2^-20 units
  float s = fmaf(m, 0.00223214295692741870880126953125f, m * -9.97845626e-11f);
  if (m < 8.2718e-25f) s = fmaxf(__fdiv_rn(m, 448.f), 1.17549435e-38f);    // 2^-80: the second part leaves the normals
  return make_scale(s, s > 1.17549435e-38f ? fmaf(448.f, s, -m) : 0.f);
}

// A token's 2 Hk head vectors take 2 Hk TPR threads (in rounds, if more than the
// block has); a block holds as many tokens side by side as fit. A thread keeps
// its place (K or V, head, 16 dims) and steps through the tokens, UN of them at
// once so that their slots and then their 32 bytes are in flight together. Two
// tokens and 4 blocks per SM, one wave: 16384 tokens x 8 heads x 128 20 us (22.5
// with per-token scales); 5 blocks 26 (24.5), 1 token and 6 blocks 24.5 (24.5), 4
// tokens and 3 blocks 20.4 (22.4).
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
    const float sk = __ldg(p.k_scale), sv = __ldg(p.v_scale);
    fixed_k = make_scale(sk, side_of(sk, threadIdx.x & 31));
    fixed_v = make_scale(sv, side_of(sv, threadIdx.x & 31));
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
          uint32_t m2 = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) amax2(m2, w[j]);
          float m = fmaxf(bf_lo(m2), bf_hi(m2));
#pragma unroll
          for (int o = TPR / 2; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
          c = token_scale(m);
        }
        if (slot[u] < 0) continue;
        uint4 o;
        o.x = quant4<PT>(w[0], w[1], c);
        o.y = quant4<PT>(w[2], w[3], c);
        o.z = quant4<PT>(w[4], w[5], c);
        o.w = quant4<PT>(w[6], w[7], c);
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
