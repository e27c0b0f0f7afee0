// kv_append_nvfp4: new keys and values quantised to NVFP4 (e2m1 codes, an e4m3
// scale per 16 dims) and put into the pages.
//
// A thread takes one scale group: 16 elements (32 bytes in, 8 bytes of codes and
// a scale byte out). Bound: 2 bytes in and 0.5625 out per element.
//
// Rounding, exact as kv_append_fp8's: with q = x hi + x lo, hi + lo = 1/S to 2^-40, a
// quotient that is a midpoint of two codes comes out as that midpoint and one 2^-18 away
// stays on its side. x has 8 bits and a midpoint's significand 3 (e2m1) or 5 (e4m3): for one
// S all quotients within 2^-18 of a midpoint without being one lie on the same side of
// theirs (two such are equal or 2^-11, 2^-13 apart), and hi is moved by 2^-20 to that side.
//  * s = e4m3(a / 6g), a the group's largest |x|: S = 6 g, the same for the whole call.
//  * code = e2m1(x / (s g)): S = s g, held as two floats (28 bits: exact), one of 126 for
//    a call. A block makes the 126 pairs (hi, lo) once, into shared memory, and a group
//    looks its own up. (Made per group: 170 instructions more, ALU-bound, 27 us for 16384
//    tokens x 8 heads x 128 where the table takes 22.)
#include "qpa.h"
#include "common.cuh"
#include "qpa_internal.h"

namespace qpa {

namespace {

constexpr int kThreads = 256;
constexpr float kTiny = 1.2379400392853803e-27f;     // 2^-90
constexpr float kHuge = 1.2379400392853803e+27f;     // 2^90

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// max(m, |w|) of bf16 pairs; a NaN stays
__device__ __forceinline__ void amax2_nan(uint32_t& m, uint32_t w) {
  asm("{ .reg .b32 t; abs.bf16x2 t, %1; max.NaN.bf16x2 %0, %0, t; }" : "+r"(m) : "r"(w));
}

// The e4m3 code nearest to a / (6 g), ties to even, 0x01 .. 0x7E; a >= 0 finite,
// g > 0 finite.
__device__ __forceinline__ uint32_t scale_code(float a, float g) {
  if (g < 1.f) {                                   // keeps tiny products out of the subnormals (exact, or a large code)
    a *= 18446744073709551616.f;
    g *= 18446744073709551616.f;
  } else if (g > 1.2676506002282294e30f) {         // and huge scales within the division's range (2^100)
    a *= 5.421010862427522e-20f;
    g *= 5.421010862427522e-20f;
  }
  const float q = __fdividef(a, g) * 0.16666667163372040f;
  if (!(q < 464.f)) return 0x7eu;                  // 448 and its upper neighbour's midpoint
  // below the smallest normal 2^-6 the codes are 2^-9 apart, as they are in [2^-6, 2^-5)
  const float base = q < 0.015625f ? 0.015625f : 0.f;
  const uint32_t t = __float_as_uint(q + base);
  const float m = __uint_as_float((t & 0xfff00000u) | 0x00080000u) - base;
  const float r = fmaf(-6.f * m, g, a);
  uint32_t c = t >> 20;                            // exponent and 3 mantissa bits
  c += (r > 0.f || (r == 0.f && (c & 1u))) ? 1u : 0u;
  c -= (120u << 3) + (base != 0.f ? 8u : 0u);
  return max(1u, min(c, 0x7eu));
}

// The code of |x| / (s g) by exact comparisons, for scales that the reciprocal
// does not serve.
__device__ __noinline__ uint32_t e2m1_exact(float x, float s, float g) {
  const uint32_t sign = (__float_as_uint(x) >> 28) & 8u;
  float ax = fabsf(x);
  if (g < 1.f) {
    ax *= 18446744073709551616.f;
    g *= 18446744073709551616.f;
  }
  uint32_t c = 0;
#pragma unroll 1
  for (int i = 0; i < 7; ++i) {
    const float mid = i < 4 ? 0.25f + 0.5f * i : i < 6 ? 2.5f + (i - 4) : 5.f;
    const float r = fmaf(-mid * s, g, ax);         // mid s: 3 by 4 bits
    c += (r > 0.f || (r == 0.f && (i & 1))) ? 1u : 0u;
  }
  return c | sign;
}

// 8 bf16 (pairs a, b, c, d) times hi + lo as e2m1 codes, the first in the lowest nibble
__device__ __forceinline__ uint32_t quant8(uint32_t a, uint32_t b, uint32_t c, uint32_t d, float hi, float lo) {
  uint32_t r;
  asm("{ .reg .b64 x, y, z, h, l; .reg .b8 p, q, r, s; .reg .f32 u, v; mov.b64 h, {%9, %9}; mov.b64 l, {%10, %10}; "
      "mov.b64 x, {%1, %2}; mul.rn.f32x2 z, x, l; fma.rn.f32x2 x, x, h, z; mov.b64 {u, v}, x; cvt.rn.satfinite.e2m1x2.f32 p, v, u; "
      "mov.b64 x, {%3, %4}; mul.rn.f32x2 z, x, l; fma.rn.f32x2 x, x, h, z; mov.b64 {u, v}, x; cvt.rn.satfinite.e2m1x2.f32 q, v, u; "
      "mov.b64 x, {%5, %6}; mul.rn.f32x2 z, x, l; fma.rn.f32x2 x, x, h, z; mov.b64 {u, v}, x; cvt.rn.satfinite.e2m1x2.f32 r, v, u; "
      "mov.b64 x, {%7, %8}; mul.rn.f32x2 z, x, l; fma.rn.f32x2 x, x, h, z; mov.b64 {u, v}, x; cvt.rn.satfinite.e2m1x2.f32 s, v, u; "
      "mov.b32 %0, {p, q, r, s}; }"
      : "=r"(r)
      : "f"(bf_lo(a)), "f"(bf_hi(a)), "f"(bf_lo(b)), "f"(bf_hi(b)), "f"(bf_lo(c)), "f"(bf_hi(c)), "f"(bf_lo(d)),
        "f"(bf_hi(d)), "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float e4m3_value(uint32_t c) {       // 0 .. 0x7E
  const uint32_t e = c >> 3, f = c & 7u;
  return e ? __uint_as_float(((e + 120u) << 23) | (f << 20)) : (float)f * 0.001953125f;
}

// hi + lo = 1/(s g), hi moved past the near midpoints of significands 1, 3, .. up to `odd`.
// g in (2^-90, 2^90), s in 2^-9 .. 448.
__device__ __forceinline__ float2 reciprocal(float s, float g, int odd) {
  const float S = s * g, Sl = fmaf(s, g, -S);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(S));       // within 2^-23
  const float h = r * (1.f - 2.38418579e-7f);                 // 2^-22: below 1/S, so that lo has the sign of hi
  const float lo = (fmaf(-S, h, 1.f) - Sl * h) * h;
  float side = 0.f;                                           // the sign of m S - x for the near midpoints
  for (int k = 1; k <= odd; k += 2) {
    const float v = k * S, x = __bfloat162float(__float2bfloat16_rn(v));
    const float d = fmaf(k * s, g, -x);
    side = (fabsf(v - x) <= v * 3.81469727e-6f && d != 0.f) ? d : side;
  }
  return make_float2(h * (side > 0.f ? 1.f - 9.53674316e-7f : side < 0.f ? 1.f + 9.53674316e-7f : 1.f), lo);
}

// A plane's scale: g, its kind, 1/6g
struct Tensor {
  float g;
  bool ok, fast;           // positive and finite; within the reciprocals' range
  float2 sixth;
};

// 16 elements (bf16 pairs w) -> 8 bytes of codes, the scale byte in `sc`
__device__ __forceinline__ uint2 quantise16(const uint32_t (&w)[8], const Tensor& t, const float2* table, uint32_t& sc) {
  uint32_t m2 = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax2_nan(m2, w[j]);
  float a = fmaxf(bf_lo(m2), bf_hi(m2));
  // (a NaN's bits are above infinity's; fmaxf keeps a number beside a NaN)
  const bool nan = max(m2 & 0xffffu, m2 >> 16) > 0x7f80u;
  a = fminf(a, 3.38953139e38f);                    // an infinity counts as the largest bf16
  if (!t.fast) {
    if (nan || !t.ok) {
      sc = 0x7fu;
      return make_uint2(0, 0);
    }
    sc = scale_code(a, t.g);
    const float s = e4m3_value(sc);
    uint32_t o[2];
#pragma unroll 1
    for (int h = 0; h < 2; ++h) {
      uint32_t v = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t x = h ? w[4 + j] : w[j];
        v |= (e2m1_exact(bf_lo(x), s, t.g) | (e2m1_exact(bf_hi(x), s, t.g) << 4)) << (8 * j);
      }
      o[h] = v;
    }
    return make_uint2(o[0], o[1]);
  }
  const float q = fmaf(a, t.sixth.x, a * t.sixth.y);
  sc = max(f32x2_to_e4m3x2(q, 0.f), 1u);
  const float2 r = table[sc];
  if (nan) sc = 0x7fu;
  return nan ? make_uint2(0, 0) : make_uint2(quant8(w[0], w[1], w[2], w[3], r.x, r.y), quant8(w[4], w[5], w[6], w[7], r.x, r.y));
}

// A token's planes * Hk head vectors take TPR threads each (in rounds, if more than
// the block has); a block holds as many tokens side by side as fit. A thread keeps its
// place (plane, head, 16 dims) and steps through the tokens; the next one's elements and the
// slot after that are on their way meanwhile. (16384 tokens x 8 heads x 128: 21.9 us, 26.0 with
// L2 flushed; loaded as two tokens at a time, four blocks per SM, 23.4 and 27.9.)
template <int HD>
__global__ void __launch_bounds__(kThreads, 3) append4_kernel(const Append4Launch p, const int log2_bs, const int side) {
  constexpr int TPR = HD / 16;                 // threads per head vector
  const int Hk = p.num_kv_heads, bs = p.block_size;
  const int tpt = p.planes * Hk * TPR;         // threads per token
  const long long slots = (long long)p.num_blocks * bs;
  const uint32_t chunk = uint32_t(bs) * (HD / 2 + HD / 16), block_bytes = p.planes * Hk * chunk;   // at most 2.4 GB
  const int mine = threadIdx.x / tpt;          // token of the block's side-by-side ones
  const int round = kThreads / TPR * TPR;      // threads of a round (tpt > kThreads: one token)
  const int step = gridDim.x * side;
  __shared__ float2 s_table[2][128];           // [plane][scale code] 1/(s g)
  for (int i = threadIdx.x; i < 128 * p.planes; i += kThreads) {
    const float g = __ldg(i < 128 ? p.k_scale : p.v_scale);
    if ((i & 127) > 0 && (i & 127) < 127 && g > kTiny && g < kHuge) s_table[i >> 7][i & 127] = reciprocal(e4m3_value(i & 127), g, 7);
  }
  __syncthreads();
  for (int i0 = 0; i0 < tpt; i0 += round) {
    const int i = side > 1 ? threadIdx.x - mine * tpt : i0 + threadIdx.x;
    const bool place = side > 1 ? mine < side : i < tpt;
    const int part = i % TPR, vec = i / TPR, kv = vec >= Hk && p.planes > 1, h = vec - kv * Hk;
    const uint16_t* src = static_cast<const uint16_t*>(kv ? p.v : p.k) + h * (kv ? p.v_stride_head : p.k_stride_head) + 16 * part;
    const long long stride = kv ? p.v_stride_tok : p.k_stride_tok;
    uint8_t* const to = p.kv + size_t(kv * Hk + h) * chunk;
    Tensor ten;
    ten.g = __ldg(kv ? p.v_scale : p.k_scale);
    ten.ok = ten.g > 0.f && ten.g < INFINITY;
    ten.fast = ten.g > kTiny && ten.g < kHuge;
    ten.sixth = ten.fast ? reciprocal(6.f, ten.g, 31) : make_float2(0.f, 0.f);
    const float2* table = s_table[kv];
    // whole warps stay in the loop (the scale bytes are shuffled together)
    const uint32_t n = p.num_tokens, ahead = side > 1 ? mine : 0;
    uint32_t t = blockIdx.x * (uint32_t)side + ahead;           // (below 2^31 + 3 steps)
    const uint16_t* from = src + (long long)t * stride;
    const int64_t* slot_of = p.slots + t;
    const long long hop = (long long)step * stride;
    auto get_slot = [&](uint32_t at) -> long long {
      const long long s = place && at < n ? __ldg(slot_of) : -1;
      slot_of += step;
      return s;
    };
    auto load = [&](long long& s, uint4& a, uint4& b) {
      if (s >= slots) {
        atomicExch(&g_kernel_error, (int)KERR_BAD_BLOCK);
        s = -1;
      }
      a = b = make_uint4(0, 0, 0, 0);
      if (s >= 0) {
        a = __ldcs(reinterpret_cast<const uint4*>(from));
        b = __ldcs(reinterpret_cast<const uint4*>(from) + 1);
      }
      from += hop;
    };
    long long s0 = get_slot(t), s1 = get_slot(t + step);
    uint4 a, b;
    load(s0, a, b);
    for (; t - ahead < n; t += step) {
      const long long slot = s0;
      const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      s0 = s1;
      s1 = get_slot(t + 2 * step);
      load(s0, a, b);
      uint32_t sc;
      const uint2 code = quantise16(w, ten, table, sc);
      // the scale bytes of four neighbours as one word
      uint32_t s4 = sc << (8 * (part & 3));
      s4 |= __shfl_xor_sync(0xffffffffu, s4, 1);
      s4 |= __shfl_xor_sync(0xffffffffu, s4, 2);
      if (slot < 0) continue;
      const uint32_t blk = (uint32_t)(slot >> log2_bs), off = (uint32_t)slot & (bs - 1);
      uint8_t* dst = to + (unsigned long long)blk * block_bytes;
      *reinterpret_cast<uint2*>(dst + (off * (HD / 2) + 8 * part)) = code;
      if ((part & 3) == 0) *reinterpret_cast<uint32_t*>(dst + (bs * (HD / 2) + off * (HD / 16) + part)) = s4;
    }
    if (side > 1) break;
  }
}

}  // namespace

cudaError_t launch_append4(const Append4Launch& a, cudaStream_t stream) {
  int log2_bs = 0;
  while ((1 << log2_bs) < a.block_size) ++log2_bs;
  const long long tpt = (long long)a.planes * a.num_kv_heads * (a.head_dim / 16);
  const int side = (int)std::max(1LL, kThreads / tpt);
  const long long want = ((long long)a.num_tokens + side - 1) / side;
  const int grid = (int)std::min(want, (long long)a.num_sms * 3);
  if (a.head_dim == 64) append4_kernel<64><<<grid, kThreads, 0, stream>>>(a, log2_bs, side);
  else append4_kernel<128><<<grid, kThreads, 0, stream>>>(a, log2_bs, side);
  return cudaGetLastError();
}

}  // namespace qpa
