// kv_gather_nvfp4, kv_gather_fp8: tokens read back from the pages as bf16 or float32
// rows.
//
// A block takes a tile of consecutive rows. First its threads find one row each: the
// request by a binary search of query_start, the token's slot through the block table,
// into shared memory. Then a thread keeps its place (plane, head, 8 dims) and steps
// through the tile, UN rows in flight: 4 bytes of e2m1 codes and a scale byte, or 8 e4m3
// codes, to 16 bytes of bf16. Bound: 0.5625 (fp8: 1) bytes in and 2 out per element.
//
// A value is code * group scale (x, at most 6 bits, exact in f16) times a scale g of 24
// bits, rounded once. Rounded to float32 first, a product next to a midpoint of two bf16
// would land on it and then go to the wrong side. For one g all such products lie on the
// same side of theirs: g is m / x times 1 + d, |d| < 2^-24, for a midpoint m of 9 bits, and
// two such quotients are equal or 2^-15 apart. So a g per tensor is moved by one step to
// d's side where there is such an x (13 odd ones tried by as many lanes), and a value
// costs one multiplication. Scales per token keep the lost bits of a truncated product as
// a sticky last bit instead (fp8 pages, 38 k tokens x 8 heads x 128: 47.5 us, 45 with a g per
// tensor). (Sticky bits for all: 7.5 instructions per element, ALU 62 % busy, 52 us for 37 k
// tokens x 8 heads x 128 where this takes 39, 5.0 TB/s; cudaMemset takes 43 us for as many bytes
// as are written.)
#include <type_traits>

#include "qpa.h"
#include "common.cuh"
#include "qpa_internal.h"

namespace qpa {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTile = 64;        // rows of a block
enum : long long { kSkip = -1, kZero = -2 };

// x * g cut to float32, the last bit set if bits were lost and `keep` is 1
__device__ __forceinline__ float mul_sticky(float x, float g, uint32_t keep) {
  const float p = __fmul_rz(x, g);
  return __uint_as_float(__float_as_uint(p) | min(__float_as_uint(fmaf(x, g, -p)), keep));
}
// g such that x * g in float32 rounds to bf16 as the exact product does, for the x of at
// most 6 bits that codes and group scales make; in every lane of a warp.
__device__ __forceinline__ float side_of_midpoints(float g, int lane) {
  // odd parts of (1, 3) by (1, 3, .. 15): 1, 3, .. 15, 21, 27, 33, 39, 45
  const int odd = (lane & 15) < 8 ? 2 * (lane & 7) + 1 : min(21 + 6 * (lane & 7), 45);
  const float x = (float)odd, p = x * g, d = fmaf(x, g, -p);
  const bool on = (__float_as_uint(p) & 0xffffu) == 0x8000u;
  // (relative to g's sign, so that the step is one of g's magnitude)
  const unsigned above = __ballot_sync(0xffffffffu, on && (g > 0.f ? d > 0.f : d < 0.f));
  const unsigned below = __ballot_sync(0xffffffffu, on && (g > 0.f ? d < 0.f : d > 0.f));
  return above ? __uint_as_float(__float_as_uint(g) + 1) : below ? __uint_as_float(__float_as_uint(g) - 1) : g;
}
__device__ __forceinline__ uint32_t mul_bf16x2(float a, float b, float g) {
  uint32_t r;
  asm("{ .reg .b64 x, y; mov.b64 x, {%1, %2}; mov.b64 y, {%3, %3}; mul.rn.f32x2 x, x, y; .reg .f32 u, v; "
      "mov.b64 {u, v}, x; cvt.rn.bf16x2.f32 %0, v, u; }" : "=r"(r) : "f"(a), "f"(b), "f"(g));
  return r;
}

// 8 dims of a token: `lo`, `hi` the code bytes (NVFP4: lo only), `s` the group scale
// byte (NVFP4), `g` the tensor's or token's scale
template <bool FP4>
__device__ __forceinline__ void values8(uint32_t lo, uint32_t hi, uint32_t s, float (&x)[8]) {
  uint32_t h[4];
  if constexpr (FP4) {
    const uint32_t sc = e4m3x2_lo_to_f16x2(s | (s << 8));
    h[0] = hmul2(e2m1x2_to_f16x2<0>(lo), sc);
    h[1] = hmul2(e2m1x2_to_f16x2<1>(lo), sc);
    h[2] = hmul2(e2m1x2_to_f16x2<2>(lo), sc);
    h[3] = hmul2(e2m1x2_to_f16x2<3>(lo), sc);
  } else {
    h[0] = e4m3x2_lo_to_f16x2(lo);
    h[1] = e4m3x2_hi_to_f16x2(lo);
    h[2] = e4m3x2_lo_to_f16x2(hi);
    h[3] = e4m3x2_hi_to_f16x2(hi);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] = f16_lo_to_f32(h[j]);
    x[2 * j + 1] = f16_hi_to_f32(h[j]);
  }
}

// (four blocks per SM: 72 registers and three of them took the fp8 pages' 38 k tokens x 8 heads x 128 from 45 us to 57)
template <bool FP4, int HD, bool F32>
__global__ void __launch_bounds__(kThreads, 4) gather_kernel(const GatherLaunch p, const int log2_bs, const int side,
                                                             const int tile) {
  constexpr int TPR = HD / 8;                  // threads per head vector
  constexpr int UN = 4;
  __shared__ long long s_at[kMaxTile];        // the row's code bytes (of plane 0, head 0) in the cache, or kSkip, kZero
  __shared__ long long s_scale[FP4 ? 1 : kMaxTile];   // its scale of head 0 (per token)
  __shared__ int s_off[kMaxTile];              // its offset in the block
  const int Hk = p.num_kv_heads, bs = p.block_size, R = p.num_reqs;
  constexpr int CB = FP4 ? HD / 2 : HD;        // code bytes of a token and head
  const size_t chunk = size_t(bs) * (FP4 ? HD / 2 + HD / 16 : HD), block_bytes = p.planes * Hk * chunk;
  const long long row0 = (long long)blockIdx.x * tile;
  const int rows = (int)min((long long)tile, p.num_tokens - row0);
  if ((int)threadIdx.x < rows) {
    // the request: the largest r with start[r] <= row (starts clamped to [0, num_tokens])
    const int row = (int)row0 + threadIdx.x;
    auto start = [&](unsigned r) { return max(0, min(__ldg(p.query_start + r), p.num_tokens)); };
    unsigned lo = 0, hi = R + 1u;              // (up to 2^31)
    while (lo < hi) {                          // first entry above row
      const unsigned mid = (lo + hi) >> 1;
      if (start(mid) <= row) lo = mid + 1;
      else hi = mid;
    }
    const int r = (int)lo - 1;
    long long at = kSkip;
    int off = 0;
    if (r >= 0 && r < R) {
      const long long cap = (long long)p.max_blocks * bs;
      const long long L = max(0LL, min((long long)__ldg(p.seq_lens + r), cap));
      const long long t = L - (start(r + 1) - row);
      at = kZero;
      if (t >= 0) {
        int blk = __ldg(p.block_table + r * p.table_stride + (t >> log2_bs));
        if (blk < 0 || blk >= p.num_blocks) {
          atomicExch(&g_kernel_error, (int)KERR_BAD_BLOCK);
          blk = 0;
        }
        off = (int)(t & (bs - 1));
        at = (long long)(blk * block_bytes) + off * CB;
        if (!FP4) s_scale[threadIdx.x] = (long long)blk * Hk * bs + off;
      }
    }
    s_at[threadIdx.x] = at;
    s_off[threadIdx.x] = off;
  }
  float gk = 0.f, gv = 0.f;
  if (!F32 && !p.per_token) {
    gk = side_of_midpoints(__ldg(p.k_scale), threadIdx.x & 31);
    gv = side_of_midpoints(__ldg(p.v_scale), threadIdx.x & 31);
  }
  __syncthreads();
  const int tpt = p.planes * Hk * TPR;         // threads per token
  const int mine = threadIdx.x / tpt;
  for (int i0 = 0; i0 < tpt; i0 += kThreads) {
    const int i = side > 1 ? threadIdx.x - mine * tpt : i0 + threadIdx.x;
    if (side > 1 ? mine >= side : i >= tpt) break;
    const int part = i % TPR, vec = i / TPR, kv = vec >= Hk && p.planes > 1, h = vec - kv * Hk;
    const float* scales = kv ? p.v_scale : p.k_scale;
    const float g0 = p.per_token ? 0.f : F32 ? __ldg(scales) : kv ? gv : gk;
    const size_t esz = F32 ? 4 : 2;
    const uint8_t* in = p.kv + (size_t(kv) * Hk + h) * chunk + part * (FP4 ? 4 : 8);
    const uint32_t to_scale = bs * CB + (part >> 1) - 4 * part;         // (NVFP4, at offset 0)
    const size_t row_bytes = size_t(Hk) * (HD * esz);
    uint8_t* out = static_cast<uint8_t*>(kv ? p.out_v : p.out_k) + (row0 * Hk + h) * (HD * esz) + part * (8 * esz);
    for (int r0 = side > 1 ? mine : 0; r0 < rows; r0 += UN * side) {
      uint32_t lo[UN], hi[UN], sc[UN];
      float g[UN];
      long long at[UN];
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        const int r = r0 + u * side;
        at[u] = r < rows ? s_at[r] : (long long)kSkip;
        lo[u] = hi[u] = sc[u] = 0;
        g[u] = g0;
        if (at[u] >= 0) {
          const uint8_t* src = in + at[u];
          if constexpr (FP4) {
            lo[u] = __ldg(reinterpret_cast<const uint32_t*>(src));
            sc[u] = __ldg(src + to_scale - s_off[r] * (CB - HD / 16));
          } else {
            const uint2 v = __ldg(reinterpret_cast<const uint2*>(src));
            lo[u] = v.x;
            hi[u] = v.y;
            if (p.per_token) {
              g[u] = __ldg(scales + s_scale[r] + (long long)h * bs);
            }
          }
        }
      }
#pragma unroll
      for (int u = 0; u < UN; ++u) {
        if (at[u] == kSkip) continue;
        float x[8];
        values8<FP4>(lo[u], hi[u], sc[u], x);
        if (at[u] < 0) g[u] = 0.f;
        uint8_t* dst = out + size_t(r0 + u * side) * row_bytes;
        if constexpr (F32) {
          reinterpret_cast<float4*>(dst)[0] = make_float4(x[0] * g[u], x[1] * g[u], x[2] * g[u], x[3] * g[u]);
          reinterpret_cast<float4*>(dst)[1] = make_float4(x[4] * g[u], x[5] * g[u], x[6] * g[u], x[7] * g[u]);
        } else {
          uint32_t w[4];
          if (!FP4 && p.per_token) {
            // a small g is taken 2^64 times (a residual would lose its own bits below 2^-149); an infinite one loses no bits, and
            // its residual is NaN
            const bool small = fabsf(g[u]) < 8.67361738e-19f;                  // 2^-60
            const float gs = small ? g[u] * 18446744073709551616.f : g[u], back = small ? 5.42101086e-20f : 1.f;
            const uint32_t keep = fabsf(gs) < INFINITY ? 1u : 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = mul_bf16x2(mul_sticky(x[2 * j], gs, keep), mul_sticky(x[2 * j + 1], gs, keep), back);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = mul_bf16x2(x[2 * j], x[2 * j + 1], g[u]);
          }
          *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    if (side > 1) break;
  }
}

}  // namespace

cudaError_t launch_gather(const GatherLaunch& a, cudaStream_t stream) {
  int log2_bs = 0;
  while ((1 << log2_bs) < a.block_size) ++log2_bs;
  const long long tpt = (long long)a.planes * a.num_kv_heads * (a.head_dim / 8);
  const int side = (int)std::max(1LL, kThreads / tpt);
  // tiles small enough that every SM has a few blocks, large enough to share the search
  const long long per = ((long long)a.num_tokens + 4LL * a.num_sms - 1) / (4LL * a.num_sms);
  const int tile = (int)std::min<long long>(kMaxTile, std::max<long long>(per, side));
  const int grid = (int)(((long long)a.num_tokens + tile - 1) / tile);
  auto launch = [&](auto kernel) { kernel<<<grid, kThreads, 0, stream>>>(a, log2_bs, side, tile); };
  auto by_out = [&](auto f32) {
    constexpr bool F = decltype(f32)::value;
    if (a.fp4) a.head_dim == 64 ? launch(gather_kernel<true, 64, F>) : launch(gather_kernel<true, 128, F>);
    else a.head_dim == 64 ? launch(gather_kernel<false, 64, F>) : launch(gather_kernel<false, 128, F>);
  };
  if (a.out_f32) by_out(std::true_type{});
  else by_out(std::false_type{});
  return cudaGetLastError();
}

}  // namespace qpa
