// pa_decode_nvfp4: attention of one new token per sequence over the 4-bit pages.
//
// One CTA per (sequence, query head); its warps take the tokens in turn, each with
// its own running maximum, sum and output, merged at the end. No tensor core: the
// kernel to compare others with.
#include "qpa.h"
#include "common.cuh"
#include "qpa_internal.h"

namespace qpa {

namespace {

constexpr int kWarps = 4;

__device__ __forceinline__ float e2m1_value(uint32_t c) {
  const float m = (c & 7u) < 2u ? 0.5f * (c & 1u) : __uint_as_float((126u + ((c >> 1) & 3u)) << 23 | (c & 1u) << 22);
  return (c & 8u) ? -m : m;
}

template <int HD>
__global__ void __launch_bounds__(32 * kWarps) decode4_simple_kernel(const Decode4Launch p, const int log2_bs) {
  constexpr int N = HD / 32;                        // dims of a lane
  __shared__ float s_o[kWarps][HD], s_m[kWarps], s_l[kWarps];
  const int Hq = p.num_kv_heads * p.qg, bs = p.block_size;
  const int seq = blockIdx.x / Hq, hq = blockIdx.x % Hq, h = hq / p.qg;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int L = max(0, min(__ldg(p.seq_lens + seq), p.max_blocks * bs));
  const size_t chunk = size_t(bs) * (HD / 2 + HD / 16);
  const uint16_t* qp = static_cast<const uint16_t*>(p.q) + seq * p.q_stride_seq + hq * p.q_stride_head + lane * N;
  float q[N], o[N], m = -INFINITY, l = 0.f;
  const float c = p.softmax_scale * __ldg(p.k_scale);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    q[i] = __uint_as_float(uint32_t(qp[i]) << 16) * c;
    o[i] = 0.f;
  }
  for (int t = warp; t < L; t += kWarps) {
    int blk = __ldg(p.block_table + seq * p.table_stride + (t >> log2_bs));
    if (blk < 0 || blk >= p.num_blocks) {
      if (lane == 0) atomicExch(&g_kernel_error, (int)KERR_BAD_BLOCK);
      blk = 0;
    }
    const int off = t & (bs - 1);
    const uint8_t* kc = p.kv + ((size_t(blk) * 2) * p.num_kv_heads + h) * chunk;
    const uint8_t* vc = kc + p.num_kv_heads * chunk;
    float k[N], v[N];
    const size_t code = size_t(off) * (HD / 2) + lane * (N / 2), sc = size_t(bs) * (HD / 2) + off * (HD / 16) + lane * N / 16;
    const float ks = f16_lo_to_f32(e4m3x2_lo_to_f16x2(kc[sc])), vs = f16_lo_to_f32(e4m3x2_lo_to_f16x2(vc[sc]));
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      k[i] = e2m1_value((kc[code + i / 2] >> (4 * (i & 1))) & 15u) * ks;
      v[i] = e2m1_value((vc[code + i / 2] >> (4 * (i & 1))) & 15u) * vs;
      dot = fmaf(q[i], k[i], dot);
    }
#pragma unroll
    for (int s = 16; s; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
    const float mn = fmaxf(m, dot), alpha = m == -INFINITY ? 0.f : __expf(m - mn), w = __expf(dot - mn);
    l = fmaf(l, alpha, w);
    m = mn;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = fmaf(o[i], alpha, w * v[i]);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) s_o[warp][lane * N + i] = o[i];
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  __syncthreads();
  float M = -INFINITY, den = 0.f;
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
  const float vg = __ldg(p.v_scale);
  for (int d = threadIdx.x; d < HD; d += blockDim.x) {
    float num = 0.f;
    den = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      if (s_l[w] == 0.f) continue;
      const float f = __expf(s_m[w] - M);
      num = fmaf(f, s_o[w][d], num);
      den = fmaf(f, s_l[w], den);
    }
    static_cast<__nv_bfloat16*>(p.out)[(size_t(seq) * Hq + hq) * HD + d] = __float2bfloat16_rn(L > 0 ? num / den * vg : 0.f);
  }
}

}  // namespace

size_t decode4_workspace_bytes(int, int) { return 256; }

cudaError_t launch_decode4(const Decode4Launch& a, cudaStream_t stream) {
  int log2_bs = 0;
  while ((1 << log2_bs) < a.block_size) ++log2_bs;
  const unsigned grid = unsigned((long long)a.num_seqs * a.num_kv_heads * a.qg);
  if (a.head_dim == 64) decode4_simple_kernel<64><<<grid, 32 * kWarps, 0, stream>>>(a, log2_bs);
  else decode4_simple_kernel<128><<<grid, 32 * kWarps, 0, stream>>>(a, log2_bs);
  return cudaGetLastError();
}

}  // namespace qpa
