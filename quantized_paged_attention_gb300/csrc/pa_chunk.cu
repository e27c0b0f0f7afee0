// pa_chunk_fp8: attention of a chunk of new tokens per request over the fp8
// paged cache. One warp per (query row, head): the lanes split head_dim, one
// pass over the visible tokens with the running maximum and sum of a softmax.
#include "qpa.h"
#include "common.cuh"
#include "qpa_internal.h"

namespace qpa {

namespace {

template <int HD>
__global__ void __launch_bounds__(256) chunk_simple_kernel(const ChunkLaunch p, const int log2_bs) {
  constexpr int E = HD / 32;
  const int lane = threadIdx.x & 31;
  const int Hq = p.num_kv_heads * p.qg;
  const long long row = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int t = (int)(row / Hq), hq = (int)(row % Hq);
  if (t >= p.num_tokens) return;
  // the request that owns row t: the last one starting at or before it
  int lo = 0, hi = p.num_reqs;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.query_start[mid] <= t) lo = mid;
    else hi = mid;
  }
  const int q0 = max(0, p.query_start[lo]), q1 = min(p.num_tokens, p.query_start[lo + 1]);
  if (t < q0 || t >= q1) return;
  const int L = max(0, min(p.seq_lens[lo], p.max_blocks << log2_bs));
  const int see = min(L, L - (q1 - q0) + (t - q0) + 1);
  const int h = hq / p.qg, bs = p.block_size;
  const uint16_t* q = static_cast<const uint16_t*>(p.q) + t * p.q_stride_tok + hq * p.q_stride_head + lane * E;
  float qv[E], o[E], m = -INFINITY, l = 0.f;
  const float c = p.softmax_scale * (p.per_token ? 1.f : *p.k_scale);
  for (int e = 0; e < E; ++e) {
    qv[e] = __uint_as_float((uint32_t)q[e] << 16);
    o[e] = 0.f;
  }
  for (int tok = 0; tok < see; ++tok) {
    int b = p.block_table[lo * p.table_stride + (tok >> log2_bs)];
    if (b < 0 || b >= p.num_blocks) {
      if (lane == 0) atomicExch(&g_kernel_error, (int)KERR_BAD_BLOCK);
      b = 0;
    }
    const long long off = tok & (bs - 1);
    const long long kr = ((long long)b * 2 * p.num_kv_heads + h) * bs + off;
    const uint8_t* kp = p.kv + kr * HD + lane * E;
    const uint8_t* vp = kp + (long long)p.num_kv_heads * bs * HD;
    uint32_t kw = 0, vw = 0;
    for (int e = 0; e < E; ++e) {
      kw |= (uint32_t)kp[e] << (8 * e);
      vw |= (uint32_t)vp[e] << (8 * e);
    }
    const uint32_t k2[2] = {e4m3x2_lo_to_f16x2(kw), e4m3x2_hi_to_f16x2(kw)};
    const uint32_t v2[2] = {e4m3x2_lo_to_f16x2(vw), e4m3x2_hi_to_f16x2(vw)};
    float s = 0.f;
    for (int e = 0; e < E; ++e) s = fmaf(qv[e], (e & 1) ? f16_hi_to_f32(k2[e / 2]) : f16_lo_to_f32(k2[e / 2]), s);
    for (int w = 16; w >= 1; w >>= 1) s += __shfl_xor_sync(0xffffffffu, s, w);
    const long long sr = ((long long)b * p.num_kv_heads + h) * bs + off;
    s *= c * (p.per_token ? p.k_scale[sr] : 1.f);
    const float vs = p.per_token ? p.v_scale[sr] : 1.f;
    const float mn = fmaxf(m, s), al = expf(m - mn), w = expf(s - mn);
    m = mn;
    l = l * al + w;
    for (int e = 0; e < E; ++e)
      o[e] = o[e] * al + w * vs * ((e & 1) ? f16_hi_to_f32(v2[e / 2]) : f16_lo_to_f32(v2[e / 2]));
  }
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + row * HD + lane * E;
  const float f = see > 0 ? (p.per_token ? 1.f : *p.v_scale) / l : 0.f;
  for (int e = 0; e < E; ++e) dst[e] = __float2bfloat16(see > 0 ? o[e] * f : 0.f);
}

}  // namespace

size_t chunk_workspace_bytes(int, int, int) { return 256; }

cudaError_t launch_chunk(const ChunkLaunch& a, cudaStream_t stream) {
  int log2_bs = 0;
  while ((1 << log2_bs) < a.block_size) ++log2_bs;
  const long long rows = (long long)a.num_tokens * a.num_kv_heads * a.qg;
  const long long grid = (rows + 7) / 8;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (a.head_dim == 64) chunk_simple_kernel<64><<<(unsigned)grid, 256, 0, stream>>>(a, log2_bs);
  else chunk_simple_kernel<128><<<(unsigned)grid, 256, 0, stream>>>(a, log2_bs);
  return cudaGetLastError();
}

}  // namespace qpa
