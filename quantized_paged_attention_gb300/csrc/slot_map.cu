// paged_slot_map: block table, slots, positions and lengths of a step from the
// requests' lengths, in one kernel.
//
// Two exclusive running sums over the requests carry everything: start[r] of
// the new tokens and base[r] of the blocks taken. Token i belongs to the
// request with start[r] <= i < start[r+1], and the k-th id of the free list to
// the request with base[r] <= k < base[r+1]; both are found by a binary search
// in shared memory, so tokens and table entries spread evenly over the
// threads however ragged the requests are. Every CTA makes the two sums itself
// (2 * 4 bytes per request out of L2) instead of waiting for another CTA or a
// first kernel: the call is latency-bound, its bytes are 16 per request, 12
// per token and 8 per taken block.
// A new token's block comes from the free list directly, never through the
// table entry that another CTA may be writing. Replayed back to back it takes 6.3
// us for 256 requests or 103 k tokens alike, 2 us more than the least a kernel
// takes so: the lengths' round trip and the searches.
#include "qpa.h"
#include "common.cuh"
#include "qpa_internal.h"

namespace qpa {

namespace {

constexpr int kThreads = 512;
constexpr uint32_t kSat = 0x7fffffffu;

// a + b for a, b <= INT32_MAX, saturating there (associative)
__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return min(a + b, kSat); }

// the largest r in [0, n) with s[r] <= x (s non-decreasing, s[0] = 0)
__device__ __forceinline__ int find(const uint32_t* s, int n, uint32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kThreads) slot_map_kernel(const SlotMapLaunch p, const int log2_bs) {
  extern __shared__ uint32_t sm[];
  const int B = p.num_reqs;
  uint32_t* start = sm;              // [B + 1]
  uint32_t* base = sm + B + 1;       // [B + 1]
  __shared__ uint32_t warp_tok[kThreads / 32], warp_blk[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int bs = p.block_size;
  auto blocks = [&](uint32_t n) -> uint32_t { return (n + bs - 1) >> log2_bs; };   // n <= INT32_MAX: no wrap

  // ---- the two sums, kThreads requests a round
  uint32_t carry_t = 0, carry_b = 0;
  for (int r0 = 0; r0 < B; r0 += kThreads) {
    const int r = r0 + tid;
    uint32_t n = 0, taken = 0;
    if (r < B) {
      n = (uint32_t)max(0, __ldg(p.new_lens + r));
      const uint32_t c = (uint32_t)max(0, __ldg(p.cached_lens + r));
      const uint32_t len = sat_add(c, n);
      taken = blocks(len) - blocks(c);
      if (blockIdx.x == 0) p.seq_lens[r] = (int)len;
    }
    uint32_t it = n, ib = taken;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t a = __shfl_up_sync(0xffffffffu, it, o), b = __shfl_up_sync(0xffffffffu, ib, o);
      if (lane >= o) {
        it = sat_add(it, a);
        ib = sat_add(ib, b);
      }
    }
    if (lane == 31) {
      warp_tok[warp] = it;
      warp_blk[warp] = ib;
    }
    __syncthreads();
    uint32_t wt = carry_t, wb = carry_b;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) {
        wt = sat_add(wt, warp_tok[w]);
        wb = sat_add(wb, warp_blk[w]);
      }
      carry_t = sat_add(carry_t, warp_tok[w]);
      carry_b = sat_add(carry_b, warp_blk[w]);
    }
    if (r < B) {
      start[r + 1] = sat_add(wt, it);
      base[r + 1] = sat_add(wb, ib);
    }
    __syncthreads();
  }
  if (tid == 0) {
    start[0] = 0;
    base[0] = 0;
  }
  __syncthreads();
  const uint32_t total = carry_t, need = carry_b;
  const uint32_t gtid = blockIdx.x * kThreads + tid, gsize = gridDim.x * kThreads;
  if (blockIdx.x == 0) {
    for (int r = tid; r <= B; r += kThreads) p.query_start[r] = (int)start[r];
    if (tid == 0) *p.num_taken = (int)need;
  }

  int err = KERR_NONE;
  // ---- table entries of the taken blocks
  // (counts up to INT32_MAX, steps below 2^18: 32 unsigned bits hold the sums)
  const uint32_t have = min(need, (uint32_t)p.num_free);
  for (uint32_t k = gtid; k < have; k += gsize) {
    const int r = find(base, B, k);
    const uint32_t e = blocks((uint32_t)max(0, __ldg(p.cached_lens + r))) + (k - base[r]);
    if (e < (uint32_t)p.max_blocks) p.block_table[r * p.table_stride + e] = __ldg(p.free_blocks + k);
    else err = KERR_CAPACITY;
  }
  if (need > (uint32_t)p.num_free) err = KERR_CAPACITY;

  // ---- slots and positions
  for (uint32_t i = gtid; i < (uint32_t)p.max_tokens; i += gsize) {
    long long slot = -1;
    uint32_t pos = 0;
    if (i < total) {
      const int r = find(start, B, i);
      const uint32_t c = (uint32_t)max(0, __ldg(p.cached_lens + r));
      pos = sat_add(c, i - start[r]);
      const uint32_t e = pos >> log2_bs, held = blocks(c);
      int32_t blk = -1;
      bool room = e < (uint32_t)p.max_blocks;
      if (room) {
        if (e < held) {
          blk = p.block_table[r * p.table_stride + e];
        } else {
          const uint32_t k = sat_add(base[r], e - held);
          room = k < (uint32_t)p.num_free;
          if (room) blk = __ldg(p.free_blocks + k);
        }
      }
      if (!room) err = KERR_CAPACITY;
      else if (blk < 0) err = err == KERR_NONE ? (int)KERR_BAD_BLOCK : err;
      else slot = (long long)blk * bs + (pos & (bs - 1));
    }
    p.slots[i] = slot;
    p.positions[i] = (int)pos;
  }
  if (err != KERR_NONE) atomicExch(&g_kernel_error, err);
}

}  // namespace

cudaError_t launch_slot_map(const SlotMapLaunch& a, cudaStream_t stream) {
  int log2_bs = 0;
  while ((1 << log2_bs) < a.block_size) ++log2_bs;
  const size_t smem = 2 * (size_t(a.num_reqs) + 1) * sizeof(uint32_t);
  if (smem > 40 * 1024) {
    constexpr int most = 2 * (kMaxReqs + 1) * sizeof(uint32_t);   // always the same, see kMaxDynamicSmem
    const cudaError_t e = cudaFuncSetAttribute(slot_map_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
  }
  // two tokens a thread; the free list's ids spread over the same threads
  const long long want = ((long long)a.max_tokens + 2 * kThreads - 1) / (2 * kThreads);
  const int grid = (int)std::max(1LL, std::min(want, (long long)a.num_sms));
  slot_map_kernel<<<grid, kThreads, smem, stream>>>(a, log2_bs);
  return cudaGetLastError();
}

}  // namespace qpa
