// pa_chunk_fp8: attention of a chunk of new tokens per request over the fp8
// paged cache, on the 5th-generation tensor core.
//
// Mathematics: softmax(scale q k^T + causal) v with one pass over the keys, a
// reference m and a sum l per row: p = 2^(s c - m), O += p v, and O, l are
// rescaled only when the maximum has grown by more than 2^8 since m was taken
// (O / l does not depend on m). m lies 2^7 below the maximum, so that p, up to
// 2^15, uses f16's range: the sum of many small weights is lost only where each is
// below 2^-32 of the largest.
//
//  * Item: 256 query rows of one KV head, i.e. 256 / G whole tokens with their
//    G heads (rows of a group share their keys), as two tiles of 128 rows,
//    walked in key tiles of 128. An item costs a unit per key tile and some to
//    begin; the units of all items (heads, then requests, then tokens) are cut
//    into equal contiguous ranges, one per CTA, whatever the batch looks like. An
//    item that crosses a cut leaves float32 partials (m, l, O / l) in the
//    workspace, and the combine kernel merges them in order (no atomics: the
//    result is the same every time). A CTA needs no plan from memory: the units of
//    a request are a sum of floors of an arithmetic progression, in closed form,
//    so a scan over the requests and one search find its range.
//  * QK: S = Q K^T as kind::f8f6f4. K enters as the cache's e4m3 bytes; a query
//    row, scaled by a power of two to a largest |q| in [128, 256), enters as
//    the sum of 2 e4m3 terms into the same accumulator (8 significant bits:
//    exact for a bf16 of magnitude >= 2^-2, else within 2^-10). Two fp8 passes
//    cost what one bf16 pass does, and K needs no conversion.
//  * PV: O += P V as kind::f16. P goes from the softmax registers to tensor
//    memory (over the S it came from), V is converted e4m3 -> f16 (exact) once
//    per tile by four warps. f16 keeps 11 bits of p, where two e4m3 terms would
//    keep 8 and cost the softmax warps 2.5 instructions per element; the
//    conversion is 0.4.
//  * Per-token V scales: V enters as f16(scale 2^-e) times its codes, and the power of
//    two 2^e goes into P, of which a row keeps a reference of its own: what f16 drops is
//    small against the row's largest p times scale, whatever the tokens' scales are that it
//    does not see or hardly weighs. A key tile has one e where its scales (but those of
//    zeros) lie within 2^7 or so; otherwise each token has its own and the tile takes the long way
//    (apart_tile).
//  * Roles: 2 x 4 softmax warps (a thread owns one row: no exchange between
//    lanes), one per row tile, so that the tensor core works for one while the
//    other computes; 4 warps that convert V and build the next item's query
//    operand; an MMA warp (head_dim 64: two); a warp that walks the schedule and
//    issues the TMA copies (one box per page of the tile, one page per lane); a
//    warp that brings the next items' query rows to L2.
//  * Tokens past the sequence's end are zeroed in V and masked in S; a NaN code
//    in V is taken out of the product, and at the item's end put back into the
//    rows that see its token, so it cannot leak through 0 * NaN.
// Bound: a key tile's products take the tensor core 2048 clocks (head_dim 128),
// the two row tiles' turns come every 3100: per row tile S, the softmax (its
// maximum comes with the load of S from tensor memory, its exponentials take the
// special function unit 512 clocks, twice) and P V follow one another, and only
// the other row tile's chain overlaps them. Tensor memory is full (S and O of
// both), so a third chain does not fit. What per-token scales cost was measured in
// parts: without the K scales' loads (a scale per score, by each of 8 warps) 1.4 to
// 4 %, without multiplying by them and the maximum from registers another 0 to 12 %
// (head_dim 64 over a long context); with head_dim 64 no unit is over 39 % busy, and
// what else holds it back has not been taken apart.
// Measured (GB300), calls in a row, and with pauses between them (the power limit is
// not reached then): 1024 new tokens over 65536, 8 x 4 heads of 128, 776 us, 1.43
// PFLOP/s, 74 % of the measured bf16 rate (711 us), with per-token scales (810 to 824
// us); a prompt of 8192, 8 x 8 heads, 822 us, 1.34 PFLOP/s (784 us; 5 us between
// items); 64 single tokens over 1024..16384 302 us, 3.5 TB/s; head_dim 64, 1024 over
// 65536 (497 us, 1.1 PFLOP/s), with per-token scales (744 us). Between items: the query
// rows' copies 2.5 us, row tile 0's operand 2, its S and softmax 1.
// Tried and slower: both row tiles' pipelines on alternate key tiles of an item
// that has 128 rows at most, and its next S in the idle row tile's buffer (the
// registers cost every other case 10 to 18 % and such items gained nothing: their
// V waits for the conversion); an eighth or a quarter of the exponentials as
// polynomials on the FMA pipe (+7 %, +12 %); P in stores of 16 columns; with
// per-token scales S in the layout where a thread holds a quarter of 4 rows and
// needs a quarter of the scales (+16 %, +33 %: its tensor memory accesses); V of
// an item's first key tile before row tile 1's operand, with that tile's first S
// behind the first product (prompt +8 %, long context +7 %) or before it (+3 %, +1 %).
// Every wait has a time limit; a timeout raises the error word and all roles
// leave through the common teardown.
#define QPA_WHOLE_UNIT
#include "qpa.h"
#include "common.cuh"
#include "qpa_internal.h"
#include "tc.cuh"
#include "chunk_schedule.h"
#include <climits>

namespace qpa {

namespace chunk {
constexpr int ROWS = 256;            // query rows per item (two tiles)
constexpr int MAX_GRID = 160;        // CTAs at most (bounds the workspace)
constexpr int THREADS = 512;
constexpr int W_CONV = 8, W_MMA = 12, W_MMA1 = 13, W_LOAD = 14, W_PREF = 15;
constexpr int NK = 3, NV = 2, NW = 2;   // stages of K, V bytes, V f16
constexpr int NC = 4;                // stages of the per-token scales for the softmax
constexpr int IR = 4;                // item ring
constexpr float kNoMax = -1e30f;     // reference of a row that has seen no token
constexpr float kRoom = 7.f;         // the reference lies so far (log2) below the maximum
constexpr float kLazy = 8.f;         // growth of the maximum (log2) that rescales
constexpr int kSpread = 7;           // V scales of a tile this far apart (log2) share a power of two
constexpr float kFar = 64.f;         // a row's reference so far (log2) above a tile's: P would vanish where p counts

template <int D>
struct Smem {
  static constexpr int qTerm = TILE * D, qBytes = 4 * qTerm;      // [tile][term][128 rows][D]
  static constexpr int kBytes = TILE * D, wBytes = 2 * TILE * D;
  static constexpr int qOff = 0;
  static constexpr int kOff = qOff + qBytes;
  static constexpr int vOff = kOff + NK * kBytes;
  static constexpr int wOff = vOff + NV * kBytes;
  static constexpr int crowOff = wOff + NW * wBytes;              // [2][256] logit multiplier of a row
  static constexpr int krawOff = crowOff + 2 * ROWS * 4;          // [NK][128] per-token scales as copied
  static constexpr int vrawOff = krawOff + NK * TILE * 4;
  static constexpr int kscOff = vrawOff + NV * TILE * 4;          // [NC][128] K scales for the softmax
  static constexpr int vexpOff = kscOff + NC * TILE * 4;          // [NC][128] power of two out of each token's V
  static constexpr int iringOff = vexpOff + NC * TILE * 4;        // [IR] 64 bytes
  static constexpr int qinfoOff = iringOff + IR * 64;             // [2] 64 bytes
  static constexpr int flagOff = qinfoOff + 2 * 64;               // [4 items][4 warps] V holds a NaN
  static constexpr int evOff = flagOff + 64;                      // [NC] the tile's power of two, NaN: the tokens' own
  static constexpr int schedOff = evOff + 4 * NC;                 // schedule scratch
  static constexpr int barOff = schedOff + 256;
  static constexpr int NBAR = 2 * NK + 2 * NV + 2 * NW + NC + 2 * IR + 6 + 2 + 12 + 2 + 2;
  static constexpr int miscOff = barOff + NBAR * 8;
  static constexpr int total = miscOff + 16 + 1024;
  static_assert(schedOff % 16 == 0, "sts_item");
  static_assert(total <= 227 * 1024, "shared memory");
  static_assert(NW == 2 && wBytes == TILE * D * 2, "a V buffer holds a row tile of the result");
};

struct Params {
  const uint16_t* q;
  const int32_t* block_table;
  const int32_t* query_start;
  const int32_t* seq_lens;
  const float* k_scale;
  const float* v_scale;
  __nv_bfloat16* out;
  float* part_o;           // [slots][part_rows][D]
  float2* part_ml;         // [slots][part_rows]
  int4* meta;              // [grid][2]
  long long q_stride_tok, q_stride_head, table_stride;
  int num_reqs, num_tokens, num_kv_heads, qg, log2_bs, num_blocks, max_len, part_rows;
  float softmax_scale;
};

__device__ __forceinline__ Req load_req(const Params& p, int r, int bt) {
  return make_req(__ldg(p.query_start + r), __ldg(p.query_start + r + 1), __ldg(p.seq_lens + r), p.num_tokens, p.max_len, bt);
}

// What the roles need of an item (the part of it in this CTA's range).
struct Item {
  int req, head, tok0, ntok;   // request, KV head, first query row, rows (tokens)
  int lim0, L, t0, t1;         // last key that row tok0 sees, length, key tiles [t0, t1)
  int e0, e1, slot, last;      // end of the key tiles per row tile; partial slot or -1; no more items
};
__device__ __forceinline__ Item lds_item(uint32_t a) {
  const int4 x = lds_i4(a), y = lds_i4(a + 16), z = lds_i4(a + 32);
  return Item{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w, z.x, z.y, z.z, z.w};
}
__device__ __forceinline__ void sts_item(uint32_t a, const Item& i) {
  sts_i4(a, make_int4(i.req, i.head, i.tok0, i.ntok));
  sts_i4(a + 16, make_int4(i.lim0, i.L, i.t0, i.t1));
  sts_i4(a + 32, make_int4(i.e0, i.e1, i.slot, i.last));
}

__device__ __forceinline__ void ffma2(float& a, float& b, float c, float m) {   // (a, b) = (a, b) * c + m
  asm("{ .reg .b64 x, y, z; mov.b64 x, {%0, %1}; mov.b64 y, {%2, %2}; mov.b64 z, {%3, %3}; "
      "fma.rn.f32x2 x, x, y, z; mov.b64 {%0, %1}, x; }" : "+f"(a), "+f"(b) : "f"(c), "f"(m));
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {   // NaN ignored, as fmaxf
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void fadd2(float& a, float& b, float c, float d) {
  asm("{ .reg .b64 x, y; mov.b64 x, {%0, %1}; mov.b64 y, {%2, %3}; add.rn.f32x2 x, x, y; mov.b64 {%0, %1}, x; }"
      : "+f"(a), "+f"(b) : "f"(c), "f"(d));
}
__device__ __forceinline__ void fmul2(float& a, float& b, float c, float d) {
  asm("{ .reg .b64 x, y; mov.b64 x, {%0, %1}; mov.b64 y, {%2, %3}; mul.rn.f32x2 x, x, y; mov.b64 {%0, %1}, x; }"
      : "+f"(a), "+f"(b) : "f"(c), "f"(d));
}
}  // namespace chunk

using namespace chunk;

// A warp's rows against the NaN of V among tokens [a, last): mask gets the dims in
// which a token that the lane's row sees (index at most lim) holds a NaN code,
// all of them where its V scale is not finite. Reads the pages again: about a
// byte per clock and warp, for broken inputs only.
template <int D, bool PT>
__device__ __noinline__ void find_nans(const Params& p, const uint8_t* kv, int req, int head, int a, int last, int lim, int lane,
                                       uint32_t (&mask)[D / 32]) {
  const int bs = 1 << p.log2_bs;
  for (int t = a; t < last; ++t) {
    int blk = __ldg(p.block_table + req * p.table_stride + (t >> p.log2_bs));
    if (blk < 0 || blk >= p.num_blocks) blk = 0;
    const long long off = t & (bs - 1);
    const uint8_t* v = kv + ((((long long)blk * 2 + 1) * p.num_kv_heads + head) * bs + off) * D;
    bool all = false;
    if constexpr (PT)
      all = !(fabsf(__ldg(p.v_scale + ((long long)blk * p.num_kv_heads + head) * bs + off)) < INFINITY);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint32_t w = __ballot_sync(0xffffffffu, all || (__ldg(v + 32 * i + lane) & 0x7f) == 0x7f);
      if (t <= lim) mask[i] |= w;
    }
  }
}

// O of the warp's rows in tensor memory times f (16 columns: the scores hold 128 registers)
template <int D>
__device__ __forceinline__ void rescale_o(uint32_t to, float f) {
#pragma unroll 1
  for (int j = 0; j < D; j += 16) {
    float o[16];
    tmem_ld16(to + j, o);
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] *= f;
    tmem_st16(to + j, reinterpret_cast<const uint32_t*>(o));
  }
}

// A softmax warp's work on a key tile whose V scales are too far apart for one power
// of two, or lie so far below what the row has in O that its weights would vanish
// in P: P with each token's own power of two, l by itself. Small code that loads the
// scores three times, since it may not cost the common tiles registers or room in the
// instruction cache (written out, or with the scores in registers, 4 to 12 %). 1024
// over 65536 with such scales in every tile 3570 us, 816 in none.
struct Apart {
  float c, m, l, x, e;         // m, l and x go in and out
  uint32_t ksc, vexp;          // the tile's K scales and powers of two in shared memory
  uint32_t ts, to, tp;         // S, O and P of the warp's rows in tensor memory
  uint64_t *sfull, *sfree, *pfree, *pfull;   // sfree and pfree null: S is not handed back, P is free
  int sparity, vis;            // keys 0 .. vis of the tile are seen
  bool first;
  int lane;
  volatile int* abort_flag;
};
template <int D>
__device__ __forceinline__ bool apart_tile(Apart& w) {
  if (!warp_wait(w.sfull, w.sparity, w.abort_flag, KERR_TIMEOUT_FULL)) return false;
  tc_fence_after();
  // Three passes over the scores, in one body: the maximum for m, then l and the largest
  // P for x, then P (in place of S where there is no room beside it: its columns lie
  // at or before those of the scores read so far)
  float mx = -INFINITY, g = -INFINITY, l = 0.f;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
#pragma unroll 1
    for (int j = 0; j < TILE; j += 16) {
      float y[16];
      uint32_t pw[8];
      __syncwarp();
      tmem_ld16(w.ts + j, y);
      tmem_wait_ld();
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const float4 ks = lds_f4(w.ksc + 4 * (j + i));
        float4 et = make_float4(w.e, w.e, w.e, w.e);
        if (!(w.e == w.e)) et = lds_f4(w.vexp + 4 * (j + i));
        fmul2(y[i], y[i + 1], ks.x, ks.y);
        fmul2(y[i + 2], y[i + 3], ks.z, ks.w);
        const float ep[4] = {et.x, et.y, et.z, et.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float& p = y[i + u];
          if (j + i + u > w.vis) p = -INFINITY;
          mx = fmaxf(mx, p);
          p = fmaf(p, w.c, -w.m);
          l += ex2(p);
          p += ep[u];
          g = fmaxf(g, p);
          p = ex2(p - w.x);
        }
        pw[i / 2] = f32x2_to_f16x2(y[i], y[i + 1]);
        pw[i / 2 + 1] = f32x2_to_f16x2(y[i + 2], y[i + 3]);
      }
      if (pass == 2) {
        tmem_st8(w.tp + j / 2, pw);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (w.lane == 0) {
          if (j == TILE - 16 && w.sfree) mbar_arrive(w.sfree);
          if ((j & 48) == 48) mbar_arrive(w.pfull + j / 64);
        }
      }
    }
    if (pass == 0) {
      if (fmaf(mx, w.c, -w.m) > kRoom + kLazy) {
        const float mr = fmaxf(floorf(fmaf(mx, w.c, -kRoom)), kNoMax), d = mr - w.m;
        w.l *= ex2(-d);
        w.x -= d;
        w.m = mr;
      }
      g = -INFINITY;
      l = 0.f;
    } else if (pass == 1) {
      w.l += l;
      const float x = g - w.x > kRoom + kLazy ? fmaxf(floorf(g) - kRoom, kNoMax) : w.x;
      if (w.pfree && !warp_wait(w.pfree, w.sparity ^ 1, w.abort_flag, KERR_TIMEOUT_FULL)) return false;
      tc_fence_after();
      __syncwarp();
      if (!w.first && __any_sync(0xffffffffu, x != w.x)) rescale_o<D>(w.to, ex2(w.x - x));
      w.x = x;
    }
  }
  return true;
}

template <int D, bool PT>
__global__ void __launch_bounds__(THREADS, 1)
pa_chunk_kernel(const __grid_constant__ CUtensorMap kv_map, const uint8_t* kv, const __grid_constant__ Params p) {
  using S = Smem<D>;
  constexpr uint32_t SWZ = D == 128 ? kSwizzle128B : kSwizzle64B;
  constexpr uint32_t SBO = 8 * D;                  // 8 rows of D bytes
  // Tensor memory: S of the two row tiles (128 columns each), O (D each). With
  // head_dim 64 there are 128 columns left for P, so the next S is computed
  // while the softmax still works; with 128 P overwrites its S.
  constexpr bool SEP = D == 64;
  // registers per thread: the sum over the four groups is what the block is
  // launched with (4 x 128). Fewer for the softmax than it could use, since the
  // other roles' spills cost more. Measured, softmax/conversion/rest: head_dim 128,
  // 8192-token prompt 168/88/88 794 us, 168/104/72 799, 176/88/72 807, 176/72/88
  // 812 (64 single tokens, which one row tile computes, 318, 318, 300, 304); with
  // per-token scales, 1024 over 65536, 184/64/80 810, 192/64/64 825, 176/80/80 827;
  // head_dim 64, the same 184/88/56 502, 192/72/56 515, with per-token scales
  // 200/56/56 744 (prompts 512), 192/72/56 756 (525), 184/88/56 760 (510).
  constexpr int REG_SOFTMAX = D == 128 ? (PT ? 184 : 168) : (PT ? 200 : 184);
  constexpr int REG_CONV = D == 128 ? (PT ? 64 : 88) : (PT ? 56 : 88);
  constexpr int REG_REST = D == 128 ? (PT ? 80 : 88) : 56;
  static_assert(2 * REG_SOFTMAX + REG_CONV + REG_REST <= 512, "register budget");
  constexpr uint32_t T_O = 256, T_P = SEP ? 384 : 0, P_STEP = SEP ? 64 : 128;
  constexpr uint32_t IDESC_QK = idesc_e4m3(128, 128, false, false);
  constexpr uint32_t IDESC_PV = idesc_f16(128, D, false, true);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;      // swizzle atoms need 1024-byte alignment
  uint8_t* sm = smem_raw + (sb - raw);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + S::barOff);
  uint64_t* kfull = bar;               // [NK] K tile copied
  uint64_t* kempty = kfull + NK;       // [NK] K tile read (both MMA warps; its scales: 4 warps)
  uint64_t* vfull = kempty + NK;       // [NV] V bytes copied
  uint64_t* vempty = vfull + NV;       // [NV] V bytes read (4 warps)
  uint64_t* wfull = vempty + NV;       // [NW] V f16 written (4 warps)
  uint64_t* wempty = wfull + NW;       // [NW] V f16 read (both MMA warps)
  uint64_t* cfull = wempty + NW;       // [NC] scales written (4 warps, per-token scales only)
  uint64_t* ifull = cfull + NC;        // [IR] item published
  uint64_t* iempty = ifull + IR;       // [IR] item read (4 converting warps, prefetch warp)
  uint64_t* qfull = iempty + IR;       // [2] item passed on, row tile 0's query operand built (4 warps)
  uint64_t* qfull1 = qfull + 2;        // [2] row tile 1's query operand built (4 warps)
  uint64_t* qread = qfull1 + 2;        // [2] item read (8 softmax warps, 2 MMA warps)
  uint64_t* qfree = qread + 2;         // [2] a row tile's query operand read (MMA commit)
  uint64_t* sfull = qfree + 2;         // [2] S of a row tile ready (MMA commit)
  uint64_t* sfree = sfull + 2;         // [2] S read (4 warps; SEP)
  uint64_t* pfull = sfree + 2;         // [2][2 halves] P written (4 warps)
  uint64_t* pfree = pfull + 4;         // [2] P read, O complete so far (MMA commit; SEP)
  uint64_t* ofull = pfree + 2;         // [2] O of an item ready (MMA commit)
  uint64_t* done = ofull + 2;          // [2] all MMAs of a row tile finished
  uint64_t* efree = done + 2;          // [2] results of an item out of the V buffers (8 softmax warps); two, since a
                                       // row tile without work in an item may be one item ahead of the other
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + S::miscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + S::miscOff + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NK; ++i) { mbar_init(&kfull[i], 1); mbar_init(&kempty[i], PT ? 6 : 2); }
    for (int i = 0; i < NV; ++i) { mbar_init(&vfull[i], 1); mbar_init(&vempty[i], 4); }
    for (int i = 0; i < NW; ++i) { mbar_init(&wfull[i], 4); mbar_init(&wempty[i], 2); }
    for (int i = 0; i < NC; ++i) mbar_init(&cfull[i], 4);
    for (int i = 0; i < IR; ++i) { mbar_init(&ifull[i], 1); mbar_init(&iempty[i], 5); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&qfull[i], 4);
      mbar_init(&qfull1[i], 4);
      mbar_init(&qread[i], SEP ? 10 : 9);
      mbar_init(&qfree[i], 1);
      mbar_init(&sfull[i], 1);
      mbar_init(&sfree[i], 4);
      mbar_init(&pfull[i], 4);
      mbar_init(&pfull[2 + i], 4);
      mbar_init(&pfree[i], 1);
      mbar_init(&ofull[i], 1);
      mbar_init(&done[i], 1);
      mbar_init(&efree[i], 8);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == W_MMA) tmem_alloc(tmem_slot, 512);
  if (warp == W_LOAD && lane == 0) prefetch_tmap(&kv_map);

  // ---- schedule: this CTA's range [u0, u1) of the units, its first request
  const int bt = ROWS / p.qg;                      // tokens per item
  const uint32_t gm = (65535u + p.qg) / p.qg;      // row / G = row * gm >> 16 for row < 256
  long long* sched = reinterpret_cast<long long*>(sm + S::schedOff);   // [16] warp sums, then the start
  long long W;
  long long u0, u1;
  {
    const int per = (p.num_reqs + THREADS - 1) / THREADS;
    const int r0 = threadIdx.x * per, r1 = min(p.num_reqs, r0 + per);
    long long mine = 0;
    Req only = {0, 0, 0, 0};                       // the thread's request, if it has one
#pragma unroll 1
    for (int r = r0; r < r1; ++r) {
      only = load_req(p, r, bt);
      mine += only.units(bt);
    }
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) sched[warp] = incl;
    __syncthreads();
    W = 0;
    long long base = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) base += sched[w];
      W += sched[w];
    }
    const long long U = W * p.num_kv_heads;
    const int nc = active_ctas(U, gridDim.x), bc = min((int)blockIdx.x, nc);
    u0 = nc ? div_nonneg(U * bc, nc) : 0;
    u1 = nc ? div_nonneg(U * min(bc + 1, nc), nc) : 0;
    if (u0 < u1) {
      long long off = u0 - div_nonneg(u0, W) * W - (base + incl - mine);
      if (off >= 0 && off < mine) {
        int r = r0;
        Req q = only;
        if (per > 1) {
#pragma unroll 1
          while (true) {                           // ends: off lies below this thread's sum
            q = load_req(p, r, bt);
            const long long n = q.units(bt);
            if (off < n || r + 1 >= r1) break;
            off -= n;
            ++r;
          }
        }
        sched[16] = r;
        sched[17] = off;
        sts_i4(sb + S::schedOff + 18 * 8, make_int4(q.q0, q.ql, q.L, q.nt));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < W_CONV) {
    // ======================================================== softmax warps
    reg_inc<REG_SOFTMAX>();
    const int a = warp >> 2;                       // row tile
    const int row = a * TILE + (threadIdx.x & 127);
    const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ts = tl + a * 128, to = tl + T_O + a * D, tp = tl + T_P + a * P_STEP;
    const float vscale = PT ? 1.f : __ldg(p.v_scale);
    const int G = p.qg;
    int sc = 0, oc = 0, n = 0;                     // S tiles, items of this row tile; key tiles of the CTA
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const int qb = k & 1;
      if (!warp_wait(&qfull[qb], (k >> 1) & 1, abort_flag, KERR_TIMEOUT_FULL)) break;
      // (the item is read again for its result: what the key tiles do not need
      // would hold registers through them)
      int t0, end, lim;
      float c;
      {
        const Item it = lds_item(sb + S::qinfoOff + 64 * qb);
        if (a && !warp_wait(&qfull1[qb], (k >> 1) & 1, abort_flag, KERR_TIMEOUT_FULL)) break;
        if (it.last) break;
        c = ldsf(sb + S::crowOff + 4 * (qb * ROWS + row));
        t0 = it.t0;
        end = a ? it.e1 : it.e0;
        // (rows of no token see everything: their scores are 0, and a key tile with
        // masks costs more)
        const int tok = (int)(row * gm >> 16);
        lim = tok < it.ntok ? it.lim0 + tok : INT_MAX;
      }
      float m = kNoMax, l = 0.f;
      // Per-token scales: P holds 2^(s c + e - m - x) with the tile's (or token's) power
      // of two e out of V, x the row's reference of O against m, so that what a row
      // keeps goes by p times the V scale, of the tokens that it sees. m and x are whole
      // numbers: their sums are exact
      float x = kNoMax;
      bool apart = false;                            // (per-token scales) left for a tile that apart_tile takes
      int t = t0;
    tiles:
      for (; t < end; ++t, ++sc) {
        const int nn = n + t - t0, cb = nn % NC;
        float s[4][32], mx4[4];
        float e = 0.f;                               // (per-token scales) the tile's power of two out of V
        // Per-token scales: the keys' scales are loaded while S is awaited, into the
        // registers that S times them takes then (loaded after S: 1024 over 65536 861
        // us, 812 so; head_dim 64, prompts 525, 498)
        if constexpr (PT) {
          if (!warp_wait(&cfull[cb], (nn / NC) & 1, abort_flag, KERR_TIMEOUT_FULL)) { ok = false; break; }
          // (the check stands ahead of S: no scores to keep through the long way)
          e = ldsf(sb + S::evOff + 4 * cb);
          if ((apart = __any_sync(0xffffffffu, !(x - e <= kFar)))) break;   // (NaN too)
#pragma unroll
          for (int i = 0; i < 128; i += 4) {
            const float4 ks = lds_f4(sb + S::kscOff + 4 * (cb * TILE + i));
            s[i / 32][i % 32] = ks.x;
            s[i / 32][i % 32 + 1] = ks.y;
            s[i / 32][i % 32 + 2] = ks.z;
            s[i / 32][i % 32 + 3] = ks.w;
          }
        }
        if (!warp_wait(&sfull[a], sc & 1, abort_flag, KERR_TIMEOUT_FULL)) { ok = false; break; }
        tc_fence_after();
        if constexpr (PT) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float x[32];
            tmem_ld32(ts + 32 * j, x);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; i += 2) fmul2(s[j][i], s[j][i + 1], x[i], x[i + 1]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) tmem_ld32_max(ts + 32 * j, s[j], mx4[j]);
          tmem_wait_ld();
        }
        if constexpr (SEP) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sfree[a]);
        }
        const int vis = lim - t * TILE;            // keys 0 .. vis of the tile are seen
        const bool masked = __any_sync(0xffffffffu, vis < TILE - 1);
        if (masked) {
#pragma unroll
          for (int i = 0; i < 128; ++i) s[i / 32][i % 32] = i <= vis ? s[i / 32][i % 32] : -INFINITY;
        }
        if (PT || masked) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            mx4[j] = fmaxf(s[j][0], s[j][1]);
#pragma unroll
            for (int i = 2; i < 32; i += 2) mx4[j] = fmax3(mx4[j], s[j][i], s[j][i + 1]);
          }
        }
        // The largest exponent comes from the same fma as P's (a rounded s c - m may be off by
        // a step of m, which is more than 1 from 2^24 on), so that P stays in f16's range
        const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3]));
        float nm;                                    // P = 2^(s c + nm)
        if constexpr (PT) {
          nm = e - x - m;
          if (__any_sync(0xffffffffu, t == t0 || fmaf(mx, c, -m) > kRoom + kLazy || fmaf(mx, c, nm) > kRoom + kLazy)) {
            if (fmaf(mx, c, -m) > kRoom + kLazy) {
              const float mr = fmaxf(floorf(fmaf(mx, c, -kRoom)), kNoMax), d = mr - m;
              l *= ex2(-d);
              x -= d;
              m = mr;
            }
            const float g = fmaf(mx, c, -m) + e;     // largest P, but for x
            const bool grow = g - x > kRoom + kLazy;
            if (__any_sync(0xffffffffu, grow)) {
              const float xr = grow ? fmaxf(floorf(g) - kRoom, kNoMax) : x, f = ex2(x - xr);
              x = xr;
              if (t != t0) {
                // (without SEP the S at hand came after the last product)
                if (SEP && !warp_wait(&pfree[a], (sc & 1) ^ 1, abort_flag, KERR_TIMEOUT_FULL)) { ok = false; break; }
                if (SEP) tc_fence_after();
                rescale_o<D>(to, f);
              }
            }
            nm = e - x - m;
          }
        } else {
          const float mr = fmaf(mx, c, -kRoom);
          if (t == t0) {
            m = fmaxf(mr, kNoMax);
          } else {
            const bool grow = fmaf(mx, c, -m) > kRoom + kLazy;
            if (__any_sync(0xffffffffu, grow)) {
              const float al = grow ? ex2(m - mr) : 1.f;
              if (grow) m = mr;
              l *= al;
              if (SEP && !warp_wait(&pfree[a], (sc & 1) ^ 1, abort_flag, KERR_TIMEOUT_FULL)) { ok = false; break; }
              if (SEP) tc_fence_after();
              rescale_o<D>(to, al);
            }
          }
          nm = -m;
        }
        float la[4] = {0.f, 0.f, 0.f, 0.f};
        // P in two halves: the product with the first 64 keys runs while the
        // exponentials of the others are still computed
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t pw[32];
#pragma unroll
          for (int i = 0; i < 64; i += 4) {
            float* y = &s[2 * hf + i / 32][i % 32];
            ffma2(y[0], y[1], c, nm);
            ffma2(y[2], y[3], c, nm);
#pragma unroll
            for (int u = 0; u < 4; ++u) y[u] = ex2(y[u]);
            fadd2(la[0], la[1], y[0], y[1]);
            fadd2(la[2], la[3], y[2], y[3]);
            pw[i / 2] = f32x2_to_f16x2(y[0], y[1]);
            pw[i / 2 + 1] = f32x2_to_f16x2(y[2], y[3]);
          }
          if (SEP && hf == 0 && sc > 0) {            // the last product has read P
            if (!warp_wait(&pfree[a], (sc & 1) ^ 1, abort_flag, KERR_TIMEOUT_FULL)) { ok = false; break; }
            tc_fence_after();
          }
          tmem_st32(tp + 32 * hf, pw);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&pfull[2 * a + hf]);
        }
        if (!ok) break;
        const float sum = (la[0] + la[1]) + (la[2] + la[3]);
        l += PT ? sum * ex2(x - e) : sum;
      }
      if (PT && apart) {
        // (outside the loop, and from a 0 that the compiler does not know: what it
        // prepares for this ahead of the tiles costs them registers)
        apart = false;
        int z;
        asm volatile("mov.u32 %0, 0;" : "=r"(z));
        const int cb = (n + t - t0 + z) % NC;
        const uint32_t sz = sb + 4 * (cb * TILE), tz = tl + z;
        uint64_t* bz = sfull + a + z;
        Apart w{c, m, l, x, ldsf(sb + S::evOff + 4 * cb), sz + S::kscOff, sz + S::vexpOff, tz + a * 128, tz + T_O + a * D,
                tz + T_P + a * P_STEP, bz, SEP ? bz + 2 : nullptr, SEP && sc > 0 ? bz + (pfree - sfull) : nullptr,
                bz + a + (pfull - sfull), sc & 1, lim - t * TILE, t == t0, lane, abort_flag};
        ok = apart_tile<D>(w);
        m = w.m;
        l = w.l;
        x = w.x;
        ++t;
        ++sc;
        if (ok) goto tiles;
      }
      if (!ok) break;
      const Item it = lds_item(sb + S::qinfoOff + 64 * qb);
      __syncwarp();
      if (lane == 0) mbar_arrive(&qread[qb]);
      n += it.t1 - it.t0;
      const int tok = (int)(row * gm >> 16);
      const bool valid = tok < it.ntok;

      // ---- the item's result
      const bool any = it.t0 < end;
      if (any) {
        if (!warp_wait(&ofull[a], oc & 1, abort_flag, KERR_TIMEOUT_FULL)) break;
        ++oc;
        tc_fence_after();
      }
      // The result leaves through the V buffers (a row tile's rows fit one): a
      // lane holds a row, and 32 rows' 16 bytes a store kept the load-store unit
      // from the warps that build the next item's operand (3 us of 5 there). They
      // are free once both row tiles' last products are done, until the first V
      // of the next item, which waits for efree.
      const uint32_t stg = sb + S::wOff + a * S::wBytes + (warp & 3) * 32 * 2 * D;
      const int used = (n + 1 - a) / 2;              // times V buffer a was filled
      if (used > 0 && !warp_wait(&wempty[a], (used - 1) & 1, abort_flag, KERR_TIMEOUT_EMPTY)) break;
      const bool none = lim < 0 || l == 0.f;
      // (per-token scales: 2^(x - 7), in two factors since it may leave the normals)
      const float xh = floorf(0.5f * (x - 7.f)), sv = PT ? ex2(x - 7.f - xh) : vscale;
      const float rl = none ? 0.f : PT ? __frcp_rn(l) * ex2(xh) : __frcp_rn(l);
      float* prow = p.part_o + ((long long)it.slot * p.part_rows + row) * D;
      if (it.slot >= 0 && valid) p.part_ml[(long long)it.slot * p.part_rows + row] = make_float2(none ? -INFINITY : m, l);
      if (any) {
        // NaN codes in the item's V (none, as a rule) were taken out of the
        // products: look for them again and put NaN into the rows that see them
        uint32_t nan[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) nan[i] = 0;
        // (the converting warps' marks, each before its last V of the item)
        if (!warp_wait(&wfull[(n - 1) % NW], ((n - 1) / NW) & 1, abort_flag, KERR_TIMEOUT_FULL)) break;
        const int4 marks = lds_i4(sb + S::flagOff + 16 * (k & 3));
        const bool anynan = (marks.x | marks.y | marks.z | marks.w) != 0;
        // (end * TILE may pass 2^31 - 1 where L does not)
        const int last = (int)min((unsigned)end * TILE, (unsigned)it.L);
        if (anynan) find_nans<D, PT>(p, kv, it.req, it.head, it.t0 * TILE, last, lim, lane, nan);
        // columns at a time: 16 keep the code small (per-token scales, head_dim 128: 931
        // us, 1040 with 32); head_dim 64 has registers for 32 (551 us, 590 with 16)
        constexpr int EC = D == 128 ? 16 : 32;
#pragma unroll 1
        for (int j = 0; j < D / EC; ++j) {
          float o[EC];
          if constexpr (EC == 16) tmem_ld16(to + EC * j, o);
          else tmem_ld32(to + EC * j, o);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < EC; ++i) o[i] = none ? 0.f : o[i] * rl * sv;
          if (anynan) {
            uint32_t w = nan[0];
#pragma unroll
            for (int i = 1; i < D / 32; ++i) w = j * EC / 32 == i ? nan[i] : w;
            w >>= EC * j % 32;
#pragma unroll
            for (int i = 0; i < EC; ++i) o[i] = ((w >> i) & 1u) ? __uint_as_float(0x7fffffffu) : o[i];
          }
          if (it.slot < 0) {
#pragma unroll
            for (int i = 0; i < EC; i += 8) {
              __nv_bfloat162 b0 = __floats2bfloat162_rn(o[i], o[i + 1]), b1 = __floats2bfloat162_rn(o[i + 2], o[i + 3]);
              __nv_bfloat162 b2 = __floats2bfloat162_rn(o[i + 4], o[i + 5]), b3 = __floats2bfloat162_rn(o[i + 6], o[i + 7]);
              sts_i4(stg + lane * (2 * D) + (((EC / 8 * j + i / 8) ^ (lane & 7)) << 4),
                     make_int4(*reinterpret_cast<int*>(&b0), *reinterpret_cast<int*>(&b1), *reinterpret_cast<int*>(&b2),
                               *reinterpret_cast<int*>(&b3)));
            }
          } else if (valid) {
#pragma unroll
            for (int i = 0; i < EC; i += 4) store4(prow + EC * j + i, o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
        }
        if (it.slot < 0) {
          // whole rows out, the warp's 32 of them a few at a time (little unrolled,
          // as all that runs once per item)
          __syncwarp();
          constexpr int CPR = D / 8, RPI = 32 / CPR;
          const int ch = lane % CPR;
#pragma unroll 2
          for (int i = lane / CPR; i < 32; i += RPI) {
            const int r = a * TILE + (warp & 3) * 32 + i, rt = (int)(r * gm >> 16);
            const int4 v = lds_i4(stg + i * (2 * D) + ((ch ^ (i & 7)) << 4));
            if (rt < it.ntok)
              *reinterpret_cast<int4*>(p.out + ((long long)(it.tok0 + rt) * (p.num_kv_heads * G) + it.head * G + r - rt * G) * D +
                                       8 * ch) = v;
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&efree[qb]);
    }
  } else if (warp < W_MMA) {
    // ======================================================== converting warps
    reg_dec<REG_CONV>();
    const int cw = warp - W_CONV;
    const int G = p.qg;
    const float base = p.softmax_scale * (PT ? 1.f : __ldg(p.k_scale)) * kLog2e;
    const uint32_t neg = base < 0.f ? 0x8000u : 0u;
    const uint64_t pol = policy_evict_first();       // a query row is read once
    int n = 0;
    bool ok = true;
    for (int k = 0; ok; ++k) {
      const int qb = k & 1;
      if (!warp_wait(&ifull[k % IR], (k / IR) & 1, abort_flag, KERR_TIMEOUT_FULL)) break;
      const Item it = lds_item(sb + S::iringOff + 64 * (k % IR));
      __syncwarp();
      if (lane == 0) mbar_arrive(&iempty[k % IR]);
      // ---- query operand, in place: 16 dims of a row are 32 bytes of bf16 and 16
      // bytes in each term. A lane copies their halves (cp.async) to where its 16
      // bytes of the first and the second term belong and turns them into those,
      // so a row tile's copies are all in flight at once without a register and
      // no lane meets another's bytes. (Loads through registers, 16 KB in flight,
      // took 10 us per item with the tensor core idle.)
      constexpr int LPR = D / 16, RPW = 32 / LPR, RPS = 4 * RPW, NB = TILE / RPS;   // lanes per row, rows per step, steps
      const int part = lane % LPR;
      const int rows = it.last ? 0 : it.ntok * G;
      auto spot = [&](int a, int b) -> uint32_t {
        const int tr = b * RPS + cw * RPW + lane / LPR;
        return sb + S::qOff + a * 2 * S::qTerm + tr * D + ((part ^ (D == 128 ? (tr & 7) : ((tr >> 1) & 3))) << 4);
      };
      auto fetch = [&](int a) {
#pragma unroll 1
        for (int b = 0; b < NB; ++b) {
          const int row = a * TILE + b * RPS + cw * RPW + lane / LPR;
          const int tok = (int)(row * gm >> 16);
          const bool in = row < rows;
          const uint16_t* src = p.q;
          if (in)
            src += (it.tok0 + tok) * p.q_stride_tok + (long long)(it.head * G + row - tok * G) * p.q_stride_head + 16 * part;
          const uint32_t at = spot(a, b);
          cp_async16_zfill(at, src, in, pol);        // rows past the item's are zero
          cp_async16_zfill(at + S::qTerm, in ? src + 8 : src, in, pol);
        }
        cp_async_commit();
      };
      // (hardly unrolled, nor the copies: they run once per item, out of a cold
      // instruction cache. By 4 the 8192-token prompt took 849 us, by 1 815; later 797
      // by 1 and 785 by 2, two steps' chains at once; with per-token scales, whose
      // budget of registers is smaller, a prompt of 4096 302 by 1 and 332 by 2)
      auto build = [&](int a) {
#pragma unroll (PT ? 1 : 2)
        for (int b = 0; b < NB; ++b) {
          const uint32_t at = spot(a, b);
          const uint4 x0 = lds128(at), x1 = lds128(at + S::qTerm);
          const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
          // largest |q| by its bits (NaN counts as above infinity)
          uint32_t mx = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) asm("max.u16x2 %0, %0, %1;" : "+r"(mx) : "r"(w[i] & 0x7fff7fffu));
          mx = max(mx & 0xffffu, mx >> 16);
#pragma unroll
          for (int o = LPR / 2; o >= 1; o >>= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          // 2^(7 - floor(log2 max)) and its inverse for the logits; rows below
          // 2^-119 keep fewer bits (their logits vanish)
          const uint32_t e = max(mx >> 7, 8u);
          const bool inf = e >= 255;
          if (part == 0) {
            float cm = fabsf(base) * __uint_as_float((inf ? 127u : e - 7) << 23);
            // a masked score must stay -inf when multiplied; a query that is not finite gives a NaN row
            if (cm == 0.f) cm = 1.17549435e-38f;
            if (inf) cm = __uint_as_float(0x7fffffffu);
            stsf(sb + S::crowOff + 4 * (qb * ROWS + a * TILE + b * RPS + cw * RPW + lane / LPR), cm);
          }
          const uint32_t f1 = ((inf ? 127u : 261 - e) << 7) | neg;
          const uint32_t f2 = f1 | (f1 << 16);
          // the scaled value in f16 (exact from 2^-17 up: 8 bits of 11, within
          // 2^-25 below), its e4m3, and the e4m3 of what is left
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t h[2], g[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint32_t y;
              asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(w[2 * j + u]), "r"(f2));
              const uint32_t z = f32x2_to_f16x2(__uint_as_float(y << 16), __uint_as_float(y & 0xffff0000u));
              h[u] = f16x2_to_e4m3x2(z);
              g[u] = f16x2_to_e4m3x2(hsub2(z, e4m3x2_lo_to_f16x2(h[u])));
            }
            hi[j] = prmt(h[0], h[1], 0x5410u);
            lo[j] = prmt(g[0], g[1], 0x5410u);
          }
          sts_i4(at, make_int4(hi[0], hi[1], hi[2], hi[3]));
          sts_i4(at + S::qTerm, make_int4(lo[0], lo[1], lo[2], lo[3]));
        }
      };
      if (k >= 2 && !warp_wait(&qread[qb], ((k >> 1) - 1) & 1, abort_flag, KERR_TIMEOUT_EMPTY)) break;
      if (lane == 0) {
        // (a mark of this warp's own: the warps are not in step)
        asm volatile("st.shared.u32 [%0], %1;" ::"r"(sb + S::flagOff + 16 * (k & 3) + 4 * cw), "r"(0u) : "memory");
        if (cw == 0) sts_item(sb + S::qinfoOff + 64 * qb, it);
      }
      const int na = it.last ? 0 : rows > TILE ? 2 : 1;
#pragma unroll 1
      for (int a = 0; a < 2 && ok; ++a) {
        if (k >= 1 && !warp_wait(&qfree[a], (k - 1) & 1, abort_flag, KERR_TIMEOUT_EMPTY)) { ok = false; break; }
        if (a < na) fetch(a);
      }
      // row tile 0, then 1: the products of 0 start while 1 is built
#pragma unroll 1
      for (int a = 0; a < 2 && ok; ++a) {
        if (a < na) {
          if (a + 1 < na) cp_async_wait<1>();
          else cp_async_wait<0>();
          build(a);
          fence_proxy_async();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(a == 0 ? &qfull[qb] : &qfull1[qb]);
      }
      if (!ok) cp_async_wait_all();
      if (it.last || !ok) break;
      if (k >= 1 && !warp_wait(&efree[qb ^ 1], ((k - 1) >> 1) & 1, abort_flag, KERR_TIMEOUT_EMPTY)) break;

      // ---- V of the item's key tiles: e4m3 -> f16, [dims / 64][token][64 dims],
      // 128-byte swizzle (the MN-major operand of the PV product)
      for (int t = it.t0; t < it.t1; ++t, ++n) {
        const int vb = n % NV, wb = n % NW, cb = n % NC;
        const int live = it.L - t * TILE;            // tokens of the tile that exist
        if (!warp_wait(&vfull[vb], (n / NV) & 1, abort_flag, KERR_TIMEOUT_FULL)) { ok = false; break; }
        float vown = 1.f;
        if constexpr (PT) {
          // scales first, ahead of the wait for room for V: the scores need them.
          // (Room here: the last tile waited for the product three tiles back.)
          const int kb = n % NK;
          if (!warp_wait(&kfull[kb], (n / NK) & 1, abort_flag, KERR_TIMEOUT_FULL)) { ok = false; break; }
          uint32_t ax[4], hi = 0;                    // |scale|, its largest (finite), as bits
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int tk = 32 * i + lane;
            const float x = tk < live ? ldsf(sb + S::vrawOff + 4 * (vb * TILE + tk)) : 0.f;
            ax[i] = __float_as_uint(x) & 0x7fffffffu;
            if (ax[i] >= 0x7f800000u) ax[i] = 0;
            hi = max(hi, ax[i]);
            if (i == cw) vown = x;                   // token 32 cw + lane
          }
          // V enters as f16(v scale 2^(7-e)), below 2^7 (times 448: f16's range) for a
          // power of two 2^e above the scale, which goes into p: one for the tile if none of
          // its scales lies 2^kSpread further below, each token's own otherwise. (Scales up to
          // 2^-126 do not count: a token of zeros has that, and 448 times it is below 2^-117)
          hi = __reduce_max_sync(0xffffffffu, hi);
          auto pow2 = [](uint32_t x) { return max((int)(x >> 23) - 126, -119); };
          int e = pow2(hi);
          const uint32_t low = (uint32_t)(e + 126 - kSpread) << 23;   // 2^(e - 1 - kSpread)
          bool far = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) far = far || ax[i] - 0x00800001u < low - 0x00800001u;
          const bool several = __any_sync(0xffffffffu, far && e > kSpread - 125);
          const int tk = 32 * cw + lane;
          const float kx = tk < live ? ldsf(sb + S::krawOff + 4 * (kb * TILE + tk)) : 0.f;
          stsf(sb + S::kscOff + 4 * (cb * TILE + tk), kx);
          if (cw == 0 && lane == 0) stsf(sb + S::evOff + 4 * cb, several ? __uint_as_float(0x7fffffffu) : (float)e);
          if (several) {
            const uint32_t own = __float_as_uint(vown) & 0x7fffffffu;
            e = pow2(own < 0x7f800000u ? own : 0u);
            stsf(sb + S::vexpOff + 4 * (cb * TILE + tk), (float)e);
          }
          vown *= __uint_as_float((uint32_t)(134 - e) << 23);   // 2^(7 - e)
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&cfull[cb]);
            mbar_arrive(&kempty[kb]);
          }
        }
        if (n >= NW && !warp_wait(&wempty[wb], (n / NW - 1) & 1, abort_flag, KERR_TIMEOUT_EMPTY)) { ok = false; break; }
        constexpr int CPR = D / 16, TPI = 32 / CPR, NI = 32 / TPI;   // 16-byte chunks per token, tokens per step
        const int ch = lane % CPR, tr = lane / CPR;
        const uint32_t src = sb + S::vOff + vb * S::kBytes, dst = sb + S::wOff + wb * S::wBytes;
        // per token: a scale that is not finite makes every dim NaN
        const bool nf = PT && !(fabsf(vown) < INFINITY);
        const uint32_t vs16 = nf ? 0u : f32x2_to_f16x2(vown, vown);
        // a few steps at a time: fewer registers than all at once (per-token scales: 932
        // us for 1024 over 65536 with all 8, 912 with 4; head_dim 64 prompts 512 with 2 of 4,
        // 517 with 1, but without scales 517 with all, 538 with 2)
        constexpr int NH = D == 128 || PT ? 2 : NI;
#pragma unroll 1
        for (int i0 = 0; i0 < NI; i0 += NH) {
          uint32_t bad = 0;
          uint4 x[NH];
#pragma unroll
          for (int i = 0; i < NH; ++i) {
            const int tk = 32 * cw + TPI * (i0 + i) + tr;
            const uint32_t swz = D == 128 ? (tk & 7) : ((tk >> 1) & 3);
            x[i] = lds128(src + tk * D + ((ch ^ swz) << 4));
            if (tk >= live) x[i] = make_uint4(0, 0, 0, 0);
            const uint32_t y = (((x[i].x & 0x7f7f7f7fu) + 0x01010101u) | ((x[i].y & 0x7f7f7f7fu) + 0x01010101u) |
                                ((x[i].z & 0x7f7f7f7fu) + 0x01010101u) | ((x[i].w & 0x7f7f7f7fu) + 0x01010101u)) & 0x80808080u;
            bad |= y;
          }
          const bool anybad = __any_sync(0xffffffffu, bad != 0 || nf);
          if (anybad) {                                // 0 times NaN must not reach a row that does not see the token
#pragma unroll
            for (int i = 0; i < NH; ++i) {
              auto clean = [](uint32_t w) -> uint32_t {
                return w & ~(((((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xffu);
              };
              x[i] = make_uint4(clean(x[i].x), clean(x[i].y), clean(x[i].z), clean(x[i].w));
            }
            if (lane == 0) asm volatile("st.shared.u32 [%0], %1;" ::"r"(sb + S::flagOff + 16 * (k & 3) + 4 * cw), "r"(1u) : "memory");
          }
#pragma unroll
          for (int i = 0; i < NH; ++i) {
            const int tk = 32 * cw + TPI * (i0 + i) + tr;
            const uint32_t rowa = dst + (D == 128 ? (ch >> 2) * (TILE * 128) : 0) + (tk >> 3) * 1024 + (tk & 7) * 128;
            const uint32_t w4[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            uint32_t f[8];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              f[2 * j] = e4m3x2_lo_to_f16x2(w4[j]);
              f[2 * j + 1] = e4m3x2_hi_to_f16x2(w4[j]);
            }
            if constexpr (PT) {
              const uint32_t sc2 = __shfl_sync(0xffffffffu, vs16, TPI * (i0 + i) + tr);
#pragma unroll
              for (int j = 0; j < 8; ++j) f[j] = hmul2(f[j], sc2);
            }
            // the two 16-byte halves in an order that differs between the atoms, so
            // that 8 lanes of a store touch 8 different bank groups
            const bool sw = D == 128 && (ch >> 2);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int ee = sw ? 1 - e : e;
              const uint32_t addr = rowa + ((((ch & 3) * 2 + ee) ^ (tk & 7)) << 4);
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(ee ? f[4] : f[0]), "r"(ee ? f[5] : f[1]),
                           "r"(ee ? f[6] : f[2]), "r"(ee ? f[7] : f[3]) : "memory");
            }
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&wfull[wb]);
          mbar_arrive(&vempty[vb]);
        }
      }
    }
  } else {
    reg_dec<REG_REST>();
    if (warp == W_MMA || (SEP && warp == W_MMA1)) {
      // ====================================================== MMA warps
      // SEP: one per row tile, neither tile's chain (S, softmax, P V) waits for
      // the other's softmax. Otherwise one for both, in strict turns: two warps
      // drift into step there, each tile's products behind the other's and both
      // softmaxes at once (1024 new tokens over 65536: 883 us against 777). The
      // whole warp walks and waits, one elected lane issues.
      constexpr int NA = SEP ? 1 : 2;
      const int a_lo = SEP ? warp - W_MMA : 0;
      int n = 0, pc[2] = {0, 0}, qc[2] = {0, 0};     // key tiles of the CTA, products and S tiles per row tile
      bool ok = true;
      constexpr uint32_t HI = desc_hi(SBO, SWZ), HI_V = desc_hi(1024, kSwizzle128B);
      const uint32_t q_lo = desc_lo(sb + S::qOff, 16), k_lo = desc_lo(sb + S::kOff, 16);
      const uint32_t v_lo = desc_lo(sb + S::wOff, TILE * 128);
      for (int k = 0; ok; ++k) {
        const int qb = k & 1;
        if (!warp_wait(&qfull[qb], (k >> 1) & 1, abort_flag, KERR_TIMEOUT_FULL)) break;
        const Item it = lds_item(sb + S::qinfoOff + 64 * qb);
        __syncwarp();
        if (lane == 0) mbar_arrive(&qread[qb]);
        if (it.last) break;
        // S of key tile t; past the row tile's end its stage is only passed on
        // (after its copy: an earlier arrival would count for the stage's last use)
        auto issue_qk = [&](int a, int t, bool kready) -> bool {
          if (t >= it.t1) return true;
          const int end = a ? it.e1 : it.e0;
          const int nn = n + t - it.t0, kb = nn % NK;
          if (!kready && !warp_wait(&kfull[kb], (nn / NK) & 1, abort_flag, KERR_TIMEOUT_FULL)) return false;
          if (t >= end) {
            if (lane == 0) mbar_arrive(&kempty[kb]);
            return true;
          }
          if (SEP && qc[a] > 0 && !warp_wait(&sfree[a], (qc[a] - 1) & 1, abort_flag, KERR_TIMEOUT_EMPTY)) return false;
          ++qc[a];
          tc_fence_after();
          if (elect_one()) {
            const uint32_t ql = q_lo + a * (2 * S::qTerm / 16), kl = k_lo + kb * (S::kBytes / 16);
            // two query terms into one accumulator
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int i = 0; i < D / 32; ++i)
                mma_e4m3_ss(tmem + a * 128, ql + j * (S::qTerm / 16) + 2 * i, HI, kl + 2 * i, HI, IDESC_QK, j | i);
            umma_commit(&sfull[a]);
            umma_commit(&kempty[kb]);
            if (t + 1 == end) umma_commit(&qfree[a]);
          }
          __syncwarp();
          return true;
        };
#pragma unroll
        for (int i = 0; i < NA; ++i) {
          const int a = SEP ? a_lo : i;
          if (!ok) continue;
          if (a && !warp_wait(&qfull1[qb], (k >> 1) & 1, abort_flag, KERR_TIMEOUT_FULL)) ok = false;
          // a row tile without key tiles here never reads its operand
          if (it.t0 >= (a ? it.e1 : it.e0) && lane == 0) mbar_arrive(&qfree[a]);
          if (ok) ok = issue_qk(a, it.t0, false);
        }
        for (int t = it.t0; t < it.t1 && ok; ++t) {
          const int nn = n + t - it.t0, wb = nn % NW;
#pragma unroll
          for (int i = 0; i < NA; ++i) {
            const int a = SEP ? a_lo : i;
            if (!ok) continue;
            const int end = a ? it.e1 : it.e0;
            // with room for P beside S the next S goes ahead of the product, else
            // behind it (P lies in S)
            if (SEP && !issue_qk(a, t + 1, false)) { ok = false; continue; }
            if ((SEP || a == 0) && !warp_wait(&wfull[wb], (nn / NW) & 1, abort_flag, KERR_TIMEOUT_FULL)) { ok = false; continue; }
            // K of the next tile, before P so that nothing is waited for between
            // the product and the next S
            if (!SEP && a == 0 && t + 1 < it.t1 && !warp_wait(&kfull[(nn + 1) % NK], ((nn + 1) / NK) & 1, abort_flag, KERR_TIMEOUT_FULL)) { ok = false; continue; }
            if (t < end) {
              const uint32_t vl = v_lo + wb * (S::wBytes / 16);
              const uint32_t t_o = tmem + T_O + a * D, t_p = tmem + T_P + a * P_STEP;
#pragma unroll
              for (int hf = 0; hf < 2; ++hf) {
                if (!ok || !warp_wait(&pfull[2 * a + hf], pc[a] & 1, abort_flag, KERR_TIMEOUT_FULL)) { ok = false; continue; }
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                  for (int i = 4 * hf; i < 4 * hf + 4; ++i)
                    mma_f16_ts(t_o, t_p + 8 * i, vl + 128 * i, HI_V, IDESC_PV, i > 0 ? 1u : (uint32_t)(t > it.t0));
                  if (hf) {
                    umma_commit(&wempty[wb]);
                    if (SEP) umma_commit(&pfree[a]);
                    if (t == end - 1) umma_commit(&ofull[a]);
                  }
                }
                __syncwarp();
              }
              ++pc[a];
            } else if (lane == 0) {
              mbar_arrive(&wempty[wb]);
            }
            if (!SEP && ok) ok = issue_qk(a, t + 1, true);
          }
        }
        n += it.t1 - it.t0;
      }
      if (elect_one()) {
        // every issued MMA must finish before the tensor memory is released
        umma_commit(&done[a_lo]);
        if (!mbar_try_wait(&done[a_lo], 0)) {
          const unsigned long long t0 = globaltimer();
          while (!mbar_try_wait(&done[a_lo], 0)) {
            if (globaltimer() - t0 > kWaitLimitNs) {
              atomicExch(&g_kernel_error, (int)KERR_TIMEOUT_FULL);
              break;
            }
          }
        }
      }
      __syncwarp();
    } else if (warp == W_LOAD) {
      // ====================================================== schedule and copies
      const int bs = 1 << p.log2_bs;
      const int bsr = min(bs, TILE);                 // rows of a copy
      const int ppt = TILE / bsr;                    // pages per key tile
      const int Hk = p.num_kv_heads;
      int k = 0, n = 0, kn = 0, vn = 0;              // items, key tiles, K and V copies issued
      bool ok = true;
      long long left = u1 - u0;
      // for the combine: the item that starts here and is cut (head, row, tokens,
      // slot); whether the first item began earlier, whether it ends here, no items
      int4 m_start = make_int4(0, 0, 0, -1), m_cont = make_int4(0, 0, 1, 0);
      int h = 0, r = 0, j = 0;
      long long o = 0;                               // units of item j that lie before the range
      Req rq = {0, 0, 0, 0};
      if (left > 0) {
        h = (int)div_nonneg(u0, W);
        r = (int)sched[16];
        const long long off = sched[17];
        const int4 q = lds_i4(sb + S::schedOff + 18 * 8);
        rq = Req{q.x, q.y, q.z, q.w};
        int lo = 0, hi = rq.nt;                      // the item that holds unit off of the request
        while (hi - lo > 1) {
          const int probe = Req::split(lo, hi, lane);
          const int below = __popc(__ballot_sync(0xffffffffu, rq.before(probe, bt) <= off));
          const int l = __shfl_sync(0xffffffffu, probe, max(below - 1, 0)), h2 = __shfl_sync(0xffffffffu, probe, below & 31);
          lo = below > 0 ? l : lo;
          hi = below < 32 ? h2 : hi;
        }
        j = lo;
        o = off - rq.before(j, bt);
      }
      while (ok) {
        Item it;
        it.last = left <= 0;
        if (!it.last) {
          const int nk = rq.tiles(j, bt);
          const long long take = min(left, (long long)nk + ITEM_COST - o);
          it.req = r;
          it.head = h;
          it.tok0 = rq.q0 + j * bt;
          it.ntok = min(bt, rq.ql - j * bt);
          it.lim0 = rq.L - rq.ql + j * bt;
          it.L = rq.L;
          it.t0 = Req::tile_at(o);
          it.t1 = Req::tile_at(o + take);
          const int rows = it.ntok * p.qg;
          const int n0 = max(it.lim0 + (min(rows, TILE) - 1) / p.qg, 0) / TILE + 1;
          it.e0 = min(it.t1, n0);
          it.e1 = rows > TILE ? it.t1 : it.t0;
          const bool starts = it.t0 == 0, ends = it.t1 == nk;
          // slot 2 b: the CTA's first item, slot 2 b + 1: its last (if another)
          it.slot = starts && ends ? -1 : 2 * (int)blockIdx.x + (k > 0);
          left -= take;
          // ---- the next item: token range, request, head
          o = 0;
          if (left > 0 && ++j >= rq.nt) {
            j = 0;
            do {                                     // left > 0: a request with units follows
              if (++r >= p.num_reqs) {
                r = 0;
                ++h;
              }
              rq = load_req(p, r, bt);
            } while (rq.nt == 0 && h < Hk);
            if (h >= Hk) left = 0;                   // (not reached while the inputs stay as they were)
          }
          if (it.t0 == it.t1) continue;              // cut before its first key tile: the next CTA's
          if (starts && !ends) m_start = make_int4(it.head, it.tok0, it.ntok, it.slot);
          if (!starts) m_cont = make_int4(1, ends, 0, 0);
          m_cont.z = 0;
        }
        if (k >= IR && !warp_wait(&iempty[k % IR], (k / IR - 1) & 1, abort_flag, KERR_TIMEOUT_EMPTY)) break;
        if (lane == 0) {
          sts_item(sb + S::iringOff + 64 * (k % IR), it);
          mbar_arrive(&ifull[k % IR]);
        }
        if (it.last) break;
        ++k;

        const int32_t* tab = p.block_table + it.req * p.table_stride;
        const int npages = (it.L + bs - 1) >> p.log2_bs;
        // the item's block ids, 32 at a time and the next 32 in flight
        int win = (it.t0 * TILE) >> p.log2_bs;
        auto entry = [&](int e) -> int { return e < npages ? __ldg(tab + e) : 0; };
        int cur = entry(win + lane), nxt = entry(win + 32 + lane);
        for (int t = it.t0; t < it.t1; ++t, ++n) {
          const int kb = n % NK, vb = n % NV;
          const int e0 = (t * TILE) >> p.log2_bs;    // first page of the tile
          if (e0 >= win + 32) {
            cur = nxt;
            win += 32;
            nxt = entry(win + 32 + lane);
          }
          const int np = max(0, min(ppt, npages - e0));
          int blk = __shfl_sync(0xffffffffu, cur, (e0 - win + lane) & 31);
          if (lane < np && (blk < 0 || blk >= p.num_blocks)) {
            atomicExch(&g_kernel_error, (int)KERR_BAD_BLOCK);
            blk = 0;
          }
          const int y0 = bs > TILE ? (t & 1) * TILE : 0;   // 256-token pages: half a page
          const uint32_t pb = bsr * D, tx = np * (pb + (PT ? bsr * 4 : 0));
          if (n >= NK && !warp_wait(&kempty[kb], (n / NK - 1) & 1, abort_flag, KERR_TIMEOUT_EMPTY)) { ok = false; break; }
          if (lane == 0) {
            if (np) mbar_arrive_expect_tx(&kfull[kb], tx);
            else mbar_arrive(&kfull[kb]);
          }
          __syncwarp();
          if (lane < np) {
            tma_load_3d(sb + S::kOff + kb * S::kBytes + lane * pb, &kv_map, 0, it.head * bs + y0, blk, &kfull[kb]);
            if constexpr (PT)
              bulk_load(sb + S::krawOff + 4 * (kb * TILE + lane * bsr), p.k_scale + ((long long)blk * Hk + it.head) * bs + y0,
                        bsr * 4, &kfull[kb]);
          }
          kn = n + 1;
          if (n >= NV && !warp_wait(&vempty[vb], (n / NV - 1) & 1, abort_flag, KERR_TIMEOUT_EMPTY)) { ok = false; break; }
          if (lane == 0) {
            if (np) mbar_arrive_expect_tx(&vfull[vb], tx);
            else mbar_arrive(&vfull[vb]);
          }
          __syncwarp();
          if (lane < np) {
            tma_load_3d(sb + S::vOff + vb * S::kBytes + lane * pb, &kv_map, 0, (Hk + it.head) * bs + y0, blk, &vfull[vb]);
            if constexpr (PT)
              bulk_load(sb + S::vrawOff + 4 * (vb * TILE + lane * bsr), p.v_scale + ((long long)blk * Hk + it.head) * bs + y0,
                        bsr * 4, &vfull[vb]);
          }
          vn = n + 1;
        }
        if (!ok) break;
      }
      if (lane == 0) {
        p.meta[2 * blockIdx.x] = m_start;
        p.meta[2 * blockIdx.x + 1] = m_cont;
      }
      // the copies in flight must land before the CTA exits (only after an abort
      // are there any)
      if (*abort_flag && lane == 0) {
        const unsigned long long t0 = globaltimer();
        for (int i = max(0, kn - NK); i < kn; ++i)
          while (!mbar_try_wait(&kfull[i % NK], (i / NK) & 1) && globaltimer() - t0 < kWaitLimitNs) {}
        for (int i = max(0, vn - NV); i < vn; ++i)
          while (!mbar_try_wait(&vfull[i % NV], (i / NV) & 1) && globaltimer() - t0 < kWaitLimitNs) {}
      }
      __syncwarp();
    } else if (warp == W_PREF) {
      // ====================================================== query rows to L2
      // An item is published some key tiles before its query operand is built;
      // from DRAM the 64 KB of rows, 16 KB in flight, took 10 us, all of it with
      // the tensor core idle.
      for (int k = 0;; ++k) {
        if (!warp_wait(&ifull[k % IR], (k / IR) & 1, abort_flag, KERR_TIMEOUT_FULL)) break;
        const Item it = lds_item(sb + S::iringOff + 64 * (k % IR));
        __syncwarp();
        if (lane == 0) mbar_arrive(&iempty[k % IR]);
        if (it.last) break;
        constexpr int LPR = D / 64;                  // 128-byte lines per row (16-byte aligned rows may touch one more)
        const int rows = it.ntok * p.qg;
        for (int i = lane; i < rows * LPR; i += 32) {
          const int row = i / LPR, tok = (int)(row * gm >> 16);
          const uint16_t* src = p.q + (it.tok0 + tok) * p.q_stride_tok +
                                (long long)(it.head * p.qg + row - tok * p.qg) * p.q_stride_head + (i % LPR) * 64;
          asm volatile("prefetch.global.L2 [%0];" ::"l"(src));
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == W_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Merge of the items that cross a cut: block (c, y) looks at the item that
// starts in CTA c and does not end there, rows 32 y .. 32 y + 31. Its pieces are
// the starting CTA's last slot and the first slots of the CTAs behind it, found
// at once by a vote over all of them (following them one load after the other
// took 15 us where 38 CTAs shared a short request).
template <int D>
__global__ void __launch_bounds__(256) chunk_combine_kernel(const Params p, const int grid) {
  const int c = blockIdx.x;
  const int4 ms = p.meta[2 * c];
  if (ms.w < 0) return;
  __shared__ int slots[MAX_GRID + 4];
  __shared__ int stop, count;
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid == 0) stop = grid;
  __syncthreads();
  const int d = c + 1 + tid;
  int4 mc = make_int4(0, 0, 1, 0);
  if (d < grid) mc = p.meta[2 * d + 1];
  // the walk ends at the first CTA that has items and does not continue this one
  // (not part of it) or ends it (the last part); CTAs without items are passed
  if (d < grid && !mc.z && (!mc.x || mc.y)) atomicMin(&stop, d);
  __syncthreads();
  const bool mine = d < grid && !mc.z && mc.x && d <= stop;
  __shared__ unsigned votes[8];
  const unsigned vote = __ballot_sync(0xffffffffu, mine);
  if (lane == 0) votes[tid >> 5] = vote;
  __syncthreads();
  if (mine) {
    int at = 1 + __popc(vote & ((1u << lane) - 1u));
    for (int w = 0; w < (tid >> 5); ++w) at += __popc(votes[w]);
    slots[at] = 2 * d;
  }
  if (tid == 0) {
    slots[0] = ms.w;
    int n = 1;
    for (int w = 0; w < 8; ++w) n += __popc(votes[w]);
    count = n;
  }
  __syncthreads();
  constexpr int TPR = D / 4, RPB = 256 / TPR;        // threads per row (4 dims each), rows per pass
  const int col = tid % TPR, n = count;
  const int rows = ms.z * p.qg;
  for (int row = blockIdx.y * 32 + tid / TPR; row < min(rows, (int)blockIdx.y * 32 + 32); row += RPB) {
    float M = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int i = 0; i < n; i += 4) {                 // four pieces' loads at once
      float2 ml[4];
      float4 x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        ml[u] = make_float2(-INFINITY, 0.f);
        if (i + u < n) {
          const long long at = (long long)slots[i + u] * p.part_rows + row;
          ml[u] = p.part_ml[at];
          x[u] = *reinterpret_cast<const float4*>(p.part_o + at * D + 4 * col);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        // the row saw no key of it (l is not 0 but NaN then if the query is not finite)
        if (ml[u].x == -INFINITY) continue;
        const float mn = fmaxf(M, ml[u].x);
        const float a0 = ex2(M - mn), w = ml[u].y * ex2(ml[u].x - mn);
        M = mn;
        l = l * a0 + w;
        o[0] = o[0] * a0 + w * x[u].x;
        o[1] = o[1] * a0 + w * x[u].y;
        o[2] = o[2] * a0 + w * x[u].z;
        o[3] = o[3] * a0 + w * x[u].w;
      }
    }
    const float rl = l == 0.f ? 0.f : 1.f / l;
    const int tok = row / p.qg;
    __nv_bfloat16* dst = p.out + ((long long)(ms.y + tok) * (p.num_kv_heads * p.qg) + ms.x * p.qg + row - tok * p.qg) * D;
    store4(dst + 4 * col, o[0] * rl, o[1] * rl, o[2] * rl, o[3] * rl);
  }
}

namespace {
struct Layout {
  size_t ml, meta, total;
  int rows;
};
Layout chunk_layout(int num_tokens, int qg, int D) {
  Layout L;
  L.rows = (int)std::min<long long>(ROWS, (long long)num_tokens * qg);
  const size_t slots = 2 * MAX_GRID;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  L.ml = up(slots * L.rows * D * sizeof(float));
  L.meta = L.ml + up(slots * L.rows * sizeof(float2));
  L.total = L.meta + up(slots * sizeof(int4));
  return L;
}
}  // namespace

cudaError_t take_chunk_error(int* v) {
  const int z = 0;
  const cudaError_t e = cudaMemcpyFromSymbol(v, g_kernel_error, sizeof(int));
  return e == cudaSuccess && *v ? cudaMemcpyToSymbol(g_kernel_error, &z, sizeof(int)) : e;
}

size_t chunk_workspace_bytes(int num_tokens, int query_group, int head_dim) {
  return chunk_layout(num_tokens, query_group, head_dim).total;
}

cudaError_t launch_chunk(const ChunkLaunch& a, cudaStream_t stream) {
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return cudaErrorNotSupported;
  const int D = a.head_dim, bs = a.block_size;
  // (ahead of the tensor map, whose encoding needs a context that is current in this
  // host thread: the runtime's first call in a thread makes it so)
  auto kernel = D == 64 ? (a.per_token ? pa_chunk_kernel<64, true> : pa_chunk_kernel<64, false>)
                        : (a.per_token ? pa_chunk_kernel<128, true> : pa_chunk_kernel<128, false>);
  const int smem = D == 64 ? Smem<64>::total : Smem<128>::total;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  CUtensorMap map;
  const cuuint64_t page_rows = (cuuint64_t)2 * a.num_kv_heads * bs;
  const cuuint64_t dims[3] = {(cuuint64_t)D, page_rows, (cuuint64_t)a.num_blocks};
  const cuuint64_t strides[2] = {(cuuint64_t)D, page_rows * D};
  const cuuint32_t box[3] = {(cuuint32_t)D, (cuuint32_t)std::min(bs, TILE), 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  if (enc(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(a.kv), dims, strides, box, estr,
          CU_TENSOR_MAP_INTERLEAVE_NONE, D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  const Layout L = chunk_layout(a.num_tokens, a.qg, D);
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  Params p;
  p.q = static_cast<const uint16_t*>(a.q);
  p.block_table = a.block_table;
  p.query_start = a.query_start;
  p.seq_lens = a.seq_lens;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.out = static_cast<__nv_bfloat16*>(a.out);
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + L.ml);
  p.meta = reinterpret_cast<int4*>(ws + L.meta);
  p.q_stride_tok = a.q_stride_tok;
  p.q_stride_head = a.q_stride_head;
  p.table_stride = a.table_stride;
  p.num_reqs = a.num_reqs;
  p.num_tokens = a.num_tokens;
  p.num_kv_heads = a.num_kv_heads;
  p.qg = a.qg;
  p.log2_bs = 0;
  while ((1 << p.log2_bs) < bs) ++p.log2_bs;
  p.num_blocks = a.num_blocks;
  p.max_len = a.max_blocks * bs;
  p.part_rows = L.rows;
  p.softmax_scale = a.softmax_scale;
  // no more CTAs than the most units that these sizes can have would employ
  const int bt = ROWS / a.qg;
  const long long items = (long long)a.num_tokens / bt + std::min(a.num_reqs, a.num_tokens);
  const long long most = std::min(items * a.num_kv_heads, 1LL << 20) * ((p.max_len - 1) / TILE + 1 + ITEM_COST);
  const int grid = active_ctas(most, std::min(a.num_sms, MAX_GRID));
  kernel<<<grid, THREADS, smem, stream>>>(map, a.kv, p);
  const dim3 cg(grid, (L.rows + 31) / 32);
  if (D == 64) chunk_combine_kernel<64><<<cg, 256, 0, stream>>>(p, grid);
  else chunk_combine_kernel<128><<<cg, 256, 0, stream>>>(p, grid);
  return cudaGetLastError();
}

}  // namespace qpa
