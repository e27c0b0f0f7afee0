// pa_decode_nvfp4: attention of one new token per sequence over the 4-bit pages.
//
// Mathematics: out = sum_t p_t v_t / sum_t p_t, p_t = 2^(c s_t - m) with s_t the dot
// product, c the logits' factor in base 2 and m a running reference per row.
//
// Bound: the pages' bytes, 2 (D/2 + D/16) per (token, KV head), once per block of 16 query
// rows (16 x 16384 tokens, 8 heads of 128: 59 us with 8 rows, 76 with 16, 137 with 32 in two
// passes) and, with more than 8 rows or heads of 64, the chains (S, softmax, V's conversion and
// products) of as many warps as registers allow.
//
// One persistent CTA per SM, the work (KV head and block of query rows, sequence, tile
// of 128 tokens) in one list that is cut into equal ranges, an item's beginning counted as
// a few tiles:
//  * 4 copy warps stream the tiles (K and V codes and scales, 18 KB with head_dim
//    128) into a ring by cp.async, tokens past the end as zeros, and build the item's
//    query operand.
//  * One warp issues the products S^T = K Q'^T on the block-scaled fp4 tensor core
//    (kind::mxf4nvf4): the pages' e2m1 codes and e4m3 scales are the operand as they
//    are, 128 tokens x 64 dims at a time. Q' holds each query row as 6 e2m1 terms of
//    weights 1, 1/8, .. 8^-5 (3 bits each) with a power of two per 16 dims, so a query
//    is within 2^-17 of its 16 dims' largest (or 2^-31 of the row's, which e4m3's range of
//    powers leaves of much smaller ones), and exact down to 2^-9 of it. Two passes
//    accumulate terms 0, 2, 4 and 1, 3, 5, the weight 1/8 in the scales, so that S has three
//    columns per row.
//  * Groups of 4 consumer warps take the tiles in turn; each warp owns 32 tokens of a
//    tile and its own softmax state, so nothing is exchanged before the item's end: it
//    reads S from tensor memory (a lane a token), forms p in f16, and multiplies V on
//    f16 mma.sync. V is taken from shared memory once, as pairs of tokens per dim: the
//    nibbles of two tokens are put in one byte, converted (cvt, exact) and multiplied
//    with the two tokens' scales (exact in f16: 2 by 4 bits). Through the tensor core's
//    shared-memory operands the converted V would cost its bytes four times over:
//    written and read at 2 bytes an element where the page has half a byte.
//    The sum of p is one more row of V, of ones.
//  * The reference m is put 8 below the largest logit (in base 2) and moves only when one
//    exceeds it by 14: f16 holds 11 bits of p down to 2^-22 of the largest, and the common
//    path has no exchange of maxima and no rescaling. (p in f16 is a choice: a result is 2e-4 off
//    for it, its own rounding to bf16 1.6e-3; a second term of p would double V's products.)
// An item that its range does not cut is written out; pieces go to the workspace (two
// slots per CTA: a range begins in at most one cut item and ends in another), and a
// second kernel joins them in order. Where no sequence can have more than 4 tiles
// (max_blocks_per_seq * block_size <= 512) the list is of whole sequences and the second
// kernel is not launched (whole against cut, graphs in a row, heads of 128: four of up to 200
// tokens, 2 x 4 heads, 6.9 against 8.7 us; four of 512 8.2, 9.3; 64 of 512, 8 x 8 heads, 22.0, 26.7; but
// four of 1024 10.0, 9.4; 64 of up to 1024 32.1, 30.7). Wall clock of a call from Python, four of up to
// 200 tokens: 17 to 21 us; with a table of 512 columns 22 to 24.
#define QPA_WHOLE_UNIT
#include <cmath>

#include "qpa.h"
#include "common.cuh"
#include "kept_answer.h"
#include "qpa_internal.h"
#include "tc.cuh"

namespace qpa {

namespace d4 {
constexpr int TILE = 128;           // tokens per tile
constexpr int QT = 6;               // e2m1 terms of a query
constexpr int MAX_CTAS = 160;
constexpr int COMBINE_WARPS = 4;
constexpr float kNoMax = -3.40282347e38f;   // no token seen yet: the lowest float, so that no logit is below it
constexpr float kBelow = 8.f;       // the reference is set this far below the largest logit (p up to 2^8)
constexpr float kTop = 14.f;        // and moves when a logit is this far above it (p up to 2^14 in f16)

template <int NT, int HD>
struct Smem {
  static constexpr int NWG = NT == 2 ? 2 : HD == 128 ? 3 : 4;   // consumer groups of 4 warps
  static constexpr int NCW = 4 * NWG;
  static constexpr int WARP_COPY = NCW;
  static constexpr int WARP_MMA = NCW + 4;         // one per consumer group
  static constexpr int THREADS = (WARP_MMA + 4) * 32;   // (whole warpgroups, for the register budgets)
  // registers of the roles' threads; their sum is the launch's
  static constexpr int REG_CONSUMER = NWG == 4 ? 96 : NWG == 3 ? 120 : 168, REG_COPY = NWG == 4 ? 72 : NWG == 3 ? 80 : 104;
  static constexpr int REG_MMA = NWG == 4 ? 24 : NWG == 3 ? 40 : 72;
  static constexpr int REG_LAUNCH = 65536 / THREADS / 8 * 8;
  static_assert(128 * (NWG * REG_CONSUMER + REG_COPY + REG_MMA) <= THREADS * REG_LAUNCH, "registers");
  // (setmaxnreg.inc to fewer or .dec to more than a warp has is an illegal instruction)
  static_assert(REG_CONSUMER >= REG_LAUNCH && REG_COPY <= REG_LAUNCH && REG_MMA <= REG_LAUNCH, "registers of a role");
  static constexpr int R = 8 * NT;                 // query rows (padded)
  static constexpr int KS = HD / 64;               // K steps of the fp4 product
  // Passes of the product (pass k accumulates terms k, k + PASSES, ..), groups of 8 columns of S per row block. A pass
  // reads K's tile from shared memory once more, a group costs the softmax a packed FMA per pair of rows and registers.
  // 16 x 16384 tokens, 8 x 8 heads of 128: 65.1 us with 1 pass, 61.6 with 2, 63.6 with 3. 32 sequences, heads of 64: 8 x 8
  // 51.5, 43.4, 44.4 us, 8 x 16 64.2, 61.2, 60.2 (where a third pass would leave 2^-28 of a row's largest, not 2^-31).
  static constexpr int PASSES = 2, CG = QT / PASSES;
  static constexpr int NQ = (8 * CG * NT + 15) / 16 * 16;   // columns of S: row block x group x 8 rows
  static constexpr int ROW = HD / 2;               // code bytes of a token
  static constexpr int V_OFF = TILE * ROW;
  static constexpr int KS_OFF = 2 * TILE * ROW;    // K scales as V's, then (MMA warp) [KS][token % 32][token / 32][4]
  static constexpr int VS_OFF = KS_OFF + KS * 512; // V scales [token][HD / 16]
  static constexpr int SLOT = VS_OFF + TILE * (HD / 16);
  // An item's beginning (and the end before it) weighed in tiles when the work is cut. One of 131071 tokens, 4 x 16 heads of
  // 128: 34.2 us with 0, 30.8 with 2 to 8; 64 ragged 116.8, 114.3 with 5; 32 sequences, 8 x 8 heads of 64, 43.8, 41.0 with 7 to 10.
  static constexpr int BEGIN = HD == 64 ? 8 : 5;
  static constexpr int NSB = 2 * NWG;              // S buffers, two per group
  static constexpr int qBytes = PASSES * NQ * ROW;
  static constexpr int STG_ROW = HD;               // floats of a staged row
  static constexpr int stgBytes = NCW * 8 * STG_ROW * 4;   // one row block at a time
  static constexpr int pBytes = 32 * 16 * NT;      // a warp's P [32 tokens][8 rows] f16 per row block
  // Ring slots, NSG per group. A slot has one group and one copy warp, which see every phase
  // of its barriers: a wait on a parity cannot mistake a phase for the one before the last.
  static constexpr int CPG = 4 / NWG;              // copy warps of a group, taking its tiles in turn
  static constexpr int NSG = NWG == 4 ? 5 : (NWG == 3 ? 3 : 4) * (HD == 128 ? 1 : 2);
  static_assert(NSG % CPG == 0, "ring");
  static constexpr int NS = NWG * NSG;
  static constexpr int qOff = NS * SLOT;
  static constexpr int qsOff = qOff + 2 * qBytes;             // [2][PASSES][KS][512] query scales
  static constexpr int stgOff = qsOff + 2 * PASSES * KS * 512;         // [NCW][8][STG_ROW] f32
  // (a warp's P lies at the beginning of its staged rows)
  static constexpr int mlOff = stgOff + stgBytes;             // [NCW][8] {m, l}
  static constexpr int cOff = mlOff + NCW * 8 * 8;            // [2][R] logit factor per row
  static constexpr int infoOff = cOff + 2 * R * 4;            // [2] item
  static constexpr int barOff = infoOff + 2 * 64;
  static constexpr int NBAR = 2 * NS + 4 + 2 * NSB + 3;
  static constexpr int miscOff = barOff + NBAR * 8;
  static constexpr int total = miscOff + 16 + 1024;           // + alignment slack
  static_assert(pBytes <= 8 * STG_ROW * 4, "P");
  static_assert(SLOT % 1024 == 0 && qBytes % 512 == 0 && total <= 227 * 1024, "shared memory");
  // tensor memory: S buffers, K scales per S buffer, query scales per group and operand
  static constexpr int SFA_COL = NSB * NQ, SFB_COL = SFA_COL + NSB * 4 * KS;
  static constexpr int USED_COLS = SFB_COL + 2 * NWG * PASSES * 4 * KS;
  static constexpr int TMEM_COLS = USED_COLS <= 256 ? 256 : 512;
  static_assert(USED_COLS <= TMEM_COLS, "tensor memory");
};

struct Params {
  const uint16_t* q;
  const uint8_t* kv;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const float* k_scale;
  const float* v_scale;
  uint16_t* out;                    // bf16
  float* part_o;                    // [2 CTAs][16][HD], relative to m, not divided by l
  float2* part_ml;                  // [2 CTAs][16] {m, l}
  int4* meta;                       // [CTAs] {pieces (0: none), sequence, virtual head, 0}
  long long q_stride_seq, q_stride_head, table_stride;
  int num_seqs, num_kv_heads, qg, row_blocks, block_size, log2_bs, num_blocks, max_blocks;
  int whole;                        // a unit of work is a sequence, not a tile: no item is cut
  float softmax_mant;               // softmax_scale = softmax_mant 2^softmax_exp
  int softmax_exp;
};

// kind::mxf4nvf4 instruction descriptor: e2m1 operands, K-major, unsigned e4m3 scales
__host__ __device__ constexpr uint32_t idesc_fp4(int m, int n) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
__device__ __forceinline__ void mma_fp4(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t hi, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{ .reg .pred p; .reg .b64 a, b; setp.ne.b32 p, %7, 0; mov.b64 a, {%1, %3}; mov.b64 b, {%2, %3}; "
      "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], a, b, %4, [%5], [%6], p; }"
      ::"r"(d), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate) : "memory");
}
// N consecutive columns of this warp's 32 lanes (as tmem_ld32)
template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, float (&v)[N]) {
  int at = 0;
  if constexpr (N >= 32) {
    float r[32];
    tmem_ld32(taddr, r);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = r[i];
    at = 32;
  }
  if constexpr (N % 32 >= 16) {
    float r[16];
    tmem_ld16(taddr + at, r);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[(N >= 32 ? 32 : 0) + i] = r[i];
    at += 16;
  }
  if constexpr (N % 16 == 8) {
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(taddr + at));
#pragma unroll
    for (int i = 0; i < 8; ++i) v[N - 8 + i] = __uint_as_float(r[i]);
  }
}
// 512 bytes of scales (32 rows of 16) to 4 columns of all four lane quarters
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint32_t lo, uint32_t hi) {
  asm volatile("{ .reg .b64 d; mov.b64 d, {%1, %2}; tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], d; }"
               ::"r"(taddr), "r"(lo), "r"(hi) : "memory");
}
// 16 bytes, those behind the first `bytes` as zeros (and not read)
__device__ __forceinline__ void cp_async16_part(uint32_t dst, const void* src, int bytes, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;"
               ::"r"(dst), "l"(src), "r"(bytes), "l"(policy) : "memory");
}
__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ uint32_t lds8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ void sts8(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
// mbar_arrive by the lanes with `on`, without a branch (a branch of one lane costs the warp about 100 cycles)
__device__ __forceinline__ void arrive_if(bool on, uint64_t* bar) {
  asm volatile("{ .reg .pred p; .reg .b64 st; setp.ne.u32 p, %1, 0; @p mbarrier.arrive.release.cta.shared::cta.b64 st, [%0]; }"
               ::"r"(smem_u32(bar)), "r"((uint32_t)on) : "memory");
}
// warp_wait, whose own path the warp takes only if a lane's first try fails
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int err) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  return warp_wait(bar, parity, abort_flag, err);
}
// Order of the 16-byte pieces of staged rows 2 c and 2 c + 1: a store's 8 lanes of a phase (c = 0 .. 3, two dims groups
// that lie 4 (head_dim 128) or 2 pieces apart) then go to 8 different ones.
template <int HD>
__device__ __forceinline__ int stage_swizzle(int c) { return HD == 128 ? c : (c & 1) | ((c & 2) << 1); }
// (x, y) * w + (a, b)
__device__ __forceinline__ void fma2(float& x, float& y, float w, float a, float b) {
  asm("{ .reg .b64 p, q, r; mov.b64 p, {%0, %1}; mov.b64 q, {%2, %2}; mov.b64 r, {%3, %4}; "
      "fma.rn.f32x2 p, p, q, r; mov.b64 {%0, %1}, p; }" : "+f"(x), "+f"(y) : "f"(w), "f"(a), "f"(b));
}
// (x, y) * (a, b); (x, y) - (a, b)
__device__ __forceinline__ void mul2(float& x, float& y, float a, float b) {
  asm("{ .reg .b64 p, q; mov.b64 p, {%0, %1}; mov.b64 q, {%2, %3}; mul.rn.f32x2 p, p, q; mov.b64 {%0, %1}, p; }"
      : "+f"(x), "+f"(y) : "f"(a), "f"(b));
}
__device__ __forceinline__ void sub2(float& x, float& y, float a, float b) {
  asm("{ .reg .b64 p, q; mov.b64 p, {%0, %1}; mov.b64 q, {%2, %3}; sub.rn.f32x2 p, p, q; mov.b64 {%0, %1}, p; }"
      : "+f"(x), "+f"(y) : "f"(a), "f"(b));
}
__device__ __forceinline__ uint32_t f32x2_to_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{ .reg .b8 t; cvt.rn.satfinite.e2m1x2.f32 t, %2, %1; cvt.u32.u8 %0, t; }" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}

// x = m 2^e with 1 <= |m| < 2: m, and e added to `exponent`; 0, infinities and NaN as they are
__device__ __forceinline__ float mantissa(float x, int& exponent) {
  const bool small = fabsf(x) < 1.17549435e-38f;                        // 2^-126
  const uint32_t b = __float_as_uint(small ? x * 16777216.f : x), e = (b >> 23) & 255u;
  if (e == 0 || e == 255u) return x;
  exponent += (int)e - 127 - (small ? 24 : 0);
  return __uint_as_float((b & 0x807fffffu) | 0x3f800000u);
}

// A taker's tiles, every `of`-th of the CTA's: the ring slot (of the group's ns, every by-th) and
// its phase, how many so far, and the item's first one (counted from the item's beginning).
struct Turn {
  int slot, first, count, ns, of;
  uint32_t phase;
  int by;
  __device__ __forceinline__ Turn(int me, int ns_, int of_, int slot_ = 0, int by_ = 1)
      : slot(slot_), first(me), count(0), ns(ns_), of(of_), phase(0), by(by_) {}
  __device__ __forceinline__ void step() {
    ++count;
    slot += by;
    if (slot >= ns) {
      slot -= ns;
      phase ^= 1;
    }
  }
  // behind an item of nt tiles
  __device__ __forceinline__ void item(int nt) {
    const int r = (first - nt) % of;
    first = r < 0 ? r + of : r;
  }
};

// (up to 2^31 - 1 tokens)
__device__ __forceinline__ int tiles_of(int len) { return (int)(((unsigned)len + TILE - 1) / TILE); }

// The beginning of an item: sequence s of length L and T tiles, virtual head vh (KV head
// vh / RB, row block vh % RB).
struct Cursor {
  int s, vh, L, T;
  long long off;      // work of the sequences before s
  int t;              // first tile of the item
  int v;              // units of its beginning
};

}  // namespace d4

template <int NT, int HD>
__global__ void __launch_bounds__(d4::Smem<NT, HD>::THREADS, 1) decode4_kernel(const d4::Params p) {
  using namespace d4;
  using S = Smem<NT, HD>;
  constexpr int PASSES = S::PASSES, CG = S::CG;
  constexpr int R = S::R, NQ = S::NQ, NS = S::NS, NSB = S::NSB, NWG = S::NWG, NCW = S::NCW, KS = S::KS, ROW = S::ROW;
  constexpr uint32_t SWZ = HD == 128 ? kSwizzle64B : 6u;      // rows of 64 or 32 bytes
  constexpr int MT = HD / 16;                                 // m-tiles of V^T
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sb = (raw + 1023u) & ~1023u;
  uint8_t* sm = smem_raw + (sb - raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(sm + S::barOff);   // [NS] tile copied (a copy warp's lanes)
  uint64_t* empty = full + NS;         // [NS] tile consumed (MMA commit, a group's 4 warps)
  uint64_t* qfull = empty + NS;        // [2] item published (4 copy warps)
  uint64_t* qempty = qfull + 2;        // [2] item done (MMA commits, consumer warps)
  uint64_t* sfull = qempty + 2;        // [NSB] S ready (MMA commit)
  uint64_t* sfree = sfull + NSB;       // [NSB] S read (4 warps)
  uint64_t* staged = sfree + NSB;      // item states published (consumer warps)
  uint64_t* merged = staged + 1;       // item states read (consumer warps)
  uint64_t* done = merged + 1;         // all MMAs finished
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + S::miscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + S::miscOff + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // (on their way while the barriers are set up)
  const int bs = p.block_size, lbs = p.log2_bs, Hk = p.num_kv_heads, RB = p.row_blocks, B = p.num_seqs;
  auto seq_len = [&](int s) -> int { return max(0, min(__ldg(p.seq_lens + s), p.max_blocks * bs)); };
  const int len0 = lane < B ? seq_len(lane) : 0;
  const float kscale = __ldg(p.k_scale), vscale = __ldg(p.v_scale);
  static_assert(S::NBAR <= 64, "a thread each");
  if (threadIdx.x < S::NBAR) {
    uint64_t* bar = full + threadIdx.x;
    mbar_init(bar, bar < empty ? 32 : bar < qfull ? 1 + 4 : bar < qempty ? 4 : bar < sfull ? NWG + NCW : bar < sfree ? 1
                   : bar < staged ? 4 : bar < done ? NCW : NWG);
    if (threadIdx.x == 0) *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == S::WARP_MMA) tmem_alloc(tmem_slot, S::TMEM_COLS);
  // barriers and tensor memory are there: each role waits for it where it needs them (the copy warps with the first item's
  // table entries and queries on their way)
  auto all_set = [&]() {
    tc_fence_before();
    asm volatile("bar.sync 0;" ::: "memory");
    tc_fence_after();
  };
  const int Hq = Hk * p.qg;

  if (warp < NCW) {
    // ======================================================== consumer warps
    all_set();
    const uint32_t tmem = *tmem_slot;
    reg_inc<S::REG_CONSUMER>();
    const int wg = warp >> 2, wq = warp & 3;
    const int g = lane >> 2, c = lane & 3;
    // sequences without tokens give 0
    for (int s = blockIdx.x * NCW + warp; s < B; s += gridDim.x * NCW)
      if (seq_len(s) == 0)
        for (long long i = lane; i < (long long)Hq * HD / 8; i += 32)
          reinterpret_cast<uint4*>(p.out + (long long)s * Hq * HD)[i] = make_uint4(0, 0, 0, 0);
    const uint32_t tl = tmem + ((uint32_t)(wq * 32) << 16);
    const uint32_t psm = sb + S::stgOff + warp * (8 * S::STG_ROW * 4);
    // ldmatrix row of this lane: token 16 (i / 2) + 8 (i % 2) + 4 (j % 2) + j / 2 of matrix i = lane / 8, row j
    const int mi = lane >> 3, mj = lane & 7;
    const uint32_t prow = psm + 16 * (16 * (mi >> 1) + 8 * (mi & 1) + 4 * (mj & 1) + (mj >> 1));
    // V of token 4 u + c: 8 or 4 bytes, the lane's 16 or 8 dims
    const uint32_t vlane = HD == 128 ? S::V_OFF + (32 * wq + c) * 64 + (((g >> 1) ^ (c & 2)) << 4) + 8 * (g & 1)
                                     : S::V_OFF + (32 * wq + c) * 32 + 4 * g;
    const uint32_t slane = S::VS_OFF + (32 * wq + c) * (HD / 16) + (HD == 128 ? g : g >> 1);
    float o[NT][MT][4], ol[NT][4], m[R];
    Turn tn(wg, S::NSG, NWG);
    int merges = 0;                                  // row blocks joined so far
    bool ok = true;
    for (int n = 0; ok; ++n) {
      const int qb = n & 1;
      if (!wait_bar(&qfull[qb], (n >> 1) & 1, abort_flag, KERR_TIMEOUT_FULL)) break;
      const int4 inf = lds_i4(sb + S::infoOff + 64 * qb);               // L, first tile, tiles, part (-1: whole)
      const int4 who = lds_i4(sb + S::infoOff + 64 * qb + 16);          // sequence, virtual head
      const int L = inf.x, t0 = inf.y, nt = inf.z, last = (L - 1) / TILE;
      if (nt == 0) break;
#pragma unroll
      for (int nb = 0; nb < NT; ++nb) {
#pragma unroll
        for (int i = 0; i < MT; ++i) o[nb][i][0] = o[nb][i][1] = o[nb][i][2] = o[nb][i][3] = 0.f;
        ol[nb][0] = ol[nb][1] = ol[nb][2] = ol[nb][3] = 0.f;
      }
#pragma unroll
      for (int r = 0; r < R; ++r) m[r] = kNoMax;
      uint32_t w[8][HD / 64], sc[8];                 // V of this warp's 32 tokens: 4 u + c, u < 8
      float x[R];                                    // logits (base 2)
      float v[NT][8 * CG];                           // S: groups of terms x 8 rows
      // V's bytes into registers; the slot is free then
      auto load_v = [&]() -> bool {
        const int s = wg * S::NSG + tn.slot;
        if (!wait_bar(&full[s], tn.phase, abort_flag, KERR_TIMEOUT_FULL)) return false;
        const uint32_t slot = sb + s * S::SLOT;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const uint32_t a = slot + vlane + 4 * u * ROW;
          if constexpr (HD == 128) {
            const uint2 d = lds64(a);
            w[u][0] = d.x;
            w[u][1] = d.y;
          } else {
            w[u][0] = lds32(a);
          }
          sc[u] = lds8(slot + slane + 4 * u * (HD / 16));
        }
        __syncwarp();
        arrive_if(lane == 0, &empty[s]);
        return true;
      };
      // S on its way to registers
      auto wait_s = [&](int count) -> bool {
        if (!wait_bar(&sfull[2 * wg + (count & 1)], (count >> 1) & 1, abort_flag, KERR_TIMEOUT_FULL)) return false;
        tc_fence_after();
        return true;
      };
      auto load_s = [&](int count) {
#pragma unroll
        for (int nb = 0; nb < NT; ++nb) tmem_ld_cols(tl + (2 * wg + (count & 1)) * NQ + 8 * CG * nb, v[nb]);
      };
      // S has come: its groups joined, times the rows' factors (v is free then). The product is rounded before the
      // reference is taken off, as it is where the reference comes from: a fused one differs by up to half a step of the
      // logit, which is f16's room and more where logits are large.
      auto join_terms = [&]() {
        tmem_wait_ld();
#pragma unroll
        for (int nb = 0; nb < NT; ++nb) {
          const float4 f0 = lds_f4(sb + S::cOff + 4 * (qb * R + 8 * nb)), f1 = lds_f4(sb + S::cOff + 4 * (qb * R + 8 * nb) + 16);
          const float f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
#pragma unroll
          for (int r = 0; r < 8; r += 2) {
            float x0 = v[nb][8 * (CG - 1) + r], x1 = v[nb][8 * (CG - 1) + r + 1];
#pragma unroll
            for (int k = CG - 2; k >= 0; --k)
              fma2(x0, x1, 1.f / (1 << (3 * PASSES)), v[nb][8 * k + r], v[nb][8 * k + r + 1]);
            mul2(x0, x1, f[r], f[r + 1]);
            x[8 * nb + r] = x0;
            x[8 * nb + r + 1] = x1;
          }
        }
      };
      auto free_s = [&](int count) {
        tc_fence_before();
        __syncwarp();
        arrive_if(lane == 0, &sfree[2 * wg + (count & 1)]);
      };
      if (tn.first < nt) {
        if (!load_v() || !wait_s(tn.count)) { ok = false; break; }
        load_s(tn.count);
        join_terms();
        free_s(tn.count);
      }
      // (P and the staged rows share their memory)
      if (merges > 0 && !wait_bar(merged, (merges - 1) & 1, abort_flag, KERR_TIMEOUT_EMPTY)) break;
      for (int i = tn.first; i < nt; i += NWG) {
        const int tok = (t0 + i) * TILE + 32 * wq + lane;               // this lane's token
        const bool cut = t0 + i == last;                                // the sequence ends in this tile
        const bool more = i + NWG < nt;
        // ---- logits of this token relative to the rows' references (both row blocks at once: one vote, and their chains
        // overlap; 32 sequences, 8 x 16 heads of 64, 61.2 -> 58.1 us)
        float e[R];
#pragma unroll
        for (int r = 0; r < R; r += 2) {
          e[r] = x[r];
          e[r + 1] = x[r + 1];
          sub2(e[r], e[r + 1], m[r], m[r + 1]);
        }
        if (cut) {                                     // (of the whole warp: no other tile pays for it)
          const bool past = tok >= L;
#pragma unroll
          for (int r = 0; r < R; ++r) e[r] = past ? -INFINITY : e[r];
        }
        float top = -INFINITY;
#pragma unroll
        for (int r = 0; r < R; r += 8)
          top = fmaxf(top, fmaxf(fmaxf(fmaxf(e[r], e[r + 1]), fmaxf(e[r + 2], e[r + 3])), fmaxf(fmaxf(e[r + 4], e[r + 5]), fmaxf(e[r + 6], e[r + 7]))));
        if (__any_sync(0xffffffffu, top > kTop)) {
          // ---- move the references of the rows that need it
#pragma unroll
          for (int nb = 0; nb < NT; ++nb) {
            float a0 = 1.f, a1 = 1.f;                                   // of this lane's output columns, rows 2c and 2c + 1
#pragma unroll
            for (int r = 0; r < 8; ++r) {
              // (a masked token does not count; NaN is ignored)
              const float best = warp_max(cut && tok >= L ? -INFINITY : x[8 * nb + r]);
              const float old = m[8 * nb + r];
              // (decided by the rounded difference that was voted on; one below best that rounds to more than kTop below, from
              // 2^27 on, is best itself: p stays within f16)
              const float below = best - kBelow;
              const float now = best - old > kTop ? (best - below > kTop ? best : below) : old;
              const float alpha = ex2(old - now);
              m[8 * nb + r] = now;
              e[8 * nb + r] = cut && tok >= L ? -INFINITY : x[8 * nb + r] - now;
              if (r == 2 * c) a0 = alpha;
              if (r == 2 * c + 1) a1 = alpha;
            }
#pragma unroll
            for (int k = 0; k < MT; ++k) {
              o[nb][k][0] *= a0;
              o[nb][k][1] *= a1;
              o[nb][k][2] *= a0;
              o[nb][k][3] *= a1;
            }
            ol[nb][0] *= a0;
            ol[nb][1] *= a1;
          }
        }
        float ex[R];
#pragma unroll
        for (int r = 0; r < R; ++r) ex[r] = ex2(e[r]);
        // ---- p in f16, a row of the warp's P
#pragma unroll
        for (int nb = 0; nb < NT; ++nb) {
          const float* q = ex + 8 * nb;
          sts_i4(psm + 512 * nb + 16 * lane, make_int4(f32x2_to_f16x2(q[0], q[1]), f32x2_to_f16x2(q[2], q[3]), f32x2_to_f16x2(q[4], q[5]),
                                                       f32x2_to_f16x2(q[6], q[7])));
        }
        __syncwarp();
        uint32_t pb[NT][4];
#pragma unroll
        for (int nb = 0; nb < NT; ++nb) ldsm_x4_trans(prow + 512 * nb, pb[nb]);
        // ---- O^T += V^T P^T, 16 tokens at a time
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t s01 = e4m3x2_lo_to_f16x2(sc[4 * k] | (sc[4 * k + 1] << 8));
          const uint32_t s23 = e4m3x2_lo_to_f16x2(sc[4 * k + 2] | (sc[4 * k + 3] << 8));
#pragma unroll
          for (int h = 0; h < HD / 64; ++h) {
            // nibbles of two tokens per byte: dims 2 i and 2 i + 1
            const uint32_t ev01 = (w[4 * k][h] & 0x0f0f0f0fu) | ((w[4 * k + 1][h] << 4) & 0xf0f0f0f0u);
            const uint32_t od01 = ((w[4 * k][h] >> 4) & 0x0f0f0f0fu) | (w[4 * k + 1][h] & 0xf0f0f0f0u);
            const uint32_t ev23 = (w[4 * k + 2][h] & 0x0f0f0f0fu) | ((w[4 * k + 3][h] << 4) & 0xf0f0f0f0u);
            const uint32_t od23 = ((w[4 * k + 2][h] >> 4) & 0x0f0f0f0fu) | (w[4 * k + 3][h] & 0xf0f0f0f0u);
            auto tile = [&](int i, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
              a0 = hmul2(a0, s01);
              a1 = hmul2(a1, s01);
              a2 = hmul2(a2, s23);
              a3 = hmul2(a3, s23);
#pragma unroll
              for (int nb = 0; nb < NT; ++nb) mma_f16_16816(o[nb][4 * h + i], a0, a1, a2, a3, pb[nb][2 * k], pb[nb][2 * k + 1]);
            };
            tile(0, e2m1x2_to_f16x2<0>(ev01), e2m1x2_to_f16x2<0>(od01), e2m1x2_to_f16x2<0>(ev23), e2m1x2_to_f16x2<0>(od23));
            tile(1, e2m1x2_to_f16x2<1>(ev01), e2m1x2_to_f16x2<1>(od01), e2m1x2_to_f16x2<1>(ev23), e2m1x2_to_f16x2<1>(od23));
            tile(2, e2m1x2_to_f16x2<2>(ev01), e2m1x2_to_f16x2<2>(od01), e2m1x2_to_f16x2<2>(ev23), e2m1x2_to_f16x2<2>(od23));
            tile(3, e2m1x2_to_f16x2<3>(ev01), e2m1x2_to_f16x2<3>(od01), e2m1x2_to_f16x2<3>(ev23), e2m1x2_to_f16x2<3>(od23));
          }
#pragma unroll
          for (int nb = 0; nb < NT; ++nb)      // the sum of p: a row of ones
            mma_f16_16816(ol[nb], 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, pb[nb][2 * k], pb[nb][2 * k + 1]);
        }
        tn.step();
        if (more) {
          if (!wait_s(tn.count)) { ok = false; break; }
          load_s(tn.count);
          join_terms();
          free_s(tn.count);
          if (!load_v()) { ok = false; break; }
        }
      }
      if (!ok) break;
      const bool had = tn.first < nt;                 // this group had tiles of the item
      tn.item(nt);
      __syncwarp();
      arrive_if(lane == 0, &qempty[qb]);
      __syncwarp();
      // ---- item done: the warps' states to shared memory, a row block at a time; each warp
      // joins one row of it
      const int rbase = 16 * (who.y % RB), kvh = who.y / RB;
      const int rows = min(R, p.qg - rbase);
      const uint32_t stg = sb + S::stgOff;
      // (a loop, the second row block moved to the first one's registers: this runs once per item, and its code has to
      // be fetched)
#pragma unroll 1
      for (int nb = 0; nb < NT; ++nb, ++merges) {
        if (nb > 0 && !wait_bar(merged, (merges - 1) & 1, abort_flag, KERR_TIMEOUT_EMPTY)) { ok = false; break; }
        if (had)                                         // (a group without tiles stages no rows)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          // (16-byte pieces of a row in an order of the row's own: the rows of a store's lanes lie in the same banks)
          const uint32_t a = stg + 4 * ((warp * 8 + 2 * c + hh) * S::STG_ROW);
#pragma unroll
          for (int k = 0; k < MT; k += 2)
            sts_i4(a + 16 * ((MT / 2 * g + k / 2) ^ stage_swizzle<HD>(c)), make_int4(__float_as_int(o[0][k][hh]), __float_as_int(o[0][k][2 + hh]),
                                        __float_as_int(o[0][k + 1][hh]), __float_as_int(o[0][k + 1][2 + hh])));
        }
        {
          // lane r < 8: m of row r (selected: a branch per row takes 100 cycles), l from the lane c = r / 2 of g = 0
          float mr = m[0];
#pragma unroll
          for (int r = 1; r < 8; ++r) mr = lane == r ? m[r] : mr;
          const float l0 = __shfl_sync(0xffffffffu, ol[0][0], (lane >> 1) & 3), l1 = __shfl_sync(0xffffffffu, ol[0][1], (lane >> 1) & 3);
          if (lane < 8)
            asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(sb + S::mlOff + 8 * (warp * 8 + lane)), "f"(mr),
                         "f"(lane & 1 ? l1 : l0) : "memory");
        }
        if constexpr (NT > 1) {
#pragma unroll
          for (int k = 0; k < MT; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[0][k][e] = o[NT - 1][k][e];
#pragma unroll
          for (int e = 0; e < 2; ++e) ol[0][e] = ol[NT - 1][e];
#pragma unroll
          for (int r = 0; r < 8; ++r) m[r] = m[R - 8 + r];
        }
        __syncwarp();
        arrive_if(lane == 0, staged);
        if (!wait_bar(staged, merges & 1, abort_flag, KERR_TIMEOUT_FULL)) { ok = false; break; }
        const int row = 8 * nb + warp;
        if (row < rows) {
          float mw[NCW], lw[NCW], M = kNoMax, l = 0.f;
#pragma unroll
          for (int k = 0; k < NCW; ++k) {
            const uint2 d = lds64(sb + S::mlOff + 8 * (k * 8 + warp));
            mw[k] = __uint_as_float(d.x);
            lw[k] = __uint_as_float(d.y);
            M = fmaxf(M, mw[k]);
          }
          float acc[HD / 32];
#pragma unroll
          for (int d = 0; d < HD / 32; ++d) acc[d] = 0.f;
          // (rows of a warp that saw no token hold anything: taken as 0)
#pragma unroll
          for (int k = 0; k < NCW; ++k) {
            const float f = ex2(mw[k] - M);
            const bool some = lw[k] != 0.f;
            l = fmaf(f, lw[k], l);
            const uint32_t a = stg + 4 * ((k * 8 + warp) * S::STG_ROW) +
                               16 * ((lane * (HD / 32) / 4) ^ stage_swizzle<HD>((warp >> 1) & 3)) + (HD == 128 ? 0 : 8 * (lane & 1));
            if constexpr (HD == 128) {
              const float4 d = lds_f4(a);
              acc[0] = fmaf(f, some ? d.x : 0.f, acc[0]);
              acc[1] = fmaf(f, some ? d.y : 0.f, acc[1]);
              acc[2] = fmaf(f, some ? d.z : 0.f, acc[2]);
              acc[3] = fmaf(f, some ? d.w : 0.f, acc[3]);
            } else {
              const uint2 d = lds64(a);
              acc[0] = fmaf(f, some ? __uint_as_float(d.x) : 0.f, acc[0]);
              acc[1] = fmaf(f, some ? __uint_as_float(d.y) : 0.f, acc[1]);
            }
          }
          if (inf.w < 0) {
            // (v_scale last: v_scale / l may lie in float32's subnormals where the result does not)
            const float inv = 1.f / l;
            __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(p.out) +
                                 ((long long)who.x * Hq + (long long)kvh * p.qg + rbase + row) * HD + (HD / 32) * lane;
            if constexpr (HD == 128) store4(dst, acc[0] * inv * vscale, acc[1] * inv * vscale, acc[2] * inv * vscale, acc[3] * inv * vscale);
            else *reinterpret_cast<__nv_bfloat162*>(dst) = __floats2bfloat162_rn(acc[0] * inv * vscale, acc[1] * inv * vscale);
          } else {
            float* dst = p.part_o + ((long long)inf.w * 16 + row) * HD + (HD / 32) * lane;
            if constexpr (HD == 128) store4(dst, acc[0], acc[1], acc[2], acc[3]);
            else *reinterpret_cast<float2*>(dst) = make_float2(acc[0], acc[1]);
            if (lane == 0) p.part_ml[inf.w * 16 + row] = make_float2(M, l);
          }
        }
        __syncwarp();
        arrive_if(lane == 0, merged);
      }
    }
  } else if (warp < S::WARP_MMA) {
    // ======================================================== copy warps
    reg_dec<S::REG_COPY>();
    const int pw = warp - S::WARP_COPY, pt = 32 * pw + lane;
    const uint64_t pol = policy_evict_first();
    constexpr int CPR = ROW / 16, RPI = 32 / CPR;                       // 16-byte chunks per token, tokens per instruction
    const int lr = lane / CPR, cc = lane % CPR;
    const uint32_t kdst = lr * ROW + ((HD == 128 ? cc ^ ((lr >> 1) & 3) : cc ^ ((lr >> 2) & 1)) << 4);
    const uint32_t vdst = S::V_OFF + lr * ROW + ((HD == 128 ? cc ^ (lr & 2) : cc) << 4);
    const uint32_t src_lane = lr * ROW + 16 * cc;
    constexpr int SPC = 16 / (HD / 16);                                 // tokens whose scales 16 bytes hold
    const size_t chunk = size_t(bs) * (HD / 2 + HD / 16), plane = size_t(Hk) * chunk;

    // ---- the CTA's range of units, and the item that holds its first one
    // work of a sequence of T tiles, its beginning counted as BEGIN of them (32 sequences: below 2^30)
    constexpr int BEGIN = S::BEGIN;
    auto work = [&](int T) -> int { return p.whole ? min(T, 1) : T > 0 ? T + BEGIN : 0; };
    long long W = 0;
    for (int s0 = 0; s0 < B; s0 += 32)
      W += __reduce_add_sync(0xffffffffu, (unsigned)work(tiles_of(s0 == 0 ? len0 : s0 + lane < B ? seq_len(s0 + lane) : 0)));
    const long long U = W * (Hk * (long long)RB);
    const int G = gridDim.x;
    const long long per = div_nonneg(U, G), rem = U - per * G;          // the first `rem` ranges have one more
    auto first_of = [&](long long cta) -> long long { return per * cta + min(cta, rem); };
    long long u = first_of(blockIdx.x);
    const long long u1 = first_of(blockIdx.x + 1LL);
    // the first sequence with tiles behind tile x of the head's list
    auto find = [&](int s, long long off, long long x) -> Cursor {
      for (int s0 = s; s0 < B; s0 += 32) {
        const int L = s0 == 0 ? len0 : s0 + lane < B ? seq_len(s0 + lane) : 0;   // (s: of the first 32, or a later one)
        const int T = tiles_of(L);
        int incl = work(T);
#pragma unroll
        for (int sh = 1; sh < 32; sh <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, incl, sh);
          if (lane >= sh) incl += v;
        }
        const unsigned hit = __ballot_sync(0xffffffffu, off + incl > x);
        if (hit) {
          const int src = __ffs(hit) - 1;
          Cursor c;
          c.s = s0 + src;
          c.vh = 0;
          c.L = __shfl_sync(0xffffffffu, L, src);
          c.T = __shfl_sync(0xffffffffu, T, src);
          c.off = off + __shfl_sync(0xffffffffu, incl, src) - work(c.T);
          const int in = (int)(x - c.off);
          c.t = max(0, in - BEGIN);                 // (whole sequences: in is 0)
          c.v = p.whole ? 0 : max(0, BEGIN - in);
          return c;
        }
        off += __shfl_sync(0xffffffffu, incl, 31);
      }
      return Cursor{-1, 0, 0, 0, 0, 0, 0};   // (not reached: x < W)
    };
    Cursor cur{-1, 0, 0, 0, 0, 0, 0};
    if (u < u1) {
      const long long vh = div_nonneg(u, W);
      cur = find(0, 0, u - vh * W);
      cur.vh = (int)vh;
      if (u1 - u <= cur.v) cur.s = -1;              // (a beginning without a tile is the next range's)
    }
    // the item that begins at unit `at`, behind item c
    auto next = [&](const Cursor& c, long long at) -> Cursor {
      if (u1 - at <= (p.whole ? 0 : BEGIN)) return Cursor{-1, 0, 0, 0, 0, 0, 0};
      const long long off = c.off + work(c.T);
      Cursor n = off < W ? find(c.s + 1, off, off) : find(0, 0, 0);
      n.vh = off < W ? c.vh : c.vh + 1;
      return n;
    };
    // query row pt / 16 (and + 8) of a row block, dims 8 (pt % 16) ..
    const int qrow = pt >> 4, h16 = pt & 15;
    auto load_q = [&](const Cursor& c, uint4 (&qv)[NT]) {
#pragma unroll
      for (int h = 0; h < NT; ++h) {
        qv[h] = make_uint4(0, 0, 0, 0);
        if (c.s < 0 || h16 >= HD / 8) continue;
        const int row = 16 * (c.vh % RB) + qrow + 8 * h;
        if (row < p.qg)
          qv[h] = __ldg(reinterpret_cast<const uint4*>(p.q + c.s * p.q_stride_seq +
                                                       ((long long)(c.vh / RB) * p.qg + row) * p.q_stride_head) + h16);
      }
    };
    // 32 table entries from entry e0 on
    auto load_entries = [&](int s, int e0) -> int32_t {
      return s >= 0 && e0 + lane < p.max_blocks ? __ldg(p.block_table + (long long)s * p.table_stride + e0 + lane) : 0;
    };
    // the logits' factor, its power of two apart: k_scale and the softmax's scale may leave float32's range together where the
    // logits do not
    int base_exp = 0;
    const float base = mantissa(kscale, base_exp) * p.softmax_mant * kLog2e;
    base_exp += p.softmax_exp;
    uint4 qv[NT];
    load_q(cur, qv);
    int32_t ent0 = load_entries(cur.s, (int)(((long long)cur.t * TILE) >> lbs));
    all_set();
    Turn tn(pw, S::NSG, NWG * S::CPG, pw / NWG, S::CPG);                // (a warp without a group only builds operands)
    const int wg = pw % NWG;
    int n = 0;
    int4 meta = make_int4(0, 0, 0, 0);
    bool ok = true;
    while (cur.s >= 0 && ok) {
      const int te = p.whole ? cur.T : (int)min((long long)cur.T, cur.t + (u1 - u - cur.v)), nt = te - cur.t;
      const long long behind = u + (p.whole ? 1 : cur.v + nt);
      const int part = cur.t > 0 ? 2 * (int)blockIdx.x : te < cur.T ? 2 * (int)blockIdx.x + 1 : -1;
      const int L = cur.L;
      const uint64_t kbase = reinterpret_cast<uint64_t>(p.kv) + size_t(cur.vh / RB) * chunk;
      int e0 = (int)(((long long)cur.t * TILE) >> lbs);
      int32_t ent = ent0, ent_next = load_entries(cur.s, e0 + 32);
      int ti = tn.first;
      // this warp's tiles of the item, below `end`
      auto issue_to = [&](int end) -> bool {
        for (; pw < NWG * S::CPG && ti < end; ti += NWG * S::CPG, tn.step()) {
          const int s = wg * S::NSG + tn.slot, tok0 = (cur.t + ti) * TILE;
          if (tn.count * S::CPG >= S::NSG && !wait_bar(&empty[s], tn.phase ^ 1, abort_flag, KERR_TIMEOUT_EMPTY)) return false;
          while ((tok0 >> lbs) - e0 >= 32) {
            e0 += 32;
            ent = ent_next;
            ent_next = load_entries(cur.s, e0 + 32);
          }
          // (a tile's blocks never straddle two groups of 32 entries: 32 blocks are whole tiles, from a tile's first on)
          // lane q: K codes of the tile's tokens 16 q .. (which lie in one block)
          const int tok = tok0 + 16 * (lane & 7);
          int blk = __shfl_sync(0xffffffffu, ent, ((tok >> lbs) - e0) & 31);
          if (blk < 0 || blk >= p.num_blocks) {
            if (tok < L) atomicExch(&g_kernel_error, (int)KERR_BAD_BLOCK);
            blk = 0;
          }
          const int off = tok & (bs - 1);
          const uint64_t codes = kbase + size_t(blk) * (2 * plane) + uint32_t(off * ROW);
          const uint32_t to_scales = bs * ROW - off * (ROW - HD / 16);
          const uint32_t slot = sb + s * S::SLOT;
          if (L - tok0 >= TILE) {
#pragma unroll
            for (int q = 0; q < TILE / 16; ++q) {
              const uint64_t src = __shfl_sync(0xffffffffu, codes, q) + src_lane;
#pragma unroll
              for (int ii = 0; ii < 16 / RPI; ++ii) {
                cp_async16(slot + kdst + (16 * q + RPI * ii) * ROW, reinterpret_cast<const uint8_t*>(src) + RPI * ii * ROW, pol);
                cp_async16(slot + vdst + (16 * q + RPI * ii) * ROW, reinterpret_cast<const uint8_t*>(src + plane) + RPI * ii * ROW, pol);
              }
            }
            // scales: 16 bytes hold SPC tokens', a block of 16 tokens HD / 16 such pieces
#pragma unroll
            for (int q = 0; q < TILE / 32 / SPC; ++q) {
              const int piece = 32 * q + lane;
              const uint64_t src = __shfl_sync(0xffffffffu, codes + to_scales, piece / (HD / 16)) + (piece % (HD / 16)) * 16;
              cp_async16(slot + S::KS_OFF + 16 * piece, reinterpret_cast<const uint8_t*>(src), pol);
              cp_async16(slot + S::VS_OFF + 16 * piece, reinterpret_cast<const uint8_t*>(src + plane), pol);
            }
          } else {
            // the sequence ends in this tile: zeros behind it
#pragma unroll
            for (int q = 0; q < TILE / 16; ++q) {
              const uint64_t src = __shfl_sync(0xffffffffu, codes, q) + src_lane;
#pragma unroll
              for (int ii = 0; ii < 16 / RPI; ++ii) {
                const bool valid = tok0 + 16 * q + RPI * ii + lr < L;
                cp_async16_zfill(slot + kdst + (16 * q + RPI * ii) * ROW, reinterpret_cast<const uint8_t*>(src) + RPI * ii * ROW, valid, pol);
                cp_async16_zfill(slot + vdst + (16 * q + RPI * ii) * ROW, reinterpret_cast<const uint8_t*>(src + plane) + RPI * ii * ROW, valid, pol);
              }
            }
#pragma unroll
            for (int q = 0; q < TILE / 32 / SPC; ++q) {
              const int piece = 32 * q + lane;
              const uint64_t src = __shfl_sync(0xffffffffu, codes + to_scales, piece / (HD / 16)) + (piece % (HD / 16)) * 16;
              const int bytes = max(0, min(16, (L - tok0 - SPC * piece) * (HD / 16)));
              cp_async16_part(slot + S::KS_OFF + 16 * piece, reinterpret_cast<const uint8_t*>(src), bytes, pol);
              cp_async16_part(slot + S::VS_OFF + 16 * piece, reinterpret_cast<const uint8_t*>(src + plane), bytes, pol);
            }
          }
          cp_async_arrive_noinc(&full[s]);
        }
        return true;
      };
      // the first tiles go out before the operand is built
      if (n == 0 && !issue_to(min(nt, NWG * S::CPG))) break;
      const int qb = n & 1;
      if (n >= 2 && !wait_bar(&qempty[qb], ((n >> 1) - 1) & 1, abort_flag, KERR_TIMEOUT_EMPTY)) break;
      // ---- query operand (the second row block by the first one's code: code that runs once per item has to be fetched)
#pragma unroll 1
      for (int h = 0; h < NT; ++h) {
        const uint4 qw = NT > 1 && h ? qv[NT - 1] : qv[0];
        const uint32_t ws[4] = {qw.x, qw.y, qw.z, qw.w};
        float x[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[2 * k] = __uint_as_float(ws[k] << 16);
          x[2 * k + 1] = __uint_as_float(ws[k] & 0xffff0000u);
        }
        float amax = 0.f;
        bool finite = true;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          amax = fmaxf(amax, fabsf(x[k]));
          finite = finite && fabsf(x[k]) < INFINITY;
        }
        // rows with a value that is not finite give NaN through their factor
        const unsigned fin = __ballot_sync(0xffffffffu, finite);
        const bool row_ok = ((fin >> (lane & 16)) & 0xffffu) == 0xffffu;
        if (!row_ok) amax = 0.f;
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));      // of 16 dims
        // exponent eb that puts the 16 dims' largest into [2, 4]: amax <= 2^(eb + 2), amax >= 2^(eb + 1); the row's
        // largest exponent er
        const uint32_t ab = __float_as_uint(amax);
        const int eb = ab == 0 ? -200 : int(ab >> 23) - 128 + ((ab & 0x7fffffu) != 0 ? 0 : -1);   // (subnormals as 2^-126)
        int er = eb;
#pragma unroll
        for (int sh = 2; sh < 16; sh <<= 1) er = max(er, __shfl_xor_sync(0xffffffffu, er, sh));
        const bool zero = er == -200;
        if (zero) er = 0;
        const int rel = max(eb - er, -17 + 3 * (PASSES - 1));           // scales 2^8 .. 2^-9, those of the last pass too
        // x 2^-(er + rel), in two factors that are floats
        const int sh = -(er + rel), s1 = max(-126, min(126, sh)), s2 = sh - s1;
        const float up = __uint_as_float(uint32_t(127 + s1) << 23), up2 = __uint_as_float(uint32_t(127 + s2) << 23);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = row_ok ? x[k] * up * up2 : 0.f;
        uint32_t words[QT];
#pragma unroll
        for (int term = 0; term < QT; ++term) {
          words[term] = 0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t code = f32x2_to_e2m1x2(x[2 * k], x[2 * k + 1]);
            words[term] |= code << (8 * k);
            if (term < QT - 1) {
              // (x - code) 8, the residual
              const uint32_t back = e2m1x2_to_f16x2<0>(code);
              x[2 * k] = fmaf(-8.f, f16_lo_to_f32(back), 8.f * x[2 * k]);
              x[2 * k + 1] = fmaf(-8.f, f16_hi_to_f32(back), 8.f * x[2 * k + 1]);
            }
          }
        }
        if (h16 < HD / 8) {
#pragma unroll
          for (int term = 0; term < QT; ++term) {
            const int pass = term % PASSES, col = 8 * CG * h + 8 * (term / PASSES) + qrow;
            const int ch = HD == 128 ? (h16 >> 2) ^ ((col >> 1) & 3) : (h16 >> 2) ^ ((col >> 2) & 1);
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(sb + S::qOff + qb * S::qBytes + (pass * NQ + col) * ROW + 16 * ch + 4 * (h16 & 3)),
                         "r"(words[term]) : "memory");
          }
          // their scales 2^(rel + 8 - 3 pass), a byte per 16 dims
          if ((h16 & 1) == 0) {
#pragma unroll
            for (int term = 0; term < QT; ++term) {
              const int pass = term % PASSES, es = rel + 8 - 3 * pass, col = 8 * CG * h + 8 * (term / PASSES) + qrow;
              sts8(sb + S::qsOff + ((qb * PASSES + pass) * KS + (h16 >> 3)) * 512 + (col & 31) * 16 + (col >> 5) * 4 + ((h16 >> 1) & 3),
                   es >= -6 ? uint32_t(es + 7) << 3 : 1u << (es + 9));
            }
          }
        }
        if (h16 == 0) {
          // the row's factor takes 2^(er - 8) (past 2^+-252 it is 0 or infinite in any case); of a row of zeros it is 0, or NaN
          // where the scales are not finite
          const int a = er - 8 + base_exp, a1 = max(-126, min(126, a)), a2 = max(-126, min(126, a - a1));
          const float f = base * (zero ? 0.f : __uint_as_float(uint32_t(127 + a1) << 23)) * __uint_as_float(uint32_t(127 + a2) << 23);
          const bool used = 16 * (cur.vh % RB) + qrow + 8 * h < p.qg;
          stsf(sb + S::cOff + 4 * (qb * R + 8 * h + qrow), !row_ok ? __int_as_float(0x7fffffff) : used ? f : 0.f);
        }
      }
      if (pt == 0) {
        sts_i4(sb + S::infoOff + 64 * qb, make_int4(L, cur.t, nt, part));
        sts_i4(sb + S::infoOff + 64 * qb + 16, make_int4(cur.s, cur.vh, 0, 0));
      }
      fence_proxy_async();
      __syncwarp();
      arrive_if(lane == 0, &qfull[qb]);
      ++n;
      if (cur.t == 0 && te < cur.T) {
        // begins here and goes on: the pieces are this CTA's and those of the ranges up to the sequence's last unit
        const long long last = u + cur.v + cur.T - 1, head = rem * (per + 1);
        const long long cta = last < head ? div_nonneg(last, per + 1) : rem + div_nonneg(last - head, per);
        meta = make_int4((int)cta - (int)blockIdx.x + 1, cur.s, cur.vh, 0);
      }
      const Cursor nxt = next(cur, behind);
      load_q(nxt, qv);
      ent0 = load_entries(nxt.s, (int)(((long long)nxt.t * TILE) >> lbs));
      if (!issue_to(nt)) break;
      tn.item(nt);
      u = behind;
      cur = nxt;
    }
    if (cur.s < 0) {
      // no more items
      const int qb = n & 1;
      if (n < 2 || wait_bar(&qempty[qb], ((n >> 1) - 1) & 1, abort_flag, KERR_TIMEOUT_EMPTY)) {
        if (pt == 0) sts_i4(sb + S::infoOff + 64 * qb, make_int4(0, 0, 0, 0));
        __syncwarp();
        arrive_if(lane == 0, &qfull[qb]);
      }
    }
    if (pt == 0 && !p.whole) p.meta[blockIdx.x] = meta;
    cp_async_wait_all();
  } else {
    // ======================================================== MMA warps, one per consumer group
    all_set();
    const uint32_t tmem = *tmem_slot;
    reg_dec<S::REG_MMA>();
    const int wg = warp - S::WARP_MMA;
    if (wg < NWG) {
    Turn tn(wg, S::NSG, NWG);
    bool ok = true;
    const uint32_t sfb0 = tmem + S::SFB_COL + wg * 2 * PASSES * 4 * KS;
    // descriptors: the low half is the address (plus constants), the high half constant
    constexpr uint32_t OP_HI = desc_hi(8 * ROW, SWZ), SC_HI = desc_hi(128, kSwizzleNone);
    for (int n = 0; ok; ++n) {
      const int qb = n & 1;
      if (!wait_bar(&qfull[qb], (n >> 1) & 1, abort_flag, KERR_TIMEOUT_FULL)) break;
      const int nt = lds_i4(sb + S::infoOff + 64 * qb).z;
      if (nt == 0) break;
      const uint32_t sfb = sfb0 + qb * PASSES * 4 * KS;
      const uint32_t q_lo = desc_lo(sb + S::qOff + qb * S::qBytes, 16);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < PASSES * KS; ++k)
          copy_scales(sfb + 4 * k, desc_lo(sb + S::qsOff + (qb * PASSES * KS + k) * 512, 16), SC_HI);
      }
      for (int i = tn.first; i < nt; i += NWG, tn.step()) {
        const int s = wg * S::NSG + tn.slot, b = 2 * wg + (tn.count & 1);
        if ((tn.count >= 2 && !wait_bar(&sfree[b], ((tn.count >> 1) - 1) & 1, abort_flag, KERR_TIMEOUT_EMPTY)) ||
            !wait_bar(&full[s], tn.phase, abort_flag, KERR_TIMEOUT_FULL)) {
          ok = false;
          break;
        }
        // K's scales in the tensor core's order: 16 bytes are those of tokens i, i + 32, i + 64 and i + 96
        {
          const uint32_t ksm = sb + s * S::SLOT + S::KS_OFF;
          uint32_t d[4][KS];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if constexpr (KS == 2) {
              const uint2 e = lds64(ksm + 8 * (32 * q + lane));
              d[q][0] = e.x;
              d[q][1] = e.y;
            } else {
              d[q][0] = lds32(ksm + 4 * (32 * q + lane));
            }
          }
          __syncwarp();
#pragma unroll
          for (int k = 0; k < KS; ++k) sts_i4(ksm + 512 * k + 16 * lane, make_int4(d[0][k], d[1][k], d[2][k], d[3][k]));
        }
        fence_proxy_async();     // these and the copied bytes (generic proxy) become visible to the tensor core
        __syncwarp();
        tc_fence_after();
        if (elect_one()) {
          const uint32_t k_lo = desc_lo(sb + s * S::SLOT, 16), sfa = tmem + S::SFA_COL + b * 4 * KS;
#pragma unroll
          for (int k = 0; k < KS; ++k) copy_scales(sfa + 4 * k, k_lo + (S::KS_OFF + 512 * k) / 16, SC_HI);
#pragma unroll
          for (int pass = 0; pass < PASSES; ++pass)
#pragma unroll
            for (int k = 0; k < KS; ++k)
              mma_fp4(tmem + b * NQ, k_lo + 2 * k, q_lo + pass * (NQ * ROW / 16) + 2 * k, OP_HI, idesc_fp4(128, NQ), sfa + 4 * k,
                      sfb + 4 * (pass * KS + k), pass + k);
          umma_commit(&sfull[b]);
          umma_commit(&empty[s]);
        }
        __syncwarp();
      }
      if (!ok) break;
      tn.item(nt);
      if (elect_one()) umma_commit(&qempty[qb]);
      __syncwarp();
    }
    if (elect_one()) {
      // every MMA must finish before the tensor memory is released
      umma_commit(done);
      if (!mbar_try_wait(done, 0)) {
        const unsigned long long t0 = globaltimer();
        while (!mbar_try_wait(done, 0)) {
          if (globaltimer() - t0 > kWaitLimitNs) {
            atomicExch(&g_kernel_error, (int)KERR_TIMEOUT_FULL);
            break;
          }
        }
      }
    }
    __syncwarp();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == S::WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(*tmem_slot, S::TMEM_COLS);
  }
}

// Joins the pieces of the item that begins in range blockIdx.x and continues: out = sum_i
// 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i, row blockIdx.y of its row block; each warp takes
// every NW-th piece. What its first PRE ones hold is read before it is known whether there
// are such pieces (the slots exist), so that few pieces cost one trip to memory.
template <int HD>
__global__ void __launch_bounds__(32 * d4::COMBINE_WARPS) decode4_combine_kernel(const d4::Params p, const int slots) {
  using namespace d4;
  constexpr int NW = COMBINE_WARPS, V = HD / 32, PRE = 2, UN = 4;
  __shared__ float s_o[NW][HD], s_l[NW], s_m[NW];
  const int r = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  struct Piece {
    float2 ml;
    float o[V];
  };
  auto load = [&](int i) -> Piece {
    const int slot = min(i == 0 ? 2 * (int)blockIdx.x + 1 : 2 * ((int)blockIdx.x + i), slots - 1);
    Piece q;
    q.ml = p.part_ml[slot * 16 + r];
    const float* src = p.part_o + ((long long)slot * 16 + r) * HD + V * lane;
    if constexpr (HD == 128) {
      const float4 d = *reinterpret_cast<const float4*>(src);
      q.o[0] = d.x; q.o[1] = d.y; q.o[2] = d.z; q.o[3] = d.w;
    } else {
      const float2 d = *reinterpret_cast<const float2*>(src);
      q.o[0] = d.x; q.o[1] = d.y;
    }
    return q;
  };
  const int4 meta = p.meta[blockIdx.x];
  Piece pre[PRE];
#pragma unroll
  for (int i = 0; i < PRE; ++i) pre[i] = load(warp + NW * i);
  const float vscale = __ldg(p.v_scale);
  const int rbase = 16 * (meta.z % p.row_blocks);
  if (meta.x == 0 || rbase + r >= p.qg) return;
  float M = kNoMax, acc[V], l = 0.f;
#pragma unroll
  for (int d = 0; d < V; ++d) acc[d] = 0.f;
  auto add = [&](const Piece& q) {
    const float now = fmaxf(M, q.ml.x), a = ex2(M - now), f = ex2(q.ml.x - now);
    M = now;
    l = fmaf(f, q.ml.y, l * a);
#pragma unroll
    for (int d = 0; d < V; ++d) acc[d] = fmaf(f, q.o[d], acc[d] * a);
  };
#pragma unroll
  for (int i = 0; i < PRE; ++i)
    if (warp + NW * i < meta.x) add(pre[i]);
  for (int i = warp + NW * PRE; i < meta.x; i += UN * NW) {
    Piece q[UN];
#pragma unroll
    for (int u = 0; u < UN; ++u) q[u] = load(min(i + NW * u, meta.x - 1));
#pragma unroll
    for (int u = 0; u < UN; ++u)
      if (i + NW * u < meta.x) add(q[u]);
  }
#pragma unroll
  for (int d = 0; d < V; ++d) s_o[warp][V * lane + d] = acc[d];
  if (lane == 0) {
    s_l[warp] = l;
    s_m[warp] = M;
  }
  __syncthreads();
  if (threadIdx.x < HD) {
    float top = kNoMax, num = 0.f, den = 0.f;
#pragma unroll
    for (int w = 0; w < NW; ++w) top = fmaxf(top, s_m[w]);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = ex2(s_m[w] - top);
      num = fmaf(f, s_o[w][threadIdx.x], num);
      den = fmaf(f, s_l[w], den);
    }
    const long long row = (long long)meta.y * p.num_kv_heads * p.qg + (meta.z / p.row_blocks) * p.qg + rbase + r;
    reinterpret_cast<__nv_bfloat16*>(p.out)[row * HD + threadIdx.x] = __float2bfloat16_rn(num / den * vscale);
  }
}

cudaError_t take_decode4_error(int* v) {
  const int z = 0;
  const cudaError_t e = cudaMemcpyFromSymbol(v, g_kernel_error, sizeof(int));
  return e == cudaSuccess && *v ? cudaMemcpyToSymbol(g_kernel_error, &z, sizeof(int)) : e;
}

// two slots of 16 rows per CTA, and what begins in it
size_t decode4_workspace_bytes(int, int head_dim) {
  return size_t(d4::MAX_CTAS) * (2 * 16 * (size_t(head_dim) * 4 + 8) + 16);
}

template <int NT, int HD>
static cudaError_t launch_decode4_t(const d4::Params& p, int grid, cudaStream_t stream) {
  using S = d4::Smem<NT, HD>;
  // the roles' register budgets draw on what the kernel is launched with: built with less, it would wait for ever
  static std::atomic<int> kept{0};
  int registers;
  const cudaError_t e = kept_answer(kept, [](int* n) {
    cudaFuncAttributes f;
    const cudaError_t st = cudaFuncGetAttributes(&f, decode4_kernel<NT, HD>);
    *n = st == cudaSuccess ? f.numRegs : 0;
    if (st != cudaSuccess) cudaGetLastError();            // (returned here; nobody else's)
    return st;
  }, registers);
  if (e != cudaSuccess) return e;
  if (registers != S::REG_LAUNCH) return cudaErrorInvalidConfiguration;
  cudaFuncSetAttribute(decode4_kernel<NT, HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::total);
  decode4_kernel<NT, HD><<<grid, S::THREADS, S::total, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_decode4(const Decode4Launch& a, cudaStream_t stream) {
  d4::Params p;
  p.q = static_cast<const uint16_t*>(a.q);
  p.kv = a.kv;
  p.block_table = a.block_table;
  p.seq_lens = a.seq_lens;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.out = static_cast<uint16_t*>(a.out);
  p.part_o = static_cast<float*>(a.workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + size_t(d4::MAX_CTAS) * 2 * 16 * a.head_dim);
  p.meta = reinterpret_cast<int4*>(p.part_ml + size_t(d4::MAX_CTAS) * 2 * 16);
  p.q_stride_seq = a.q_stride_seq;
  p.q_stride_head = a.q_stride_head;
  p.table_stride = a.table_stride;
  p.num_seqs = a.num_seqs;
  p.num_kv_heads = a.num_kv_heads;
  p.qg = a.qg;
  p.row_blocks = (a.qg + 15) / 16;
  p.block_size = a.block_size;
  p.log2_bs = 0;
  while ((1 << p.log2_bs) < a.block_size) ++p.log2_bs;
  p.num_blocks = a.num_blocks;
  p.max_blocks = a.max_blocks;
  p.softmax_mant = std::frexp(a.softmax_scale, &p.softmax_exp);
  if (!std::isfinite(a.softmax_scale)) p.softmax_exp = 0;
  // no more CTAs than units there can be
  const long long tiles = ((long long)a.max_blocks * a.block_size + d4::TILE - 1) / d4::TILE;
  p.whole = tiles <= 4;
  const long long units = (p.whole ? 1 : std::min(tiles, 1LL << 20)) * a.num_seqs * a.num_kv_heads * p.row_blocks;
  const int grid = (int)std::min<long long>(units, std::min(a.num_sms, d4::MAX_CTAS));
  const bool one = a.qg <= 8;
  cudaError_t e = a.head_dim == 64 ? (one ? launch_decode4_t<1, 64>(p, grid, stream) : launch_decode4_t<2, 64>(p, grid, stream))
                                   : (one ? launch_decode4_t<1, 128>(p, grid, stream) : launch_decode4_t<2, 128>(p, grid, stream));
  if (e != cudaSuccess || p.whole) return e;
  const dim3 cgrid(grid, std::min(16, a.qg));
  if (a.head_dim == 64) decode4_combine_kernel<64><<<cgrid, 32 * d4::COMBINE_WARPS, 0, stream>>>(p, 2 * grid);
  else decode4_combine_kernel<128><<<cgrid, 32 * d4::COMBINE_WARPS, 0, stream>>>(p, 2 * grid);
  return cudaGetLastError();
}

}  // namespace qpa
