// C-ABI layer: argument validation, workspace carving and kernel launches on
// the caller's stream. Nothing here reads device data or synchronises (except
// qpa_kernel_error, a diagnostic).
#include <cmath>
#include <cstring>

#include "qpa.h"
#include "common.cuh"
#include "qpa_internal.h"

namespace qpa {
__device__ int g_kernel_error = 0;

namespace {

int num_sms_current() {
  static int cache[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64 && cache[dev]) return cache[dev];
  int n = 0;
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (dev >= 0 && dev < 64) cache[dev] = n;
  return n;
}

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// ------------------------------------------------------------------ fp8
struct Fp8Layout {
  size_t o_off, m_off, l_off, total;
};

bool fp8_shape_ok(const qpa_fp8_desc* d) {
  if (d->num_seqs < 0 || d->num_kv_heads < 1 || d->query_group < 1 || d->query_group > 64) return false;
  if (d->head_dim != 128 && d->head_dim != 64) return false;
  const int bs = d->block_size;
  if (!(bs == 16 || bs == 32 || bs == 64 || bs == 128 || bs == 256)) return false;
  if (d->num_blocks < 1 || d->max_blocks_per_seq < 1) return false;
  if (d->out_dtype != QPA_OUT_F32 && d->out_dtype != QPA_OUT_BF16) return false;
  if ((long long)d->max_blocks_per_seq * bs > 0x7fffffffLL) return false;
  return true;
}

// Floats per partial O row: head_dim 64 with up to 8 query rows runs the
// packed two-half kernel, whose partials keep both 64-dim halves (the combine
// adds them).
int fp8_part_dim(const qpa_fp8_desc* d, bool ext) {
  return (!ext && d->head_dim == 64 && d->query_group <= 8) ? 128 : d->head_dim;
}

Fp8Layout fp8_layout(const qpa_fp8_desc* d, int P, bool ext = false) {
  const size_t rows = size_t(d->num_seqs) * d->num_kv_heads * P * d->query_group;
  Fp8Layout L;
  L.o_off = 0;
  L.m_off = round_up(L.o_off + rows * fp8_part_dim(d, ext) * sizeof(float), 256);
  L.l_off = round_up(L.m_off + rows * sizeof(float), 256);
  L.total = round_up(L.l_off + rows * sizeof(float), 256);
  return L;
}

int fp8_check(const void* q, const uint8_t* kv, const int32_t* bt, const int32_t* sl, const float* ks,
              const float* vs, int P, const qpa_fp8_desc* d, const void* ws, size_t wsb) {
  if (!d) return QPA_ERR_NULL;
  if (!fp8_shape_ok(d)) return QPA_ERR_SHAPE;
  if (P < 1) return QPA_ERR_PARTITIONS;
  if ((long long)d->num_seqs * d->num_kv_heads * P * d->query_group > 0x7fffffffLL) return QPA_ERR_SHAPE;
  if (d->num_seqs == 0) return QPA_OK;
  if (!q || !kv || !bt || !sl || !ks || !vs || !ws) return QPA_ERR_NULL;
  const long long sh = d->q_stride_head ? d->q_stride_head : d->head_dim;
  const long long ss = d->q_stride_seq ? d->q_stride_seq : (long long)d->num_kv_heads * d->query_group * d->head_dim;
  if (sh < 0 || ss < 0 || (sh % 8) || (ss % 8)) return QPA_ERR_ALIGN;
  if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(ws, 256)) return QPA_ERR_ALIGN;
  if (wsb < fp8_layout(d, P).total) return QPA_ERR_WORKSPACE;
  return QPA_OK;
}

// ------------------------------------------------------------------ fp8, extended
int fp8x_query_len(const qpa_fp8_ext_desc* d) { return d->query_len > 1 ? d->query_len : 1; }

bool fp8x_shape_ok(const qpa_fp8_ext_desc* d) {
  if (!fp8_shape_ok(&d->base)) return false;
  if (d->query_len < 0 || d->query_len > 4) return false;
  if (fp8x_query_len(d) * d->base.query_group > 64) return false;
  if (d->kv_scale_per_token != 0 && d->kv_scale_per_token != 1) return false;
  return true;
}

Fp8Layout fp8x_layout(const qpa_fp8_ext_desc* d, int P) {
  qpa_fp8_desc rows = d->base;
  rows.query_group = d->base.query_group * fp8x_query_len(d);   // partial rows per (seq, head, partition)
  return fp8_layout(&rows, P, true);
}

// ------------------------------------------------------------------ uq hd256
bool uq_shape_ok(const qpa_uq_desc* d) {
  if (d->num_seqs < 0 || d->num_kv_heads < 1 || d->query_group < 1 || d->query_group > 16) return false;
  if (d->head_dim != 256) return false;
  const int bs = d->block_size;
  if (!(bs == 16 || bs == 32 || bs == 64 || bs == 128 || bs == 256)) return false;
  if (d->num_blocks < 1 || d->max_blocks_per_seq < 1) return false;
  if (d->padded_slot < 272 || d->padded_slot % 16) return false;
  if (d->out_dtype != QPA_OUT_F32 && d->out_dtype != QPA_OUT_BF16) return false;
  if ((long long)d->max_blocks_per_seq * bs > 0x7fffffffLL) return false;
  if (d->flags & ~(QPA_UQ_UE8M0_SCALES | QPA_UQ_Q_HAIRCUT | QPA_UQ_ROT_PERM)) return false;
  return true;
}

// Partial slots per (sequence, KV head): P times the kernel's slots per item.
int uq_slots(const qpa_uq_desc* d, int P) { return P * uq_plan(d->num_kv_heads, d->query_group).jw; }

Fp8Layout uq_layout(const qpa_uq_desc* d, int P) {
  const size_t rows = size_t(d->num_seqs) * d->num_kv_heads * uq_slots(d, P) * d->query_group;
  Fp8Layout L;
  L.o_off = 0;
  L.m_off = round_up(rows * 256 * sizeof(float), 256);
  L.l_off = round_up(L.m_off + rows * sizeof(float), 256);
  L.total = round_up(L.l_off + rows * sizeof(float), 256);
  return L;
}

int uq_check(const void* q, const uint8_t* kv, const float* cent, const int32_t* bt, const int32_t* sl, int P,
             const qpa_uq_desc* d, const void* ws, size_t wsb) {
  if (!d) return QPA_ERR_NULL;
  if (!uq_shape_ok(d)) return QPA_ERR_SHAPE;
  if (P < 1) return QPA_ERR_PARTITIONS;
  if ((long long)d->num_seqs * d->num_kv_heads * P * 8 * d->query_group > 0x7fffffffLL) return QPA_ERR_SHAPE;
  if (d->num_seqs == 0) return QPA_OK;
  if (!q || !kv || !cent || !bt || !sl || !ws) return QPA_ERR_NULL;
  const long long sh = d->q_stride_head ? d->q_stride_head : 256;
  const long long ss = d->q_stride_seq ? d->q_stride_seq : (long long)d->num_kv_heads * d->query_group * 256;
  if (sh < 0 || ss < 0 || (sh % 8) || (ss % 8)) return QPA_ERR_ALIGN;
  if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(ws, 256) || !aligned(cent, 4)) return QPA_ERR_ALIGN;
  if (wsb < uq_layout(d, P).total) return QPA_ERR_WORKSPACE;
  return QPA_OK;
}

// ------------------------------------------------------------------ nvfp4 scorer
int idx_check(const uint8_t* q, const uint8_t* pages, const int32_t* bt, const int32_t* sl, const float* sc,
              const qpa_idx_desc* d) {
  if (!d) return QPA_ERR_NULL;
  if (d->num_reqs < 0 || d->query_len < 1 || d->num_heads < 1 || d->head_dim != 128) return QPA_ERR_SHAPE;
  if (d->query_len * d->num_heads > 16 || d->num_blocks < 1 || d->max_blocks_per_seq < 1 || d->num_cols < 1)
    return QPA_ERR_SHAPE;
  if ((long long)d->num_reqs * d->query_len > 0x7fffffffLL) return QPA_ERR_SHAPE;
  if (d->flags & ~(QPA_IDX_PER_TOKEN | QPA_IDX_SHARED_PAGES)) return QPA_ERR_SHAPE;
  if (d->num_reqs == 0) return QPA_OK;
  if (!q || !pages || !bt || !sl || !sc) return QPA_ERR_NULL;
  const long long ps = d->page_stride ? d->page_stride : 9216;
  const long long qt = d->q_stride_tok ? d->q_stride_tok : (long long)d->num_heads * 128;
  const long long qh = d->q_stride_head ? d->q_stride_head : 128;
  if (ps < 9216) return QPA_ERR_SHAPE;
  if ((ps % 16) || (qt % 16) || (qh % 16) || qt < 0 || qh < 0) return QPA_ERR_ALIGN;
  if (!aligned(q, 16) || !aligned(pages, 16) || !aligned(sc, 4)) return QPA_ERR_ALIGN;
  return QPA_OK;
}

// ------------------------------------------------------------------ serving step
bool block_size_ok(int bs) { return bs == 16 || bs == 32 || bs == 64 || bs == 128 || bs == 256; }

bool overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return an && bn && x < y + bn && y < x + an;
}

struct Span {
  const void* p;
  size_t n;
};
// no output may lie in an input or in another output
template <int NO, int NI>
bool overlap(const Span (&outs)[NO], const Span (&ins)[NI]) {
  for (int o = 0; o < NO; ++o) {
    for (const Span& i : ins)
      if (overlap(outs[o].p, outs[o].n, i.p, i.n)) return true;
    for (int x = 0; x < o; ++x)
      if (overlap(outs[o].p, outs[o].n, outs[x].p, outs[x].n)) return true;
  }
  return false;
}
// bytes from the first to behind the last bf16 of [tokens][heads][dim]
size_t extent(long long tokens, long long heads, int dim, long long stride_tok, long long stride_head) {
  return (size_t(tokens - 1) * stride_tok + size_t(heads - 1) * stride_head + dim) * 2;
}

bool slot_shape_ok(const qpa_slot_desc* d) {
  if (d->num_reqs < 0 || d->num_reqs > kMaxReqs || !block_size_ok(d->block_size) || d->max_blocks_per_seq < 1) return false;
  if (d->num_free < 0 || d->max_tokens < 0 || d->reserved != 0) return false;
  if (d->table_stride != 0 && d->table_stride < d->max_blocks_per_seq) return false;
  if ((long long)d->max_blocks_per_seq * d->block_size > 0x7fffffffLL) return false;
  return true;
}

bool append_shape_ok(const qpa_append_desc* d) {
  if (d->num_tokens < 0 || d->num_kv_heads < 1 || (d->head_dim != 64 && d->head_dim != 128)) return false;
  if (!block_size_ok(d->block_size) || d->num_blocks < 1) return false;
  if (d->kv_scale_per_token != 0 && d->kv_scale_per_token != 1) return false;
  return true;
}

bool chunk_shape_ok(const qpa_chunk_desc* d) {
  if (d->num_reqs < 0 || d->num_tokens < 0 || d->num_kv_heads < 1 || d->query_group < 1 || d->query_group > 64)
    return false;
  if ((d->head_dim != 64 && d->head_dim != 128) || !block_size_ok(d->block_size)) return false;
  if (d->num_blocks < 1 || d->max_blocks_per_seq < 1) return false;
  if (d->kv_scale_per_token != 0 && d->kv_scale_per_token != 1) return false;
  if (d->table_stride != 0 && d->table_stride < d->max_blocks_per_seq) return false;
  if ((long long)d->max_blocks_per_seq * d->block_size > 0x7fffffffLL) return false;
  // the pages' rows are addressed by 32-bit tensor-map coordinates
  if ((long long)2 * d->num_kv_heads * d->block_size > 0x7fffffffLL) return false;
  return true;
}

}  // namespace
}  // namespace qpa

using namespace qpa;

extern "C" {

const char* qpa_status_string(int s) {
  switch (s) {
    case QPA_OK: return "ok";
    case QPA_ERR_NULL: return "null pointer";
    case QPA_ERR_SHAPE: return "unsupported shape";
    case QPA_ERR_ALIGN: return "misaligned pointer or stride";
    case QPA_ERR_WORKSPACE: return "workspace too small";
    case QPA_ERR_PARTITIONS: return "num_partitions must be >= 1";
    case QPA_ERR_CUDA: return "CUDA launch error";
    case QPA_ERR_OVERLAP: return "an output overlaps an input";
    default: return "unknown status";
  }
}

int qpa_version(void) { return 100; }

int qpa_kernel_error(void* stream) {
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return QPA_ERR_CUDA;
  int v = 0, z = 0;
  if (cudaMemcpyFromSymbol(&v, qpa::g_kernel_error, sizeof(int)) != cudaSuccess) return QPA_ERR_CUDA;
  if (cudaMemcpyToSymbol(qpa::g_kernel_error, &z, sizeof(int)) != cudaSuccess) return QPA_ERR_CUDA;
  // the chunk kernel's own word, for this call only if the shared one held nothing
  if (v == 0 && take_chunk_error(&v) != cudaSuccess) return QPA_ERR_CUDA;
  return v;
}

size_t pa_decode_fp8_workspace_size(const qpa_fp8_desc* d, int num_partitions) {
  if (!d || num_partitions < 1 || !fp8_shape_ok(d)) return 0;
  return fp8_layout(d, num_partitions).total;
}

int pa_decode_fp8_partition(const void* q, const uint8_t* kv_cache, const int32_t* block_table,
                            const int32_t* seq_lens, const float* k_scale, const float* v_scale,
                            int num_partitions, const qpa_fp8_desc* d, void* workspace,
                            size_t workspace_bytes, void* stream) {
  int st = fp8_check(q, kv_cache, block_table, seq_lens, k_scale, v_scale, num_partitions, d, workspace,
                     workspace_bytes);
  if (st != QPA_OK || d->num_seqs == 0) return st;
  const Fp8Layout L = fp8_layout(d, num_partitions);
  Fp8Launch a;
  a.q = q;
  a.kv = kv_cache;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.part_o = reinterpret_cast<float*>(ws + L.o_off);
  a.part_m = reinterpret_cast<float*>(ws + L.m_off);
  a.part_l = reinterpret_cast<float*>(ws + L.l_off);
  a.q_stride_head = d->q_stride_head ? d->q_stride_head : d->head_dim;
  a.q_stride_seq = d->q_stride_seq ? d->q_stride_seq : (long long)d->num_kv_heads * d->query_group * d->head_dim;
  a.num_seqs = d->num_seqs;
  a.num_kv_heads = d->num_kv_heads;
  a.qg = d->query_group;
  a.block_size = d->block_size;
  a.num_blocks = d->num_blocks;
  a.max_blocks = d->max_blocks_per_seq;
  a.num_partitions = num_partitions;
  a.softmax_scale = d->softmax_scale != 0.f ? d->softmax_scale : 1.0f / std::sqrt((float)d->head_dim);
  a.head_dim = d->head_dim;
  a.test_flags = d->test_flags;
  a.num_sms = num_sms_current();
  if (a.num_sms <= 0) return QPA_ERR_CUDA;
  return launch_fp8_partition(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? QPA_OK : QPA_ERR_CUDA;
}

int pa_decode_fp8_combine(int num_partitions, void* out, const qpa_fp8_desc* d, const void* workspace,
                          size_t workspace_bytes, void* stream) {
  if (!d) return QPA_ERR_NULL;
  if (!fp8_shape_ok(d)) return QPA_ERR_SHAPE;
  if (num_partitions < 1) return QPA_ERR_PARTITIONS;
  if (d->num_seqs == 0) return QPA_OK;
  if (!out || !workspace) return QPA_ERR_NULL;
  if (!aligned(out, 16) || !aligned(workspace, 256)) return QPA_ERR_ALIGN;
  const Fp8Layout L = fp8_layout(d, num_partitions);
  if (workspace_bytes < L.total) return QPA_ERR_WORKSPACE;
  const uint8_t* ws = static_cast<const uint8_t*>(workspace);
  CombineLaunch c;
  c.part_o = reinterpret_cast<const float*>(ws + L.o_off);
  c.part_m = reinterpret_cast<const float*>(ws + L.m_off);
  c.part_l = reinterpret_cast<const float*>(ws + L.l_off);
  c.out = out;
  c.out_bf16 = d->out_dtype == QPA_OUT_BF16;
  c.num_seqs = d->num_seqs;
  c.num_kv_heads = d->num_kv_heads;
  c.qg = d->query_group;
  c.num_partitions = num_partitions;
  c.d = d->head_dim;
  c.part_d = fp8_part_dim(d, false);
  c.out_stride_head = d->head_dim;
  c.out_stride_seq = (long long)d->num_kv_heads * d->query_group * d->head_dim;
  return launch_combine(c, static_cast<cudaStream_t>(stream)) == cudaSuccess ? QPA_OK : QPA_ERR_CUDA;
}

int pa_decode_fp8(const void* q, const uint8_t* kv_cache, const int32_t* block_table, const int32_t* seq_lens,
                  const float* k_scale, const float* v_scale, int num_partitions, void* out,
                  const qpa_fp8_desc* d, void* workspace, size_t workspace_bytes, void* stream) {
  int st = fp8_check(q, kv_cache, block_table, seq_lens, k_scale, v_scale, num_partitions, d, workspace,
                     workspace_bytes);
  if (st != QPA_OK) return st;
  if (d->num_seqs == 0) return QPA_OK;
  if (!out) return QPA_ERR_NULL;
  if (!aligned(out, 16)) return QPA_ERR_ALIGN;
  st = pa_decode_fp8_partition(q, kv_cache, block_table, seq_lens, k_scale, v_scale, num_partitions, d,
                               workspace, workspace_bytes, stream);
  if (st != QPA_OK) return st;
  return pa_decode_fp8_combine(num_partitions, out, d, workspace, workspace_bytes, stream);
}

size_t pa_decode_fp8_ext_workspace_size(const qpa_fp8_ext_desc* d, int num_partitions) {
  if (!d || num_partitions < 1 || !fp8x_shape_ok(d)) return 0;
  return fp8x_layout(d, num_partitions).total;
}

int pa_decode_fp8_ext(const void* q, const uint8_t* kv_cache, const int32_t* block_table,
                      const int32_t* seq_lens, const float* k_scale, const float* v_scale,
                      int num_partitions, void* out, const qpa_fp8_ext_desc* d, void* workspace,
                      size_t workspace_bytes, void* stream) {
  if (!d) return QPA_ERR_NULL;
  if (!fp8x_shape_ok(d)) return QPA_ERR_SHAPE;
  const qpa_fp8_desc* b = &d->base;
  const int QL = fp8x_query_len(d);
  if (num_partitions < 1) return QPA_ERR_PARTITIONS;
  if ((long long)b->num_seqs * b->num_kv_heads * num_partitions * b->query_group * QL > 0x7fffffffLL)
    return QPA_ERR_SHAPE;
  if (b->num_seqs == 0) return QPA_OK;
  if (!q || !kv_cache || !block_table || !seq_lens || !k_scale || !v_scale || !workspace || !out)
    return QPA_ERR_NULL;
  const long long hq = (long long)b->num_kv_heads * b->query_group;
  const long long sh = b->q_stride_head ? b->q_stride_head : b->head_dim;
  const long long st = d->q_stride_tok ? d->q_stride_tok : hq * b->head_dim;
  const long long ss = b->q_stride_seq ? b->q_stride_seq : QL * hq * b->head_dim;
  if (sh < 0 || st < 0 || ss < 0 || (sh % 8) || (st % 8) || (ss % 8)) return QPA_ERR_ALIGN;
  if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(workspace, 256) || !aligned(out, 16))
    return QPA_ERR_ALIGN;
  if (d->kv_scale_per_token && (!aligned(k_scale, 16) || !aligned(v_scale, 16))) return QPA_ERR_ALIGN;
  const Fp8Layout L = fp8x_layout(d, num_partitions);
  if (workspace_bytes < L.total) return QPA_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  Fp8ExtLaunch a;
  a.q = q;
  a.kv = kv_cache;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.part_o = reinterpret_cast<float*>(ws + L.o_off);
  a.part_m = reinterpret_cast<float*>(ws + L.m_off);
  a.part_l = reinterpret_cast<float*>(ws + L.l_off);
  a.q_stride_seq = ss;
  a.q_stride_tok = st;
  a.q_stride_head = sh;
  a.num_seqs = b->num_seqs;
  a.num_kv_heads = b->num_kv_heads;
  a.qg = b->query_group;
  a.query_len = QL;
  a.per_token = d->kv_scale_per_token;
  a.block_size = b->block_size;
  a.num_blocks = b->num_blocks;
  a.max_blocks = b->max_blocks_per_seq;
  a.num_partitions = num_partitions;
  a.softmax_scale = b->softmax_scale != 0.f ? b->softmax_scale : 1.0f / std::sqrt((float)b->head_dim);
  a.head_dim = b->head_dim;
  a.num_sms = num_sms_current();
  if (a.num_sms <= 0) return QPA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (launch_fp8x_partition(a, s) != cudaSuccess) return QPA_ERR_CUDA;
  Fp8ExtCombineLaunch c;
  c.part_o = a.part_o;
  c.part_m = a.part_m;
  c.part_l = a.part_l;
  c.out = out;
  c.out_bf16 = b->out_dtype == QPA_OUT_BF16;
  c.num_seqs = b->num_seqs;
  c.num_kv_heads = b->num_kv_heads;
  c.qg = b->query_group;
  c.query_len = QL;
  c.num_partitions = num_partitions;
  c.head_dim = b->head_dim;
  c.out_stride_head = b->head_dim;
  c.out_stride_tok = hq * b->head_dim;
  c.out_stride_seq = QL * hq * b->head_dim;
  return launch_fp8x_combine(c, s) == cudaSuccess ? QPA_OK : QPA_ERR_CUDA;
}

size_t uq_decode_hd256_workspace_size(const qpa_uq_desc* d, int num_partitions) {
  if (!d || num_partitions < 1 || !uq_shape_ok(d)) return 0;
  return uq_layout(d, num_partitions).total;
}

int uq_decode_hd256_partition(const void* q, const uint8_t* kv_cache, const float* centroids,
                              const int32_t* block_table, const int32_t* seq_lens, int num_partitions,
                              const qpa_uq_desc* d, void* workspace, size_t workspace_bytes, void* stream) {
  int st = uq_check(q, kv_cache, centroids, block_table, seq_lens, num_partitions, d, workspace, workspace_bytes);
  if (st != QPA_OK || d->num_seqs == 0) return st;
  const Fp8Layout L = uq_layout(d, num_partitions);
  UqLaunch a;
  a.q = q;
  a.kv = kv_cache;
  a.centroids = centroids;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.part_o = reinterpret_cast<float*>(ws + L.o_off);
  a.part_m = reinterpret_cast<float*>(ws + L.m_off);
  a.part_l = reinterpret_cast<float*>(ws + L.l_off);
  a.q_stride_head = d->q_stride_head ? d->q_stride_head : 256;
  a.q_stride_seq = d->q_stride_seq ? d->q_stride_seq : (long long)d->num_kv_heads * d->query_group * 256;
  a.num_seqs = d->num_seqs;
  a.num_kv_heads = d->num_kv_heads;
  a.qg = d->query_group;
  a.block_size = d->block_size;
  a.num_blocks = d->num_blocks;
  a.max_blocks = d->max_blocks_per_seq;
  a.num_partitions = num_partitions;
  a.padded_slot = d->padded_slot;
  a.softmax_scale = d->softmax_scale != 0.f ? d->softmax_scale : 1.0f / 16.0f;
  a.flags = d->flags;
  a.num_sms = num_sms_current();
  if (a.num_sms <= 0) return QPA_ERR_CUDA;
  return launch_uq_partition(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? QPA_OK : QPA_ERR_CUDA;
}

int uq_decode_hd256_combine(int num_partitions, void* out, const qpa_uq_desc* d, const void* workspace,
                            size_t workspace_bytes, void* stream) {
  if (!d) return QPA_ERR_NULL;
  if (!uq_shape_ok(d)) return QPA_ERR_SHAPE;
  if (num_partitions < 1) return QPA_ERR_PARTITIONS;
  if (d->num_seqs == 0) return QPA_OK;
  if (!out || !workspace) return QPA_ERR_NULL;
  if (!aligned(out, 16) || !aligned(workspace, 256)) return QPA_ERR_ALIGN;
  const Fp8Layout L = uq_layout(d, num_partitions);
  if (workspace_bytes < L.total) return QPA_ERR_WORKSPACE;
  const uint8_t* ws = static_cast<const uint8_t*>(workspace);
  CombineLaunch c;
  c.part_o = reinterpret_cast<const float*>(ws + L.o_off);
  c.part_m = reinterpret_cast<const float*>(ws + L.m_off);
  c.part_l = reinterpret_cast<const float*>(ws + L.l_off);
  c.out = out;
  c.out_bf16 = d->out_dtype == QPA_OUT_BF16;
  c.num_seqs = d->num_seqs;
  c.num_kv_heads = d->num_kv_heads;
  c.qg = d->query_group;
  c.num_partitions = uq_slots(d, num_partitions);
  c.d = 256;
  c.out_stride_head = 256;
  c.out_stride_seq = (long long)d->num_kv_heads * d->query_group * 256;
  c.rot_perm = (d->flags & QPA_UQ_ROT_PERM) != 0;
  return launch_uq_combine(c, static_cast<cudaStream_t>(stream)) == cudaSuccess ? QPA_OK : QPA_ERR_CUDA;
}

int uq_decode_hd256(const void* q, const uint8_t* kv_cache, const float* centroids, const int32_t* block_table,
                    const int32_t* seq_lens, int num_partitions, void* out, const qpa_uq_desc* d, void* workspace,
                    size_t workspace_bytes, void* stream) {
  int st = uq_check(q, kv_cache, centroids, block_table, seq_lens, num_partitions, d, workspace, workspace_bytes);
  if (st != QPA_OK) return st;
  if (d->num_seqs == 0) return QPA_OK;
  if (!out) return QPA_ERR_NULL;
  if (!aligned(out, 16)) return QPA_ERR_ALIGN;
  st = uq_decode_hd256_partition(q, kv_cache, centroids, block_table, seq_lens, num_partitions, d, workspace,
                                 workspace_bytes, stream);
  if (st != QPA_OK) return st;
  return uq_decode_hd256_combine(num_partitions, out, d, workspace, workspace_bytes, stream);
}

int nvfp4_index_score(const uint8_t* q, const uint8_t* kv_pages, const int32_t* block_table,
                      const int32_t* seq_lens, float* scores, const qpa_idx_desc* d, void* stream) {
  const int st = idx_check(q, kv_pages, block_table, seq_lens, scores, d);
  if (st != QPA_OK || d->num_reqs == 0) return st;
  IdxLaunch a;
  a.q = q;
  a.pages = kv_pages;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.scores = scores;
  a.page_stride = d->page_stride ? d->page_stride : 9216;
  a.q_stride_tok = d->q_stride_tok ? d->q_stride_tok : (long long)d->num_heads * 128;
  a.q_stride_head = d->q_stride_head ? d->q_stride_head : 128;
  a.s_stride_row = d->s_stride_row ? d->s_stride_row : d->num_cols;
  a.s_stride_head = d->s_stride_head ? d->s_stride_head : (long long)d->num_reqs * d->query_len * a.s_stride_row;
  a.num_reqs = d->num_reqs;
  a.query_len = d->query_len;
  a.num_heads = d->num_heads;
  a.max_blocks = d->max_blocks_per_seq;
  a.num_cols = d->num_cols;
  a.num_blocks = d->num_blocks;
  a.per_token = (d->flags & QPA_IDX_PER_TOKEN) != 0;
  a.shared_pages = (d->flags & QPA_IDX_SHARED_PAGES) != 0;
  a.num_sms = num_sms_current();
  if (a.num_sms <= 0) return QPA_ERR_CUDA;
  return launch_idx_score(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? QPA_OK : QPA_ERR_CUDA;
}

int paged_slot_map(const int32_t* new_lens, const int32_t* cached_lens, int32_t* block_table,
                   const int32_t* free_blocks, int32_t* query_start, int32_t* seq_lens, int64_t* slots,
                   int32_t* positions, int32_t* num_taken, const qpa_slot_desc* d, void* stream) {
  if (!d) return QPA_ERR_NULL;
  if (!slot_shape_ok(d)) return QPA_ERR_SHAPE;
  const bool reqs = d->num_reqs > 0;
  if (!query_start || !num_taken || (reqs && (!new_lens || !cached_lens || !block_table || !seq_lens)))
    return QPA_ERR_NULL;
  if ((d->max_tokens && (!slots || !positions)) || (d->num_free && !free_blocks)) return QPA_ERR_NULL;
  const void* words[] = {new_lens, cached_lens, block_table, free_blocks, query_start, seq_lens, positions, num_taken};
  for (const void* w : words)
    if (!aligned(w, 4)) return QPA_ERR_ALIGN;
  if (!aligned(slots, 8)) return QPA_ERR_ALIGN;
  SlotMapLaunch a;
  a.table_stride = d->table_stride ? d->table_stride : d->max_blocks_per_seq;
  // every CTA of the kernel reads the inputs, so an output written by one of
  // them must not lie in what another still reads
  const size_t nb = size_t(d->num_reqs) * 4, nt = size_t(d->max_tokens);
  const size_t tb = reqs ? (size_t(d->num_reqs - 1) * a.table_stride + d->max_blocks_per_seq) * 4 : 0;
  const Span in[] = {{new_lens, nb}, {cached_lens, nb}, {free_blocks, size_t(d->num_free) * 4}};
  const Span outs[] = {{block_table, tb}, {query_start, nb + 4}, {seq_lens, nb}, {slots, nt * 8}, {positions, nt * 4},
                       {num_taken, 4}};
  if (overlap(outs, in)) return QPA_ERR_OVERLAP;
  a.new_lens = new_lens;
  a.cached_lens = cached_lens;
  a.block_table = block_table;
  a.free_blocks = free_blocks;
  a.query_start = query_start;
  a.seq_lens = seq_lens;
  a.slots = slots;
  a.positions = positions;
  a.num_taken = num_taken;
  a.num_reqs = d->num_reqs;
  a.block_size = d->block_size;
  a.max_blocks = d->max_blocks_per_seq;
  a.num_free = d->num_free;
  a.max_tokens = d->max_tokens;
  a.num_sms = num_sms_current();
  if (a.num_sms <= 0) return QPA_ERR_CUDA;
  return launch_slot_map(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? QPA_OK : QPA_ERR_CUDA;
}

int kv_append_fp8(const void* k, const void* v, uint8_t* kv_cache, const int64_t* slots, float* k_scale,
                  float* v_scale, const qpa_append_desc* d, void* stream) {
  if (!d) return QPA_ERR_NULL;
  if (!append_shape_ok(d)) return QPA_ERR_SHAPE;
  if (d->num_tokens == 0) return QPA_OK;
  if (!k || !v || !kv_cache || !slots || !k_scale || !v_scale) return QPA_ERR_NULL;
  AppendLaunch a;
  const long long row = (long long)d->num_kv_heads * d->head_dim;
  a.k_stride_tok = d->k_stride_tok ? d->k_stride_tok : row;
  a.v_stride_tok = d->v_stride_tok ? d->v_stride_tok : row;
  a.k_stride_head = d->k_stride_head ? d->k_stride_head : d->head_dim;
  a.v_stride_head = d->v_stride_head ? d->v_stride_head : d->head_dim;
  for (long long s : {a.k_stride_tok, a.v_stride_tok, a.k_stride_head, a.v_stride_head})
    if (s < 0 || s % 8) return QPA_ERR_ALIGN;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(kv_cache, 16) || !aligned(slots, 8) || !aligned(k_scale, 4) ||
      !aligned(v_scale, 4))
    return QPA_ERR_ALIGN;
  const size_t scales = size_t(d->num_blocks) * d->num_kv_heads * d->block_size;
  const size_t ks_in = d->kv_scale_per_token ? 0 : 4, ks_out = d->kv_scale_per_token ? scales * 4 : 0;
  const Span in[] = {{k, extent(d->num_tokens, d->num_kv_heads, d->head_dim, a.k_stride_tok, a.k_stride_head)},
                     {v, extent(d->num_tokens, d->num_kv_heads, d->head_dim, a.v_stride_tok, a.v_stride_head)},
                     {slots, size_t(d->num_tokens) * 8}, {k_scale, ks_in}, {v_scale, ks_in}};
  const Span outs[] = {{kv_cache, scales * 2 * d->head_dim}, {k_scale, ks_out}, {v_scale, ks_out}};
  if (overlap(outs, in)) return QPA_ERR_OVERLAP;
  a.k = k;
  a.v = v;
  a.kv = kv_cache;
  a.slots = slots;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.num_tokens = d->num_tokens;
  a.num_kv_heads = d->num_kv_heads;
  a.head_dim = d->head_dim;
  a.block_size = d->block_size;
  a.num_blocks = d->num_blocks;
  a.per_token = d->kv_scale_per_token;
  a.num_sms = num_sms_current();
  if (a.num_sms <= 0) return QPA_ERR_CUDA;
  return launch_append(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? QPA_OK : QPA_ERR_CUDA;
}

size_t pa_chunk_fp8_workspace_size(const qpa_chunk_desc* d) {
  if (!d || !chunk_shape_ok(d)) return 0;
  return chunk_workspace_bytes(d->num_tokens, d->query_group, d->head_dim);
}

int pa_chunk_fp8(const void* q, const uint8_t* kv_cache, const int32_t* block_table, const int32_t* query_start,
                 const int32_t* seq_lens, const float* k_scale, const float* v_scale, void* out,
                 const qpa_chunk_desc* d, void* workspace, size_t workspace_bytes, void* stream) {
  if (!d) return QPA_ERR_NULL;
  if (!chunk_shape_ok(d)) return QPA_ERR_SHAPE;
  if (d->num_reqs == 0 || d->num_tokens == 0) return QPA_OK;
  if (!q || !kv_cache || !block_table || !query_start || !seq_lens || !k_scale || !v_scale || !out || !workspace)
    return QPA_ERR_NULL;
  ChunkLaunch a;
  a.q_stride_head = d->q_stride_head ? d->q_stride_head : d->head_dim;
  a.q_stride_tok = d->q_stride_tok ? d->q_stride_tok : (long long)d->num_kv_heads * d->query_group * d->head_dim;
  a.table_stride = d->table_stride ? d->table_stride : d->max_blocks_per_seq;
  if (a.q_stride_head < 0 || a.q_stride_tok < 0 || (a.q_stride_head % 8) || (a.q_stride_tok % 8)) return QPA_ERR_ALIGN;
  if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(out, 16) || !aligned(workspace, 256)) return QPA_ERR_ALIGN;
  if (!aligned(block_table, 4) || !aligned(query_start, 4) || !aligned(seq_lens, 4)) return QPA_ERR_ALIGN;
  const size_t sa = d->kv_scale_per_token ? 16 : 4;
  if (!aligned(k_scale, sa) || !aligned(v_scale, sa)) return QPA_ERR_ALIGN;
  const size_t ws = chunk_workspace_bytes(d->num_tokens, d->query_group, d->head_dim);
  if (workspace_bytes < ws) return QPA_ERR_WORKSPACE;
  const long long heads = (long long)d->num_kv_heads * d->query_group;
  const size_t scales = size_t(d->num_blocks) * d->num_kv_heads * d->block_size, sn = d->kv_scale_per_token ? scales * 4 : 4;
  const Span in[] = {{q, extent(d->num_tokens, heads, d->head_dim, a.q_stride_tok, a.q_stride_head)},
                     {kv_cache, scales * 2 * d->head_dim},
                     {block_table, (size_t(d->num_reqs - 1) * a.table_stride + d->max_blocks_per_seq) * 4},
                     {query_start, size_t(d->num_reqs) * 4 + 4}, {seq_lens, size_t(d->num_reqs) * 4},
                     {k_scale, sn}, {v_scale, sn}};
  const Span outs[] = {{out, size_t(d->num_tokens) * heads * d->head_dim * 2}, {workspace, ws}};
  if (overlap(outs, in)) return QPA_ERR_OVERLAP;
  a.q = q;
  a.kv = kv_cache;
  a.block_table = block_table;
  a.query_start = query_start;
  a.seq_lens = seq_lens;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.out = out;
  a.workspace = workspace;
  a.num_reqs = d->num_reqs;
  a.num_tokens = d->num_tokens;
  a.num_kv_heads = d->num_kv_heads;
  a.qg = d->query_group;
  a.head_dim = d->head_dim;
  a.block_size = d->block_size;
  a.num_blocks = d->num_blocks;
  a.max_blocks = d->max_blocks_per_seq;
  a.per_token = d->kv_scale_per_token;
  a.softmax_scale = d->softmax_scale != 0.f ? d->softmax_scale : 1.0f / std::sqrt((float)d->head_dim);
  a.num_sms = num_sms_current();
  if (a.num_sms <= 0) return QPA_ERR_CUDA;
  return launch_chunk(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? QPA_OK : QPA_ERR_CUDA;
}

}  // extern "C"
