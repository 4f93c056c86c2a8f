// pagedkv_q8.cu -- C ABI of the attention calls over an 8-bit paged cache
// (declarations and contract in include/pagedkv.h): argument validation, TMA
// tensor maps and launches.  No allocation, no synchronisation.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>
#include <cstring>

#include "pagedkv.h"
#include "attn_rows_q8.cuh"
#include "attn_split_q8.cuh"
#include "host.cuh"

static_assert(PKV_DEVERR_SCALE == pkv::kErrScale, "error bits");

namespace {

using namespace pkv;

// TMA map over one 8-bit cache view, as make_kv_map of pagedkv.cu: the box is
// a whole head row (D bytes) x box_slots slots, swizzled over D bytes.
int make_kv_map_q8(CUtensorMap *map, const void *base, const int64_t st[3], int64_t num_blocks,
                   int block_size, int Hkv, int D, int box_slots, int *head_first) {
  auto enc = encode_fn();
  if (!enc) return PKV_ERR_CUDA;
  // (one head: its axis is never stepped over, its stride says nothing)
  const bool hf = Hkv > 1 && st[2] <= st[1];
  const int64_t head = Hkv > 1 ? st[2] : st[1];
  cuuint64_t dims[4], strides[3];
  cuuint32_t box[4], estr[4] = {1, 1, 1, 1};
  dims[0] = static_cast<cuuint64_t>(D);
  dims[1] = static_cast<cuuint64_t>(hf ? Hkv : block_size);
  dims[2] = static_cast<cuuint64_t>(hf ? block_size : Hkv);
  dims[3] = static_cast<cuuint64_t>(num_blocks);
  strides[0] = static_cast<cuuint64_t>(hf ? head : st[1]);
  strides[1] = static_cast<cuuint64_t>(hf ? st[1] : head);
  strides[2] = static_cast<cuuint64_t>(st[0]);
  box[0] = static_cast<cuuint32_t>(D);
  box[1] = static_cast<cuuint32_t>(hf ? 1 : box_slots);
  box[2] = static_cast<cuuint32_t>(hf ? box_slots : 1);
  box[3] = 1;
  std::memset(map, 0, sizeof(*map));
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(base), dims, strides,
                   box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                   D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return PKV_ERR_LAYOUT;
  *head_first = hf ? 1 : 0;
  return PKV_OK;
}

// Strides of a byte cache usable by the TMA unit: positive multiples of 16.
bool strides16_ok(const int64_t *st) {
  if (!st) return false;
  for (int i = 0; i < 3; ++i)
    if (st[i] <= 0 || st[i] % 16 != 0) return false;
  return true;
}

// K and V stages.  A K tile is done with once its S^T is computed, a V tile is
// held until its P.V, 2700 cycles of softmax later.
template <int D>
constexpr int k_stages() {
  return D == 128 ? 4 : 8;
}
template <int D>
constexpr int v_stages() {
  return D == 128 ? 6 : 10;
}

// One CTA per SM, each with at most kSchedMaxMine units: more units than that
// take more CTAs (the later ones queue; none waits for another).
int q8_grid(const Q8Params &p, int dev) {
  const int sms = sm_count(dev), least = static_cast<int>(ceil_div(p.n_units, kSchedMaxMine));
  return least > sms ? least : p.n_units < sms ? p.n_units : sms;
}

template <int D, int N>
int launch_split_q8(const Q8Params &p, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t s,
                    int dev) {
  constexpr int NSK = k_stages<D>(), NSV = v_stages<D>();
  using C = Q8Cfg<D, N, NSK, NSV>;
  static_assert(C::kSmemBytes <= 232448, "shared memory budget");
  static std::atomic<bool> attr_set[kMaxDevices];
  auto kern = attn_split_q8_kernel<D, N, NSK, NSV>;
  if (dev < 0 || dev >= kMaxDevices || !attr_set[dev].load(std::memory_order_acquire)) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes) !=
        cudaSuccess)
      return PKV_ERR_CUDA;
    if (dev >= 0 && dev < kMaxDevices) attr_set[dev].store(true, std::memory_order_release);
  }
  const int grid = q8_grid(p, dev);
  Q8Params pp = p;
  pp.sched = p.n_units > grid && p.n_units <= C::kSchedScratch ? 1 : 0;  // (one unit each: nothing to deal)
  kern<<<grid, 32 * C::kWarps, C::kSmemBytes, s>>>(pp, mk, mv);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

// Decode-sized rows: the smallest unit that holds them.
int launch_split_q8_rows(int64_t rows, const Q8Params &p, const CUtensorMap &mk, const CUtensorMap &mv,
                         int D, cudaStream_t s, int dev) {
  if (D == 128)
    return rows <= 4   ? launch_split_q8<128, 4>(p, mk, mv, s, dev)
           : rows <= 8 ? launch_split_q8<128, 8>(p, mk, mv, s, dev)
                       : launch_split_q8<128, 16>(p, mk, mv, s, dev);
  return rows <= 4   ? launch_split_q8<64, 4>(p, mk, mv, s, dev)
         : rows <= 8 ? launch_split_q8<64, 8>(p, mk, mv, s, dev)
                     : launch_split_q8<64, 16>(p, mk, mv, s, dev);
}

// The row-major kernel shares out its registers between warpgroups; the
// launch is refused if the build differs from what the shares add up to.
template <int D>
int launch_rows_q8(const Q8Params &p, const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t s, int dev,
                   bool overlap) {
  using C = R8Cfg<D>;
  static_assert(C::kSmemBytes <= 232448, "shared memory budget");
  static std::atomic<bool> attr_set[kMaxDevices];
  auto kern = attn_rows_q8_kernel<D>;
  if (dev < 0 || dev >= kMaxDevices || !attr_set[dev].load(std::memory_order_acquire)) {
    cudaFuncAttributes fa{};
    if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return PKV_ERR_CUDA;
    if (fa.numRegs != kR8LaunchRegs) return PKV_ERR_CUDA;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes) !=
        cudaSuccess)
      return PKV_ERR_CUDA;
    if (dev >= 0 && dev < kMaxDevices) attr_set[dev].store(true, std::memory_order_release);
  }
  const int grid = q8_grid(p, dev);
  Q8Params pp = p;
  pp.sched = p.n_units > grid && p.n_units <= C::kSchedScratch ? 1 : 0;  // (one unit each: nothing to deal)
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kR8Threads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = overlap ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, pp, mk, mv) == cudaSuccess && cudaGetLastError() == cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

// Rows per KV head up to which a request is served by the split kernel (one
// unit of its largest size); its own row count decides, so a row's bits do not
// depend on the requests beside it.
constexpr int kSplitRows = 16;

struct PackedQ8 {
  const int32_t *cu_q;
  int total_q;
  void *fin_out;
  const int64_t *fin_strides;  // (batch, head)
  float *fin_lse;
};

int attn_q8_entry(const void *q, const int64_t q_strides[3], const void *k_cache,
                  const int64_t k_strides[3], const void *v_cache, const int64_t v_strides[3],
                  const uint8_t *k_scale, const int64_t ks_strides[2], const uint8_t *v_scale,
                  const int64_t vs_strides[2], int64_t num_blocks, const int32_t *block_table,
                  int64_t bt_stride, int max_blocks_per_seq, const int32_t *seqlens,
                  int max_seqlen_k, int batch, int seqlen_q, int Hq, int Hkv, int D, int block_size,
                  float scale, int causal, void *out, const int64_t out_strides[3], float *lse,
                  void *workspace, size_t workspace_bytes, int32_t *err, void *stream,
                  const PackedQ8 *pq = nullptr) {
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !seqlens || !out || !lse)
    return PKV_ERR_ARG;
  if (batch <= 0 || seqlen_q <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return PKV_ERR_ARG;
  if (D != 64 && D != 128) return PKV_ERR_ARG;
  if (!pow2_in(block_size, 16, 256)) return PKV_ERR_ARG;
  if (num_blocks <= 0 || num_blocks > INT32_MAX || max_blocks_per_seq <= 0 || bt_stride < max_blocks_per_seq)
    return PKV_ERR_ARG;
  if (max_seqlen_k < 0) return PKV_ERR_ARG;
  if (!strides_ok(q_strides) || !strides16_ok(k_strides) || !strides16_ok(v_strides)) return PKV_ERR_ARG;
  if (!ks_strides || !vs_strides || ks_strides[0] <= 0 || ks_strides[1] <= 0 || vs_strides[0] <= 0 ||
      vs_strides[1] <= 0)
    return PKV_ERR_ARG;
  if (!out_strides || out_strides[0] <= 0 || out_strides[1] <= 0 || out_strides[2] <= 0) return PKV_ERR_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache)) return PKV_ERR_ARG;
  if (!(scale > 0.f) || !(scale <= 8.f)) return PKV_ERR_ARG;
  if (pq && pq->fin_out && (!pq->fin_lse || !pq->fin_strides || pq->fin_strides[0] <= 0 ||
                            pq->fin_strides[1] <= 0))
    return PKV_ERR_ARG;
  const int G = Hq / Hkv;
  const int64_t R = static_cast<int64_t>(G) * seqlen_q;
  const int64_t tokens = pq ? static_cast<int64_t>(pq->total_q) : static_cast<int64_t>(batch) * seqlen_q;
  const int64_t rows = tokens * Hq;
  if (R > INT32_MAX / 2 || rows > INT32_MAX) return PKV_ERR_ARG;
  const bool split_only = R <= kSplitRows;
  const int N = split_only ? (R <= 4 ? 4 : R <= 8 ? 8 : 16) : kRowsPerTile;
  const int64_t S = max_seqlen_k > 0 ? ceil_div(max_seqlen_k, kSplitTokens) : 1;
  const int64_t RT = ceil_div(R, N);
  const int64_t units = static_cast<int64_t>(batch) * S * Hkv * RT;
  if (units > INT32_MAX) return PKV_ERR_ARG;
  const size_t need = pq ? ws_bytes(1, pq->total_q, Hq, D, max_seqlen_k)
                         : ws_bytes(batch, seqlen_q, Hq, D, max_seqlen_k);
  if (!workspace || workspace_bytes < need || !aligned16(workspace)) return PKV_ERR_WORKSPACE;

  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
  const int box_slots = block_size < kTileTokens ? block_size : kTileTokens;
  alignas(64) CUtensorMap mk, mv;
  int hf_k = 0, hf_v = 0;
  int rc = make_kv_map_q8(&mk, k_cache, k_strides, num_blocks, block_size, Hkv, D, box_slots, &hf_k);
  if (rc != PKV_OK) return rc;
  rc = make_kv_map_q8(&mv, v_cache, v_strides, num_blocks, block_size, Hkv, D, box_slots, &hf_v);
  if (rc != PKV_OK) return rc;
  if (hf_k != hf_v) return PKV_ERR_LAYOUT;  // K and V must order head/slot alike

  float *ws_acc = static_cast<float *>(workspace);
  float *ws_ml = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + ws_acc_bytes(rows, S, D));
  Q8Params p{};
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.q_sb = q_strides[0];
  p.q_ss = q_strides[1];
  p.q_sh = q_strides[2];
  p.block_table = block_table;
  p.bt_stride = bt_stride;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.seqlens = seqlens;
  p.batch = batch;
  p.seqlen_q = seqlen_q;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = G;
  p.block_shift = log2i(block_size);
  p.box_slots = box_slots;
  p.box_shift = log2i(box_slots);
  p.map_head_first = hf_k;
  p.n_row_tiles = static_cast<int>(RT);
  p.n_splits = static_cast<int>(S);
  p.n_units = static_cast<int>(units);
  p.max_seqlen_k = max_seqlen_k;
  p.wait_ns = kWaitTimeoutNs;
  p.cscale = scale * 1.4426950408889634f;  // host IEEE multiply, one rounding
  p.causal = causal ? 1 : 0;
  p.ws_acc = ws_acc;
  p.ws_ml = ws_ml;
  p.err = err;
  p.nq_lo = 0;
  p.nq_hi = INT_MAX;
  p.k_sc = k_scale;
  p.v_sc = v_scale;
  p.ksc_sb = ks_strides[0];
  p.ksc_sh = ks_strides[1];
  p.vsc_sb = vs_strides[0];
  p.vsc_sh = vs_strides[1];
  if (pq) {
    p.cu_q = pq->cu_q;
    p.total_q = pq->total_q;
    if (pq->fin_out) {
      p.fin_out = static_cast<__nv_bfloat16 *>(pq->fin_out);
      p.fo_sb = pq->fin_strides[0];
      p.fo_sh = pq->fin_strides[1];
      p.fin_lse = pq->fin_lse;
    }
  }
  p.direct = S == 1 ? 1 : 0;
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.o_sb = out_strides[0];
  p.o_ss = out_strides[1];
  p.o_sh = out_strides[2];
  p.lse = lse;
  p.out_vec = (aligned16(out) && out_strides[0] % 8 == 0 && out_strides[1] % 8 == 0 &&
               out_strides[2] % 8 == 0)
                  ? 1
                  : 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // In a packed call that needs the row-major kernel the short requests take
  // the split kernel, each launch skipping the other's sequences.  How many rows
  // they have is known on the device only, so they share the instantiation that
  // holds the largest.  (One launch for up to 4 rows and one for up to 16, each
  // skipping the other's: 35 + 63 us in place of 66 for that batch.)  The second
  // overlaps the first's end (32 requests, contexts to 4096: 209 -> 201 us; the
  // merge launched to overlap in the same way: 198 -> 202 for 4 x 131072).
  const int small_nq = G <= kSplitRows ? kSplitRows / G : 0;
  const bool both = pq && !split_only && small_nq > 0;
  if (both) {
    Q8Params ps = p;
    ps.nq_lo = 1;
    ps.nq_hi = small_nq;
    ps.n_row_tiles = 1;
    ps.n_units = static_cast<int>(static_cast<int64_t>(batch) * S * Hkv);
    rc = launch_split_q8_rows(static_cast<int64_t>(small_nq) * G, ps, mk, mv, D, s, dev);
    if (rc != PKV_OK) return rc;
    p.nq_lo = small_nq + 1;
  }
  rc = split_only ? launch_split_q8_rows(R, p, mk, mv, D, s, dev)
       : D == 128 ? launch_rows_q8<128>(p, mk, mv, s, dev, both)
                  : launch_rows_q8<64>(p, mk, mv, s, dev, both);
  if (rc != PKV_OK || p.direct) return rc;

  MergeParams m{};
  m.seqlens = seqlens;
  m.seqlen_q = seqlen_q;
  m.Hq = Hq;
  m.n_splits = static_cast<int>(S);
  m.causal = p.causal;
  m.ws_acc = ws_acc;
  m.ws_ml = ws_ml;
  m.out = p.out;
  m.o_sb = out_strides[0];
  m.o_ss = out_strides[1];
  m.o_sh = out_strides[2];
  m.lse = lse;
  m.cu_q = p.cu_q;
  m.batch = batch;
  m.total_q = p.total_q;
  m.fin_out = p.fin_out;
  m.fo_sb = p.fo_sb;
  m.fo_sh = p.fo_sh;
  m.fin_lse = p.fin_lse;
  m.rows = rows;
  m.skip_single = split_only ? 0 : 1;
  m.skip_min_nq = both ? small_nq + 1 : 0;
  m.n_local = static_cast<int>(S);
  return D == 128 ? launch_merge<128, true>(m, rows, s) : launch_merge<64, true>(m, rows, s);
}

}  // namespace

extern "C" {

int pkv_paged_decode_attn_q8(const void *q, const int64_t q_strides[3], const void *k_cache,
                             const int64_t k_strides[3], const void *v_cache,
                             const int64_t v_strides[3], const uint8_t *k_scale,
                             const int64_t ks_strides[2], const uint8_t *v_scale,
                             const int64_t vs_strides[2], int64_t num_blocks,
                             const int32_t *block_table, int64_t bt_stride, int max_blocks_per_seq,
                             const int32_t *seqlens, int max_seqlen_k, int batch, int seqlen_q,
                             int Hq, int Hkv, int D, int block_size, float scale, int causal,
                             void *out, const int64_t out_strides[3], float *lse, void *workspace,
                             size_t workspace_bytes, int32_t *err, void *stream) {
  return attn_q8_entry(q, q_strides, k_cache, k_strides, v_cache, v_strides, k_scale, ks_strides,
                       v_scale, vs_strides, num_blocks, block_table, bt_stride, max_blocks_per_seq,
                       seqlens, max_seqlen_k, batch, seqlen_q, Hq, Hkv, D, block_size, scale, causal,
                       out, out_strides, lse, workspace, workspace_bytes, err, stream);
}

int pkv_paged_prefill_attn_q8(const void *q, const int64_t q_strides[3], const void *k_cache,
                              const int64_t k_strides[3], const void *v_cache,
                              const int64_t v_strides[3], const uint8_t *k_scale,
                              const int64_t ks_strides[2], const uint8_t *v_scale,
                              const int64_t vs_strides[2], int64_t num_blocks,
                              const int32_t *block_table, int64_t bt_stride, int max_blocks_per_seq,
                              const int32_t *seqlens, int max_seqlen_k, int batch, int seqlen_q,
                              int Hq, int Hkv, int D, int block_size, float scale, int causal,
                              void *out, const int64_t out_strides[3], float *lse, void *workspace,
                              size_t workspace_bytes, int32_t *err, void *stream) {
  return attn_q8_entry(q, q_strides, k_cache, k_strides, v_cache, v_strides, k_scale, ks_strides,
                       v_scale, vs_strides, num_blocks, block_table, bt_stride, max_blocks_per_seq,
                       seqlens, max_seqlen_k, batch, seqlen_q, Hq, Hkv, D, block_size, scale, causal,
                       out, out_strides, lse, workspace, workspace_bytes, err, stream);
}

int pkv_paged_varlen_attn_q8(const void *q, const int64_t q_strides[2], const int32_t *cu_seqlens_q,
                             int total_q, int max_seqlen_q, const void *k_cache,
                             const int64_t k_strides[3], const void *v_cache,
                             const int64_t v_strides[3], const uint8_t *k_scale,
                             const int64_t ks_strides[2], const uint8_t *v_scale,
                             const int64_t vs_strides[2], int64_t num_blocks,
                             const int32_t *block_table, int64_t bt_stride, int max_blocks_per_seq,
                             const int32_t *seqlens, int max_seqlen_k, int batch, int Hq, int Hkv,
                             int D, int block_size, float scale, int causal, void *out,
                             const int64_t out_strides[2], float *lse, void *final_out,
                             const int64_t final_strides[2], float *final_lse, void *workspace,
                             size_t workspace_bytes, int32_t *err, void *stream) {
  if (!q_strides || !out_strides || !cu_seqlens_q || total_q <= 0 || max_seqlen_q <= 0)
    return PKV_ERR_ARG;
  const int64_t qs[3] = {q_strides[0], q_strides[0], q_strides[1]};
  const int64_t os[3] = {out_strides[0], out_strides[0], out_strides[1]};
  const PackedQ8 pq{cu_seqlens_q, total_q, final_out, final_strides, final_lse};
  return attn_q8_entry(q, qs, k_cache, k_strides, v_cache, v_strides, k_scale, ks_strides, v_scale,
                       vs_strides, num_blocks, block_table, bt_stride, max_blocks_per_seq, seqlens,
                       max_seqlen_k, batch, max_seqlen_q, Hq, Hkv, D, block_size, scale, causal, out,
                       os, lse, workspace, workspace_bytes, err, stream, &pq);
}

}  // extern "C"
