// pagedkv_rope.cu -- C ABI of the rotary calls: rotation alone, the rotating
// append and its backward, and the append into an 8-bit cache (declarations
// and contract in include/pagedkv.h).  No allocation, no synchronisation.
#include <cuda_runtime.h>

#include <climits>

#include "pagedkv.h"
#include "append_q8.cuh"
#include "host.cuh"
#include "rope.cuh"

namespace {

using namespace pkv;

bool rope_freq(RopeFreq *f, const pkv_rope_params *r, int D, int inverse) {
  if (!r || !r->inv_freq || r->rotary_dim <= 0 || r->rotary_dim > D || r->rotary_dim % 16 != 0) return false;
  if (!(r->mscale > 0.f) || !(r->mscale < 3.0e38f)) return false;
  f->inv_freq = r->inv_freq;
  f->half = r->rotary_dim / 2;
  f->interleaved = r->interleaved ? 1 : 0;
  f->mscale = r->mscale;
  f->sign = inverse ? -1.f : 1.f;
  return true;
}

// One tensor's rows: pointers and strides are fit for 16-byte access.
bool rope_rows(RopeRows *x, const void *src, const int64_t *s, void *dst, const int64_t *d, int heads,
               int rotate) {
  if (!src || !dst || heads <= 0 || !aligned16(src) || !aligned16(dst) || !strides_ok(s) || !strides_ok(d))
    return false;
  x->src = static_cast<const uint16_t *>(src);
  x->dst = static_cast<uint16_t *>(dst);
  x->s0 = s[0];
  x->s1 = s[1];
  x->s2 = s[2];
  x->d0 = d[0];
  x->d1 = d[1];
  x->d2 = d[2];
  x->heads = heads;
  x->rotate = rotate;
  return true;
}

// Warps per token, each with at most kRopePasses passes of its rows, evenly.
void rope_chunks(RopeParams *p) {
  const int rows = p->x[0].heads + p->x[1].heads + p->x[2].heads, per_pass = 32 / (p->D / 16);
  p->chunks = static_cast<int>(ceil_div(rows, kRopePasses * per_pass));
  p->passes = static_cast<int>(ceil_div(ceil_div(rows, p->chunks), per_pass));
}

int launch_rope(RopeParams &p, cudaStream_t s) {
  if (p.tokens == 0) return PKV_OK;
  rope_chunks(&p);
  const int64_t blocks = ceil_div(p.tokens * p.chunks, kRopeWarps) + (p.cu ? 1 : 0);  // (and check_ranges)
  if (blocks > INT32_MAX) return PKV_ERR_ARG;
  rope_kernel<<<static_cast<unsigned>(blocks), kRopeThreads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

// The token layout and the cache's table, common to the appending calls.
int cache_tokens(RopeParams *p, const int32_t *cu, int total_new, int batch, int n_new, int D,
                 int64_t num_blocks, const int32_t *block_table, int64_t bt_stride,
                 int max_blocks_per_seq, const int32_t *seqlens, int block_size, int32_t *err) {
  if (!block_table || !seqlens || batch <= 0 || n_new < 0 || (cu && total_new < 0)) return PKV_ERR_ARG;
  if (D != 64 && D != 128) return PKV_ERR_ARG;
  if (!pow2_in(block_size, 16, 256)) return PKV_ERR_ARG;
  if (num_blocks <= 0 || num_blocks > INT32_MAX || max_blocks_per_seq <= 0 || bt_stride < max_blocks_per_seq)
    return PKV_ERR_ARG;
  p->tokens = cu ? total_new : static_cast<int64_t>(batch) * n_new;
  if (p->tokens > INT32_MAX) return PKV_ERR_ARG;
  p->batch = batch;
  p->n = n_new;
  p->cu = cu;
  p->seqlens = seqlens;
  p->block_table = block_table;
  p->bt_stride = bt_stride;
  p->num_blocks = num_blocks;
  p->max_blocks_per_seq = max_blocks_per_seq;
  p->block_shift = log2i(block_size);
  p->D = D;
  p->err = err;
  return PKV_OK;
}

}  // namespace

extern "C" {

int pkv_rope(const void *q, const int64_t q_strides[3], void *q_out, const int64_t qo_strides[3], int Hq,
             const void *k, const int64_t k_strides[3], void *k_out, const int64_t ko_strides[3], int Hk,
             const int32_t *positions, int batch, int n, int D, const pkv_rope_params *rope, int inverse,
             void *stream) {
  RopeParams p{};
  if (!positions || batch < 0 || n < 0 || (D != 64 && D != 128)) return PKV_ERR_ARG;
  if (!rope_freq(&p.f, rope, D, inverse)) return PKV_ERR_ARG;
  if (!rope_rows(&p.x[0], q, q_strides, q_out, qo_strides, Hq, 1)) return PKV_ERR_ARG;
  if ((k || k_out) && !rope_rows(&p.x[1], k, k_strides, k_out, ko_strides, Hk, 1)) return PKV_ERR_ARG;
  p.tokens = static_cast<int64_t>(batch) * n;
  if (p.tokens > INT32_MAX) return PKV_ERR_ARG;
  p.batch = batch;
  p.n = n;
  p.D = D;
  p.positions = positions;
  return launch_rope(p, static_cast<cudaStream_t>(stream));
}

int pkv_kv_append_rope(const void *q, const int64_t q_strides[3], void *q_out, const int64_t qo_strides[3],
                       int Hq, const void *k_new, const int64_t kn_strides[3], const void *v_new,
                       const int64_t vn_strides[3], const int32_t *cu_seqlens_new, int total_new,
                       void *k_cache, const int64_t k_strides[3], void *v_cache, const int64_t v_strides[3],
                       int64_t num_blocks, const int32_t *block_table, int64_t bt_stride,
                       int max_blocks_per_seq, const int32_t *seqlens, int batch, int n_new, int Hkv, int D,
                       int block_size, const pkv_rope_params *rope, int32_t *err, void *stream) {
  RopeParams p{};
  int rc = cache_tokens(&p, cu_seqlens_new, total_new, batch, n_new, D, num_blocks, block_table, bt_stride,
                        max_blocks_per_seq, seqlens, block_size, err);
  if (rc != PKV_OK) return rc;
  if (!rope_freq(&p.f, rope, D, 0)) return PKV_ERR_ARG;
  if ((q || q_out) && !rope_rows(&p.x[0], q, q_strides, q_out, qo_strides, Hq, 1)) return PKV_ERR_ARG;
  if (!rope_rows(&p.x[1], k_new, kn_strides, k_cache, k_strides, Hkv, 1) ||
      !rope_rows(&p.x[2], v_new, vn_strides, v_cache, v_strides, Hkv, 0))
    return PKV_ERR_ARG;
  p.dst_paged = 1;
  return launch_rope(p, static_cast<cudaStream_t>(stream));
}

int pkv_kv_append_rope_bwd(const void *dq_rot, const int64_t dqr_strides[3], void *dq,
                           const int64_t dq_strides[3], int Hq, const void *dk_cache,
                           const int64_t dkc_strides[3], const void *dv_cache, const int64_t dvc_strides[3],
                           void *dk_new, const int64_t dkn_strides[3], void *dv_new,
                           const int64_t dvn_strides[3], const int32_t *cu_seqlens_new, int total_new,
                           int64_t num_blocks, const int32_t *block_table, int64_t bt_stride,
                           int max_blocks_per_seq, const int32_t *seqlens, int batch, int n_new, int Hkv,
                           int D, int block_size, const pkv_rope_params *rope, int32_t *err, void *stream) {
  RopeParams p{};
  int rc = cache_tokens(&p, cu_seqlens_new, total_new, batch, n_new, D, num_blocks, block_table, bt_stride,
                        max_blocks_per_seq, seqlens, block_size, err);
  if (rc != PKV_OK) return rc;
  if (!rope_freq(&p.f, rope, D, 1)) return PKV_ERR_ARG;
  if ((dq_rot || dq) && !rope_rows(&p.x[0], dq_rot, dqr_strides, dq, dq_strides, Hq, 1)) return PKV_ERR_ARG;
  if (!rope_rows(&p.x[1], dk_cache, dkc_strides, dk_new, dkn_strides, Hkv, 1) ||
      !rope_rows(&p.x[2], dv_cache, dvc_strides, dv_new, dvn_strides, Hkv, 0))
    return PKV_ERR_ARG;
  p.src_paged = 1;
  return launch_rope(p, static_cast<cudaStream_t>(stream));
}

int pkv_kv_append_q8(const void *q, const int64_t q_strides[3], void *q_out, const int64_t qo_strides[3],
                     int Hq, const void *k_new, const int64_t kn_strides[3], const void *v_new,
                     const int64_t vn_strides[3], const int32_t *cu_seqlens_new, int total_new,
                     void *k_cache, const int64_t k_strides[3], void *v_cache, const int64_t v_strides[3],
                     uint8_t *k_scale, const int64_t ks_strides[2], uint8_t *v_scale,
                     const int64_t vs_strides[2], int64_t num_blocks, const int32_t *block_table,
                     int64_t bt_stride, int max_blocks_per_seq, const int32_t *seqlens, int batch, int n_new,
                     int Hkv, int D, int block_size, const pkv_rope_params *rope, int32_t *err,
                     void *stream) {
  AppendQ8Params a{};
  RopeParams &p = a.r;
  int rc = cache_tokens(&p, cu_seqlens_new, total_new, batch, n_new, D, num_blocks, block_table, bt_stride,
                        max_blocks_per_seq, seqlens, block_size, err);
  if (rc != PKV_OK) return rc;
  if (rope && !rope_freq(&p.f, rope, D, 0)) return PKV_ERR_ARG;
  if (q || q_out) {
    if (!rope || !rope_rows(&p.x[0], q, q_strides, q_out, qo_strides, Hq, 1)) return PKV_ERR_ARG;
  }
  // the new rows are sources only; their destinations are bytes
  if (!rope_rows(&a.kv[0], k_new, kn_strides, k_cache, kn_strides, Hkv, 0) ||
      !rope_rows(&a.kv[1], v_new, vn_strides, v_cache, vn_strides, Hkv, 0))
    return PKV_ERR_ARG;
  const int64_t *cst[2] = {k_strides, v_strides}, *sst[2] = {ks_strides, vs_strides};
  uint8_t *scales[2] = {k_scale, v_scale};
  void *caches[2] = {k_cache, v_cache};
  for (int w = 0; w < 2; ++w) {
    if (!cst[w] || !sst[w] || !scales[w]) return PKV_ERR_ARG;
    for (int i = 0; i < 3; ++i)
      if (cst[w][i] <= 0 || cst[w][i] % 16 != 0) return PKV_ERR_ARG;
    if (sst[w][0] <= 0 || sst[w][1] <= 0) return PKV_ERR_ARG;
    a.cache[w] = static_cast<uint8_t *>(caches[w]);
    a.c0[w] = cst[w][0];
    a.c1[w] = cst[w][1];
    a.c2[w] = cst[w][2];
    a.scale[w] = scales[w];
    a.s0[w] = sst[w][0];
    a.s1[w] = sst[w][1];
  }
  a.Hkv = Hkv;
  a.rotate = rope ? 1 : 0;
  if (p.tokens == 0) return PKV_OK;
  a.groups = cu_seqlens_new ? (p.tokens >> p.block_shift) + 2 * static_cast<int64_t>(batch)
                            : batch * dense_groups(n_new, p.block_shift);
  // slots that P pieces per thread cover, and the blocks of threads that a
  // cache block then takes
  const int per_p = kRopeThreads / (D / 16) / 2;
  const int P = block_size <= per_p ? 1 : 2;  // (4: two blocks of threads per SM, a quarter slower)
  a.cluster = static_cast<int>(ceil_div(block_size, P * per_p));
  // one head per block of threads while that fills the device a few times over
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return PKV_ERR_CUDA;
  const int64_t many = 3 * static_cast<int64_t>(sm_count(dev));
  a.heads = 1;
  while (a.heads < Hkv && a.heads < kAppendHeads && a.groups * a.cluster * ceil_div(Hkv, 2 * a.heads) >= many)
    a.heads *= 2;
  a.kv_blocks = a.groups * ceil_div(Hkv, a.heads) * a.cluster;
  p.chunks = 1;
  if (p.x[0].heads) rope_chunks(&p);
  int64_t blocks = a.kv_blocks + (p.x[0].heads ? ceil_div(p.tokens * p.chunks, kRopeWarps) : 0) +
                   (p.cu ? 1 : 0);  // (check_ranges)
  blocks = ceil_div(blocks, a.cluster) * a.cluster;  // (a warp past the last query row returns at once)
  if (blocks > INT32_MAX) return PKV_ERR_ARG;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(a.cluster);
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = &attr;
  cfg.numAttrs = a.cluster > 1 ? 1 : 0;
  auto kern = P == 1 ? append_q8_kernel<1> : append_q8_kernel<2>;
  return cudaLaunchKernelEx(&cfg, kern, a) == cudaSuccess && cudaGetLastError() == cudaSuccess ? PKV_OK
                                                                                           : PKV_ERR_CUDA;
}

}  // extern "C"
