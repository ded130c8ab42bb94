// C ABI of the MSA hot path: host-side argument checks, TMA tensor-map
// encoding and kernel dispatch.  Every call validates first and enqueues on
// the caller's stream; nothing here allocates, frees or synchronises.
#include <cudaTypedefs.h>

#include <cmath>
#include <cstring>
#include <mutex>

#include "common.cuh"
#include "layer_args.cuh"

namespace msa {
cudaError_t launch_index_score_prefill(const CUtensorMap&, const CUtensorMap&, int, int64_t,
                                       int64_t, int64_t, int32_t, int32_t, float*, int64_t,
                                       int32_t*, cudaStream_t);
cudaError_t launch_index_score_decode(const CUtensorMap&, const void*, int64_t, int64_t,
                                      int64_t, int64_t, int32_t, float*, int64_t, int32_t*,
                                      cudaStream_t);
cudaError_t launch_topk_blocks(const float*, int64_t, int64_t, int64_t, int64_t, int32_t*,
                               cudaStream_t);
size_t block_lists_workspace(int64_t, int64_t, int64_t, int64_t);
cudaError_t launch_block_lists(const int32_t*, int64_t, int64_t, int64_t, int64_t, int64_t,
                               int32_t*, int32_t*, int32_t*, int64_t, void*, int32_t*,
                               cudaStream_t);
cudaError_t launch_sparse_attn(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                               const CUtensorMap&, const CUtensorMap&, const void*, int64_t,
                               int64_t, int64_t, const int32_t*, const int32_t*, int64_t,
                               int64_t, int64_t, int64_t, int32_t, int32_t, int32_t, int32_t,
                               float, float*, void*, bool, int32_t*, cudaStream_t);
cudaError_t launch_sparse_attn_decode(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                      const int32_t*, const int32_t*, int64_t, int64_t, int64_t,
                                      int32_t, int32_t, int32_t, float, float*, float*, int32_t*,
                                      cudaStream_t);
size_t recall_workspace(int64_t, int32_t, int32_t, int32_t);
cudaError_t launch_selection_recall(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                    const int64_t*, int64_t, const void*, int64_t, int64_t,
                                    int64_t, int64_t, int64_t, int64_t, int32_t, int32_t,
                                    int32_t, int32_t, int32_t, float, const int32_t*, float*,
                                    int64_t, float*, float*, float*, float*, void*, int32_t*,
                                    cudaStream_t);
cudaError_t launch_sparse_attn_bwd(const CUtensorMap&, const CUtensorMap&, const void*, int64_t,
                                   int64_t, int64_t, const void*, int64_t, int64_t, int64_t,
                                   const void*, int64_t, int64_t, int64_t, const float*,
                                   const int32_t*, const int32_t*, int64_t, int64_t, int64_t,
                                   int64_t, int64_t, int32_t, int32_t, int32_t, int32_t, float,
                                   float*, float*, float*, float*, float*, int32_t*,
                                   cudaStream_t);
size_t token_select_workspace(int64_t, int32_t, int64_t);
cudaError_t launch_token_select_attention(const CUtensorMap&, const int64_t*, int64_t,
                                          const void*, int64_t, int64_t, int64_t, const void*,
                                          int64_t, int64_t, int64_t, const void*, int64_t,
                                          int64_t, int64_t, const void*, int64_t, int64_t,
                                          int64_t, int64_t, int64_t, int64_t, int64_t, int32_t,
                                          int32_t, int32_t, int32_t, float, int64_t, int32_t*,
                                          float*, float*, void*, int32_t*, cudaStream_t);
cudaError_t launch_index_score_e4m3(const CUtensorMap&, const CUtensorMap&, int64_t, int64_t,
                                   int64_t, int32_t, int32_t, float*, int64_t, const float*,
                                   const float*, int32_t*, cudaStream_t);
cudaError_t launch_quantize_e4m3(const void*, int64_t, void*, float*, cudaStream_t);
uint64_t set_attn_wait_limit(uint64_t);
cudaError_t launch_norm_rope(NormRopeArgs, int32_t, bool, bool, cudaStream_t);
size_t norm_rope_bwd_workspace(int32_t);
cudaError_t launch_norm_rope_bwd(NormRopeBwdArgs, int32_t, bool, bool, float*, float*,
                                 cudaStream_t);
size_t paged_decode_workspace(int64_t, int32_t);
int64_t paged_decode_max_batch();
int32_t paged_decode_tile();
cudaError_t launch_paged_decode(const CUtensorMap&, const CUtensorMap&, PagedDecodeArgs, void*,
                                cudaStream_t);
cudaError_t launch_window_attn_fwd(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                   const CUtensorMap&, const CUtensorMap&, const WindowArgs&,
                                   cudaStream_t);
size_t window_attn_bwd_workspace(const WindowArgs&);   // 0: too many work items
cudaError_t launch_window_attn_bwd(const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                   const CUtensorMap&, const CUtensorMap&, const CUtensorMap&,
                                   WindowArgs, void*, cudaStream_t);
cudaError_t launch_merge(const int32_t*, const float*, const void*, bool, void*, float*,
                         int64_t, int64_t, int32_t, int32_t, int64_t, int32_t*, cudaStream_t);
}  // namespace msa

namespace {

constexpr int64_t kMaxBlocks = 50000;   // shared-memory histogram bound of the inversion

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }
bool is_pow2(int64_t x) { return x > 0 && (x & (x - 1)) == 0; }

// Query window of the block->query lists: dims->q_window when positive, else
// the largest power of two W >= 128 whose gathered query rows of one group,
// W * (h_q / h_kv) * 256 bytes, fit in 32 MiB (about a quarter of L2).
int64_t query_window(const msa_dims* d) {
  if (d->q_window > 0) return d->q_window;
  const int64_t R = d->h_q / d->h_kv;
  int64_t w = MSA_BLOCK_TOKENS;
  while (2 * w * R * 256 <= (int64_t(32) << 20)) w *= 2;
  return w;
}

int64_t num_windows(const msa_dims* d) {
  const int64_t w = query_window(d);
  return (d->n_q + w - 1) / w;
}

msa_status check_dims(const msa_dims* d) {
  if (d == nullptr) return MSA_ERR_INVALID_ARG;
  if (d->batch < 1 || d->n_q < 1 || d->n_kv < 1 || d->q_pos0 < 0) return MSA_ERR_INVALID_ARG;
  if (d->q_pos0 + d->n_q > d->n_kv) return MSA_ERR_INVALID_ARG;
  if (d->h_kv < 1 || d->h_q < 1 || d->h_q % d->h_kv != 0) return MSA_ERR_INVALID_ARG;
  if (d->h_kidx != 1 && d->h_kidx != d->h_kv) return MSA_ERR_INVALID_ARG;
  if (!(d->scale > 0.f) || !std::isfinite(d->scale)) return MSA_ERR_INVALID_ARG;
  const int64_t R = d->h_q / d->h_kv;
  if (!is_pow2(R) || R > 16) return MSA_ERR_UNSUPPORTED;
  if (d->d_idx != 64 && d->d_idx != 128) return MSA_ERR_UNSUPPORTED;
  const int64_t nblk = (d->n_kv + MSA_BLOCK_TOKENS - 1) / MSA_BLOCK_TOKENS;
  if (nblk > kMaxBlocks) return MSA_ERR_UNSUPPORTED;
  if (d->n_kv > (int64_t(1) << 31) - 1) return MSA_ERR_UNSUPPORTED;
  if (d->n_q > (int64_t(1) << 26)) return MSA_ERR_UNSUPPORTED;   // entries pack i << 4
  if (d->batch > 65535 || d->batch * d->h_kv > 65535) return MSA_ERR_UNSUPPORTED;
  if (d->n_q / 128 + 1 > 65535) return MSA_ERR_UNSUPPORTED;
  if (d->q_window < 0 || d->q_window % MSA_BLOCK_TOKENS != 0) return MSA_ERR_INVALID_ARG;
  if (d->batch * d->h_kv * num_windows(d) > 65535) return MSA_ERR_UNSUPPORTED;
  return MSA_OK;
}

msa_status check_tensor(const msa_tensor& t) {
  if (t.ptr == nullptr) return MSA_ERR_INVALID_ARG;
  if (!aligned16(t.ptr)) return MSA_ERR_ALIGNMENT;
  if (t.s_batch < 0 || t.s_tok < 0 || t.s_head < 0) return MSA_ERR_INVALID_ARG;
  if ((t.s_batch % 8) || (t.s_tok % 8) || (t.s_head % 8)) return MSA_ERR_ALIGNMENT;
  return MSA_OK;
}

// total (query, selected block) pairs of one (batch, group)
int64_t entries_per_bg(const msa_dims* d) {
  int64_t total = 0;
  // queries with own(t) >= 15 contribute 16; earlier ones own + 1
  const int64_t t0 = d->q_pos0, t1 = d->q_pos0 + d->n_q;   // [t0, t1)
  const int64_t full_from = 15 * MSA_BLOCK_TOKENS;           // first t with own >= 15
  const int64_t a = t0, bnd = std::min(t1, std::max(t0, full_from));
  for (int64_t t = a; t < bnd; ++t) total += t / MSA_BLOCK_TOKENS + 1;
  if (t1 > bnd) total += (t1 - bnd) * MSA_TOPK_BLOCKS;
  return total;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// 4-D bf16 map: dims {inner, d1, d2, d3} with byte strides of d1..d3, box
// {64, b1, b2, 1}, 128-byte swizzle, zero fill out of bounds.
msa_status make_map(CUtensorMap* map, const void* ptr, uint64_t inner, uint64_t d1, uint64_t d2,
                    uint64_t d3, int64_t s1, int64_t s2, int64_t s3, uint32_t b1, uint32_t b2) {
  auto fn = encode_fn();
  if (fn == nullptr) return MSA_ERR_CUDA;
  cuuint64_t dims[4] = {inner, d1, d2, d3};
  cuuint64_t strides[3] = {(cuuint64_t)s1 * 2, (cuuint64_t)s2 * 2, (cuuint64_t)s3 * 2};
  // a dimension of extent 1 still needs a legal stride
  for (int i = 0; i < 3; ++i)
    if (strides[i] == 0) strides[i] = 16;
  cuuint32_t box[4] = {64, b1, b2, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MSA_OK : MSA_ERR_CUDA;
}

// 3-D map over the pieces' rows of 128 values (fp32: 512-byte rows; bf16:
// 256-byte rows) seen as {128 bytes of a row, rows, 128-byte panels of a row},
// box {128 bytes, box_rows, panels}: one store writes box_rows consecutive
// rows (an entry's heads) across `panels` panels, from shared memory staged
// [panel][row][128 B] with the 128-byte swizzle.
msa_status make_map_piece_rows(CUtensorMap* map, void* ptr, uint64_t rows, bool bf16,
                               uint32_t box_rows, uint32_t panels) {
  auto fn = encode_fn();
  if (fn == nullptr) return MSA_ERR_CUDA;
  const uint64_t row_bytes = bf16 ? 256 : 512;
  cuuint64_t dims[3] = {bf16 ? 64u : 32u, rows, row_bytes / 128};
  cuuint64_t strides[2] = {row_bytes, 128};
  cuuint32_t box[3] = {bf16 ? 64u : 32u, box_rows, panels};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                  3, ptr, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MSA_OK : MSA_ERR_CUDA;
}

msa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MSA_OK : MSA_ERR_CUDA; }

// 5-D bf16 view of q [B, n_q, H, 128] for the attention kernel's gather: dims
// {64 columns, H heads, 2 panels of 64 columns, n_q, B} with byte strides
// {head, 128, token, batch}; box {64, 8, 2, 1, 1} = eight heads of one query,
// both panels, 2 KB, landing as [panel][8 rows][128 B] (128-byte swizzle).
msa_status make_map_q_groups(CUtensorMap* map, const msa_dims* d, const msa_tensor& q) {
  auto fn = encode_fn();
  if (fn == nullptr) return MSA_ERR_CUDA;
  cuuint64_t dims[5] = {64, (cuuint64_t)d->h_q, 2, (cuuint64_t)d->n_q, (cuuint64_t)d->batch};
  cuuint64_t strides[4] = {(cuuint64_t)q.s_head * 2, 128, (cuuint64_t)q.s_tok * 2,
                           (cuuint64_t)q.s_batch * 2};
  for (int i = 0; i < 4; ++i)
    if (strides[i] == 0) strides[i] = 16;      // a dimension of extent 1 still needs a stride
  cuuint32_t box[5] = {64, 8, 2, 1, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(q.ptr), dims,
                  strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MSA_OK : MSA_ERR_CUDA;
}

// 4-D uint8 map (e4m3 codes): dims {inner, d1, d2, d3}, byte strides, box
// {128, b1, b2, 1}, 128-byte swizzle, zero fill out of bounds.
msa_status make_map_u8(CUtensorMap* map, const void* ptr, uint64_t inner, uint64_t d1,
                       uint64_t d2, uint64_t d3, int64_t s1, int64_t s2, int64_t s3, uint32_t b1,
                       uint32_t b2) {
  auto fn = encode_fn();
  if (fn == nullptr) return MSA_ERR_CUDA;
  cuuint64_t dims[4] = {inner, d1, d2, d3};
  cuuint64_t strides[3] = {(cuuint64_t)s1, (cuuint64_t)s2, (cuuint64_t)s3};
  for (int i = 0; i < 3; ++i)
    if (strides[i] == 0) strides[i] = 16;
  cuuint32_t box[4] = {128, b1, b2, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(ptr), dims, strides,
                  box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MSA_OK : MSA_ERR_CUDA;
}

msa_status check_tensor_u8(const msa_tensor& t) {
  if (t.ptr == nullptr) return MSA_ERR_INVALID_ARG;
  if (!aligned16(t.ptr)) return MSA_ERR_ALIGNMENT;
  if (t.s_batch < 0 || t.s_tok < 0 || t.s_head < 0) return MSA_ERR_INVALID_ARG;
  if ((t.s_batch % 16) || (t.s_tok % 16) || (t.s_head % 16)) return MSA_ERR_ALIGNMENT;
  return MSA_OK;
}



}  // namespace

namespace msa {
// the dims check of every entry point, for the allocation-free list builder
// (library-internal: hidden like everything but the C ABI)
msa_status validate_dims(const msa_dims* d) { return check_dims(d); }
}  // namespace msa

extern "C" {

int64_t msa_num_blocks(const msa_dims* d) {
  if (d == nullptr || d->n_kv < 1) return 0;
  return (d->n_kv + MSA_BLOCK_TOKENS - 1) / MSA_BLOCK_TOKENS;
}

int64_t msa_num_entries(const msa_dims* d) {
  if (check_dims(d) != MSA_OK) return 0;
  return d->batch * d->h_kv * entries_per_bg(d);
}

int64_t msa_query_window(const msa_dims* d) {
  if (check_dims(d) != MSA_OK) return 0;
  return query_window(d);
}

int64_t msa_num_segments(const msa_dims* d) {
  if (check_dims(d) != MSA_OK) return 0;
  return d->batch * d->h_kv * num_windows(d) * msa_num_blocks(d);
}

msa_status msa_index_score_maxpool(const msa_dims* d, msa_tensor q_idx, msa_tensor k_idx,
                                   float* pooled, int64_t pooled_row_stride, int32_t* dev_err,
                                   void* stream) {
  msa_status s = check_dims(d);
  if (s != MSA_OK) return s;
  if ((s = check_tensor(q_idx)) != MSA_OK) return s;
  if ((s = check_tensor(k_idx)) != MSA_OK) return s;
  if (pooled == nullptr) return MSA_ERR_INVALID_ARG;
  if (!aligned16(pooled)) return MSA_ERR_ALIGNMENT;
  const int64_t nblk = msa_num_blocks(d);
  if (pooled_row_stride < nblk || pooled_row_stride % 4 != 0) return MSA_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int32_t G = d->h_kv;
  if (d->n_q == 1 && d->h_kidx == 1 && d->d_idx == 128 && G <= 8) {
    // k_idx [B, 1, n_kv, 128]: dims {128, n_kv, 1, B}, box {64, 128, 1, 1} (one key block
    // per pair of loads)
    CUtensorMap tk;
    if ((s = make_map(&tk, k_idx.ptr, d->d_idx, d->n_kv, d->h_kidx, d->batch, k_idx.s_tok,
                      k_idx.s_head, k_idx.s_batch, 128, 1)) != MSA_OK)
      return s;
    return from_cuda(msa::launch_index_score_decode(tk, q_idx.ptr, q_idx.s_batch, q_idx.s_head,
                                                    d->batch, d->q_pos0, G, pooled,
                                                    pooled_row_stride, dev_err, st));
  }
  CUtensorMap tq, tk;
  // q_idx [B, n_q, G, d_idx]: dims {d_idx, G, n_q, B}, box {64, 1, 128, 1}
  if ((s = make_map(&tq, q_idx.ptr, d->d_idx, G, d->n_q, d->batch, q_idx.s_head, q_idx.s_tok,
                    q_idx.s_batch, 1, 128)) != MSA_OK)
    return s;
  // k_idx [B, h_kidx, n_kv, d_idx]: dims {d_idx, n_kv, h_kidx, B}, box {64, 256, 1, 1}
  // (two key blocks per load)
  if ((s = make_map(&tk, k_idx.ptr, d->d_idx, d->n_kv, d->h_kidx, d->batch, k_idx.s_tok,
                    k_idx.s_head, k_idx.s_batch, 256, 1)) != MSA_OK)
    return s;
  return from_cuda(msa::launch_index_score_prefill(tq, tk, d->d_idx, d->batch, d->n_q,
                                                   d->q_pos0, G, d->h_kidx, pooled,
                                                   pooled_row_stride, dev_err, st));
}

msa_status msa_topk_blocks(const msa_dims* d, const float* pooled, int64_t pooled_row_stride,
                           int32_t* sel, int32_t* dev_err, void* stream) {
  (void)dev_err;
  msa_status s = check_dims(d);
  if (s != MSA_OK) return s;
  if (pooled == nullptr || sel == nullptr) return MSA_ERR_INVALID_ARG;
  if (!aligned16(pooled) || !aligned16(sel)) return MSA_ERR_ALIGNMENT;
  if (pooled_row_stride < msa_num_blocks(d) || pooled_row_stride % 4 != 0)
    return MSA_ERR_INVALID_ARG;
  const int64_t n_rows = d->batch * d->h_kv * d->n_q;
  return from_cuda(msa::launch_topk_blocks(pooled, pooled_row_stride, n_rows, d->n_q, d->q_pos0,
                                           sel, reinterpret_cast<cudaStream_t>(stream)));
}

size_t msa_block_query_lists_workspace(const msa_dims* d) {
  if (check_dims(d) != MSA_OK) return 0;
  return msa::block_lists_workspace(d->batch * d->h_kv, d->n_q, msa_num_blocks(d),
                                   query_window(d));
}

msa_status msa_build_block_query_lists(const msa_dims* d, const int32_t* sel,
                                       int32_t* blk_offsets, int32_t* entries,
                                       int32_t* entry_pos, void* ws, size_t ws_bytes,
                                       int32_t* dev_err, void* stream) {
  msa_status s = check_dims(d);
  if (s != MSA_OK) return s;
  if (sel == nullptr || blk_offsets == nullptr || entries == nullptr || entry_pos == nullptr ||
      ws == nullptr)
    return MSA_ERR_INVALID_ARG;
  if (!aligned16(sel) || !aligned16(ws)) return MSA_ERR_ALIGNMENT;
  if (ws_bytes < msa_block_query_lists_workspace(d)) return MSA_ERR_WORKSPACE_TOO_SMALL;
  const int64_t total = msa_num_entries(d);
  if (total >= (int64_t(1) << 31)) return MSA_ERR_UNSUPPORTED;
  return from_cuda(msa::launch_block_lists(sel, d->batch * d->h_kv, d->n_q, d->q_pos0,
                                           msa_num_blocks(d), query_window(d), blk_offsets,
                                           entries, entry_pos, total, ws, dev_err,
                                           reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

msa_status sparse_attn_fwd(const msa_dims* d, msa_tensor q, msa_tensor k, msa_tensor v,
                           const int32_t* blk_offsets, const int32_t* entries, float* part_ml,
                           void* part_acc, bool compact, int32_t* dev_err, void* stream) {
  msa_status s = check_dims(d);
  if (s != MSA_OK) return s;
  if ((s = check_tensor(q)) != MSA_OK) return s;
  if ((s = check_tensor(k)) != MSA_OK) return s;
  if ((s = check_tensor(v)) != MSA_OK) return s;
  if (blk_offsets == nullptr || entries == nullptr || part_ml == nullptr || part_acc == nullptr)
    return MSA_ERR_INVALID_ARG;
  if (!aligned16(part_ml) || !aligned16(part_acc)) return MSA_ERR_ALIGNMENT;
  const int64_t nblk = msa_num_blocks(d);
  const int64_t nwin = num_windows(d);
  const int64_t n_seg = d->batch * d->h_kv * nwin * nblk;
  const int64_t total = msa_num_entries(d);
  if (total >= (int64_t(1) << 31)) return MSA_ERR_UNSUPPORTED;
  const int64_t R = d->h_q / d->h_kv;
  // one query per sequence with R <= 8 runs on the warp-level decode kernel,
  // which writes fp32 pieces only
  const bool decode = d->n_q == 1 && R <= 8;
  if (compact && decode) return MSA_ERR_UNSUPPORTED;
  CUtensorMap tk, tv;
  // k, v [B, h_kv, n_kv, 128]: dims {128, n_kv, h_kv, B}, box {64, 128, 1, 1}
  if ((s = make_map(&tk, k.ptr, MSA_HEAD_DIM, d->n_kv, d->h_kv, d->batch, k.s_tok, k.s_head,
                    k.s_batch, 128, 1)) != MSA_OK)
    return s;
  if ((s = make_map(&tv, v.ptr, MSA_HEAD_DIM, d->n_kv, d->h_kv, d->batch, v.s_tok, v.s_head,
                    v.s_batch, 128, 1)) != MSA_OK)
    return s;
  // part_acc [entries, R, 128] as rows of 128-byte panels; for R >= 8 a
  // warp's 32 adjacent rows are written by TMA stores of 32 rows x 2 panels
  // (fp32: half rows; bf16: whole rows), a partly covered warp's by 8-row,
  // one-panel stores
  CUtensorMap to, to8, tq;
  std::memset(&to, 0, sizeof(to));
  std::memset(&to8, 0, sizeof(to8));
  std::memset(&tq, 0, sizeof(tq));
  if (decode) {
    // one query per sequence: warp-level tiles, heads as the 8-wide side.
    // q [B, 1, H, 128]: dims {128, H, 1, B}, box {64, R, 1, 1} (the query's heads of a group)
    if ((s = make_map(&tq, q.ptr, MSA_HEAD_DIM, d->h_q, d->n_q, d->batch, q.s_head, q.s_tok,
                      q.s_batch, (uint32_t)R, 1)) != MSA_OK)
      return s;
    return from_cuda(msa::launch_sparse_attn_decode(
        tq, tk, tv, blk_offsets, entries, d->batch * d->h_kv, d->n_q, d->q_pos0, d->h_kv,
        d->h_q, (int32_t)nblk, d->scale, part_ml, reinterpret_cast<float*>(part_acc), dev_err,
        reinterpret_cast<cudaStream_t>(stream)));
  }
  if (R >= 8) {
    // q: one box per group of eight heads of an entry (both 64-column panels)
    if ((s = make_map_q_groups(&tq, d, q)) != MSA_OK) return s;
    const int64_t rows = total * R;
    if (rows >= (int64_t(1) << 31)) return MSA_ERR_UNSUPPORTED;
    s = make_map_piece_rows(&to, part_acc, (uint64_t)rows, compact, 32, 2);
    if (s != MSA_OK) return s;
    s = make_map_piece_rows(&to8, part_acc, (uint64_t)rows, compact, 8, 1);
    if (s != MSA_OK) return s;
  }
  return from_cuda(msa::launch_sparse_attn(
      tq, tk, tv, to, to8, q.ptr, q.s_batch, q.s_tok, q.s_head, blk_offsets, entries, n_seg, total,
      d->n_q, d->q_pos0, d->h_kv, d->h_q, (int32_t)nblk, (int32_t)nwin, d->scale, part_ml,
      part_acc, compact, dev_err, reinterpret_cast<cudaStream_t>(stream)));
}

msa_status merge_partials(const msa_dims* d, const int32_t* entry_pos, const float* part_ml,
                          const void* part_acc, bool compact, void* out, float* lse,
                          int32_t* dev_err, void* stream) {
  msa_status s = check_dims(d);
  if (s != MSA_OK) return s;
  if (entry_pos == nullptr || part_ml == nullptr || part_acc == nullptr || out == nullptr ||
      lse == nullptr)
    return MSA_ERR_INVALID_ARG;
  if (!aligned16(part_ml) || !aligned16(part_acc) || !aligned16(out))
    return MSA_ERR_ALIGNMENT;
  const int64_t n_rows = d->batch * d->n_q * d->h_q;
  return from_cuda(msa::launch_merge(entry_pos, part_ml, part_acc, compact, out, lse, n_rows,
                                     d->n_q, d->h_q, d->h_kv, msa_num_entries(d), dev_err,
                                     reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

msa_status msa_sparse_attn_fwd(const msa_dims* d, msa_tensor q, msa_tensor k, msa_tensor v,
                               const int32_t* blk_offsets, const int32_t* entries,
                               float* part_ml, float* part_acc, int32_t* dev_err,
                               void* stream) {
  return sparse_attn_fwd(d, q, k, v, blk_offsets, entries, part_ml, part_acc, false, dev_err,
                         stream);
}

msa_status msa_sparse_attn_fwd_compact(const msa_dims* d, msa_tensor q, msa_tensor k,
                                       msa_tensor v, const int32_t* blk_offsets,
                                       const int32_t* entries, float* part_ml,
                                       void* part_acc_bf16, int32_t* dev_err, void* stream) {
  return sparse_attn_fwd(d, q, k, v, blk_offsets, entries, part_ml, part_acc_bf16, true,
                         dev_err, stream);
}

msa_status msa_merge_partials(const msa_dims* d, const int32_t* entry_pos, const float* part_ml,
                              const float* part_acc, void* out, float* lse, int32_t* dev_err,
                              void* stream) {
  return merge_partials(d, entry_pos, part_ml, part_acc, false, out, lse, dev_err, stream);
}

msa_status msa_merge_partials_compact(const msa_dims* d, const int32_t* entry_pos,
                                      const float* part_ml, const void* part_acc_bf16,
                                      void* out, float* lse, int32_t* dev_err, void* stream) {
  return merge_partials(d, entry_pos, part_ml, part_acc_bf16, true, out, lse, dev_err, stream);
}

msa_status msa_quantize_e4m3(const void* x, int64_t n, void* codes, float* scale,
                             void* stream) {
  if (n < 0) return MSA_ERR_INVALID_ARG;
  if (scale == nullptr || (n > 0 && (x == nullptr || codes == nullptr))) return MSA_ERR_INVALID_ARG;
  return from_cuda(msa::launch_quantize_e4m3(x, n, codes, scale,
                                             reinterpret_cast<cudaStream_t>(stream)));
}

msa_status msa_index_score_maxpool_e4m3(const msa_dims* d, msa_tensor q_idx8, msa_tensor k_idx8,
                                        const float* scale_q, const float* scale_k,
                                        float* pooled, int64_t pooled_row_stride,
                                        int32_t* dev_err, void* stream) {
  msa_status s = check_dims(d);
  if (s != MSA_OK) return s;
  if (d->d_idx != 128) return MSA_ERR_UNSUPPORTED;   // one 128-byte row per index vector
  if ((s = check_tensor_u8(q_idx8)) != MSA_OK) return s;
  if ((s = check_tensor_u8(k_idx8)) != MSA_OK) return s;
  if (pooled == nullptr || scale_q == nullptr || scale_k == nullptr) return MSA_ERR_INVALID_ARG;
  if (!aligned16(pooled)) return MSA_ERR_ALIGNMENT;
  if (pooled_row_stride < msa_num_blocks(d) || pooled_row_stride % 4 != 0)
    return MSA_ERR_INVALID_ARG;
  CUtensorMap tq, tk;
  // q_idx codes [B, n_q, G, 128]: dims {128, G, n_q, B}, box {128, 1, 128, 1}
  if ((s = make_map_u8(&tq, q_idx8.ptr, 128, d->h_kv, d->n_q, d->batch, q_idx8.s_head,
                       q_idx8.s_tok, q_idx8.s_batch, 1, 128)) != MSA_OK)
    return s;
  // k_idx codes [B, h_kidx, n_kv, 128]: dims {128, n_kv, h_kidx, B}, box {128, 256, 1, 1}
  if ((s = make_map_u8(&tk, k_idx8.ptr, 128, d->n_kv, d->h_kidx, d->batch, k_idx8.s_tok,
                       k_idx8.s_head, k_idx8.s_batch, 256, 1)) != MSA_OK)
    return s;
  return from_cuda(msa::launch_index_score_e4m3(tq, tk, d->batch, d->n_q, d->q_pos0, d->h_kv,
                                                d->h_kidx, pooled, pooled_row_stride, scale_q,
                                                scale_k, dev_err,
                                                reinterpret_cast<cudaStream_t>(stream)));
}

size_t msa_selection_recall_workspace(const msa_dims* d, int64_t n_rows) {
  if (check_dims(d) != MSA_OK || n_rows < 0) return 0;
  return msa::recall_workspace(n_rows, d->h_kv, d->h_q / d->h_kv, (int32_t)msa_num_blocks(d));
}

msa_status msa_selection_recall(const msa_dims* d, msa_tensor q, msa_tensor k, msa_tensor q_idx,
                                msa_tensor k_idx, const int32_t* sel, const int64_t* rows,
                                int64_t n_rows, float* block_mass, int64_t mass_stride,
                                float* recall, float* kl_pq, float* kl_qp, float* lse_full,
                                void* ws,
                                size_t ws_bytes, int32_t* dev_err, void* stream) {
  msa_status s = check_dims(d);
  if (s != MSA_OK) return s;
  if ((s = check_tensor(q)) != MSA_OK) return s;
  if ((s = check_tensor(k)) != MSA_OK) return s;
  if ((s = check_tensor(q_idx)) != MSA_OK) return s;
  if ((s = check_tensor(k_idx)) != MSA_OK) return s;
  if (n_rows < 0) return MSA_ERR_INVALID_ARG;
  if (n_rows == 0) return MSA_OK;
  if (sel == nullptr || rows == nullptr || block_mass == nullptr || recall == nullptr ||
      kl_pq == nullptr || kl_qp == nullptr || ws == nullptr)
    return MSA_ERR_INVALID_ARG;
  if (!aligned16(ws)) return MSA_ERR_ALIGNMENT;
  const int64_t nblk = msa_num_blocks(d);
  const int64_t R = d->h_q / d->h_kv;
  if (R > 8) return MSA_ERR_UNSUPPORTED;            // heads are the 8-wide side of the tiles
  if (mass_stride < nblk) return MSA_ERR_INVALID_ARG;
  if (n_rows * d->h_kv > 0x7FFFFFFF) return MSA_ERR_UNSUPPORTED;
  if (ws_bytes < msa_selection_recall_workspace(d, n_rows)) return MSA_ERR_WORKSPACE_TOO_SMALL;
  CUtensorMap tq, tk, tki;
  // q [B, n_q, H, 128]: box {64, R, 1, 1} (one query's heads of a group)
  if ((s = make_map(&tq, q.ptr, MSA_HEAD_DIM, d->h_q, d->n_q, d->batch, q.s_head, q.s_tok,
                    q.s_batch, (uint32_t)R, 1)) != MSA_OK)
    return s;
  // k [B, h_kv, n_kv, 128] and k_idx [B, h_kidx, n_kv, d_idx]: one 128-token block per box
  if ((s = make_map(&tk, k.ptr, MSA_HEAD_DIM, d->n_kv, d->h_kv, d->batch, k.s_tok, k.s_head,
                    k.s_batch, 128, 1)) != MSA_OK)
    return s;
  if ((s = make_map(&tki, k_idx.ptr, d->d_idx, d->n_kv, d->h_kidx, d->batch, k_idx.s_tok,
                    k_idx.s_head, k_idx.s_batch, 128, 1)) != MSA_OK)
    return s;
  return from_cuda(msa::launch_selection_recall(
      tq, tk, tki, rows, n_rows, q_idx.ptr, q_idx.s_batch, q_idx.s_tok, q_idx.s_head, d->batch,
      d->n_q, d->q_pos0, d->h_kv, d->h_q, d->d_idx, d->h_kidx, (int32_t)nblk, d->scale, sel,
      block_mass, mass_stride, recall, kl_pq, kl_qp, lse_full, ws, dev_err,
      reinterpret_cast<cudaStream_t>(stream)));
}

msa_status msa_sparse_attn_bwd(const msa_dims* d, msa_tensor q, msa_tensor k, msa_tensor v,
                               msa_tensor o, msa_tensor d_o, const float* lse,
                               const int32_t* blk_offsets, const int32_t* entries, float* delta,
                               float* part_dq, float* dq, float* dk, float* dv, int32_t* dev_err,
                               void* stream) {
  msa_status s = check_dims(d);
  if (s != MSA_OK) return s;
  if ((s = check_tensor(q)) != MSA_OK) return s;
  if ((s = check_tensor(k)) != MSA_OK) return s;
  if ((s = check_tensor(v)) != MSA_OK) return s;
  if ((s = check_tensor(o)) != MSA_OK) return s;
  if ((s = check_tensor(d_o)) != MSA_OK) return s;
  if (lse == nullptr || blk_offsets == nullptr || entries == nullptr || delta == nullptr ||
      part_dq == nullptr || dq == nullptr || dk == nullptr || dv == nullptr)
    return MSA_ERR_INVALID_ARG;
  // dq pieces, dk and dv leave in 32-byte stores
  if (!aligned32(part_dq) || !aligned16(dq) || !aligned32(dk) || !aligned32(dv))
    return MSA_ERR_ALIGNMENT;
  const int64_t nblk = msa_num_blocks(d);
  const int64_t total = msa_num_entries(d);
  if (total >= (int64_t(1) << 31)) return MSA_ERR_UNSUPPORTED;
  CUtensorMap tk, tv;
  // k, v [B, h_kv, n_kv, 128]: dims {128, n_kv, h_kv, B}, box {64, 128, 1, 1}
  if ((s = make_map(&tk, k.ptr, MSA_HEAD_DIM, d->n_kv, d->h_kv, d->batch, k.s_tok, k.s_head,
                    k.s_batch, 128, 1)) != MSA_OK)
    return s;
  if ((s = make_map(&tv, v.ptr, MSA_HEAD_DIM, d->n_kv, d->h_kv, d->batch, v.s_tok, v.s_head,
                    v.s_batch, 128, 1)) != MSA_OK)
    return s;
  return from_cuda(msa::launch_sparse_attn_bwd(
      tk, tv, q.ptr, q.s_batch, q.s_tok, q.s_head, o.ptr, o.s_batch, o.s_tok, o.s_head, d_o.ptr,
      d_o.s_batch, d_o.s_tok, d_o.s_head, lse, blk_offsets, entries, total, d->batch, d->n_q,
      d->n_kv, d->q_pos0, d->h_kv, d->h_q, (int32_t)nblk, (int32_t)num_windows(d), d->scale,
      delta, part_dq, dq, dk, dv, dev_err, reinterpret_cast<cudaStream_t>(stream)));
}

size_t msa_token_select_workspace(const msa_dims* d, int64_t n_rows) {
  if (check_dims(d) != MSA_OK || n_rows < 0) return 0;
  return msa::token_select_workspace(n_rows, d->h_kv, d->n_kv);
}

msa_status msa_token_select_attention(const msa_dims* d, msa_tensor q, msa_tensor k,
                                      msa_tensor v, msa_tensor q_idx, msa_tensor k_idx,
                                      const int64_t* rows, int64_t n_rows, int64_t budget,
                                      int32_t* tokens, float* out, float* lse, void* ws,
                                      size_t ws_bytes, int32_t* dev_err, void* stream) {
  msa_status s = check_dims(d);
  if (s != MSA_OK) return s;
  if ((s = check_tensor(q)) != MSA_OK) return s;
  if ((s = check_tensor(k)) != MSA_OK) return s;
  if ((s = check_tensor(v)) != MSA_OK) return s;
  if ((s = check_tensor(q_idx)) != MSA_OK) return s;
  if ((s = check_tensor(k_idx)) != MSA_OK) return s;
  if (n_rows < 0 || budget < 1 || budget > 0x7FFFFFFF) return MSA_ERR_INVALID_ARG;
  if (n_rows == 0) return MSA_OK;
  if (rows == nullptr || tokens == nullptr || out == nullptr || lse == nullptr || ws == nullptr)
    return MSA_ERR_INVALID_ARG;
  if (!aligned16(ws) || !aligned16(out)) return MSA_ERR_ALIGNMENT;
  const int64_t R = d->h_q / d->h_kv;
  if (R > 8) return MSA_ERR_UNSUPPORTED;            // heads are the 8-wide side of the tiles
  if (n_rows * d->h_kv > 0x7FFFFFFF) return MSA_ERR_UNSUPPORTED;
  if (ws_bytes < msa_token_select_workspace(d, n_rows)) return MSA_ERR_WORKSPACE_TOO_SMALL;
  CUtensorMap tki;
  // k_idx [B, h_kidx, n_kv, d_idx]: one 128-token block of 64 dims per box
  if ((s = make_map(&tki, k_idx.ptr, d->d_idx, d->n_kv, d->h_kidx, d->batch, k_idx.s_tok,
                    k_idx.s_head, k_idx.s_batch, 128, 1)) != MSA_OK)
    return s;
  return from_cuda(msa::launch_token_select_attention(
      tki, rows, n_rows, q.ptr, q.s_batch, q.s_tok, q.s_head, q_idx.ptr, q_idx.s_batch,
      q_idx.s_tok, q_idx.s_head, k.ptr, k.s_batch, k.s_tok, k.s_head, v.ptr, v.s_batch, v.s_tok,
      v.s_head, d->batch, d->n_q, d->n_kv, d->q_pos0, d->h_kv, d->h_q, d->d_idx, d->h_kidx,
      d->scale, budget, tokens, out, lse, ws, dev_err, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"

namespace {

msa_status check_norm_rope(const msa_norm_rope_dims* d, const float* w_q, const float* w_k,
                           const float* table, int64_t n_pos, const int64_t* positions) {
  if (d == nullptr) return MSA_ERR_INVALID_ARG;
  if (d->batch < 1 || d->n_tok < 1 || d->pos0 < 0 || d->h_q < 0 || d->h_k < 0)
    return MSA_ERR_INVALID_ARG;
  if (d->h_q == 0 && d->h_k == 0) return MSA_ERR_INVALID_ARG;
  if (!(d->eps >= 0.f) || !std::isfinite(d->eps)) return MSA_ERR_INVALID_ARG;
  if (d->interleaved != 0 && d->interleaved != 1) return MSA_ERR_INVALID_ARG;
  if (d->d != 64 && d->d != 128) return MSA_ERR_UNSUPPORTED;
  if (d->rot < 0 || d->rot > d->d || d->rot % 16 != 0) return MSA_ERR_UNSUPPORTED;
  // token x head counts in 40 bits: every index below fits 64
  if (d->batch > (int64_t(1) << 31) || d->n_tok > (int64_t(1) << 31) || d->h_q > 65535 ||
      d->h_k > 65535 || d->batch * d->n_tok > (int64_t(1) << 31))
    return MSA_ERR_UNSUPPORTED;
  if (n_pos < 0 || (d->rot > 0 && table == nullptr)) return MSA_ERR_INVALID_ARG;
  if (positions == nullptr && d->pos0 > n_pos - d->n_tok) return MSA_ERR_INVALID_ARG;
  if (!aligned16(table) || !aligned16(w_q) || !aligned16(w_k)) return MSA_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(positions) & 7u) != 0) return MSA_ERR_ALIGNMENT;
  return MSA_OK;
}

msa_status check_paged(const msa_paged_kv* c) {
  if (c == nullptr || c->k == nullptr || c->v == nullptr || c->block_table == nullptr)
    return MSA_ERR_INVALID_ARG;
  if (c->n_pages < 1 || c->table_stride < 1 || c->h_kv < 1) return MSA_ERR_INVALID_ARG;
  if (c->s_page < 0 || c->s_tok < 0 || c->s_head < 0) return MSA_ERR_INVALID_ARG;
  // tokens, heads and pages of a cache are places of their own
  if (c->s_tok == 0 || (c->s_head == 0 && c->h_kv > 1) || (c->s_page == 0 && c->n_pages > 1))
    return MSA_ERR_INVALID_ARG;
  if (!is_pow2(c->page_size) || c->page_size < 16 || c->n_pages > 0x7FFFFFFF)
    return MSA_ERR_UNSUPPORTED;
  if (!aligned16(c->k) || !aligned16(c->v)) return MSA_ERR_ALIGNMENT;
  if ((c->s_page % 8) || (c->s_tok % 8) || (c->s_head % 8)) return MSA_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(c->block_table) & 3u) ||
      (reinterpret_cast<uintptr_t>(c->seq_lens) & 3u))
    return MSA_ERR_ALIGNMENT;
  return MSA_OK;
}

// every (batch, token, head) row has a place of its own
bool rows_apart(const msa_tensor& t, int64_t batch, int64_t tok, int64_t heads) {
  return (t.s_batch > 0 || batch == 1) && (t.s_tok > 0 || tok == 1) &&
         (t.s_head > 0 || heads == 1);
}
// outputs of the norms: checked like inputs, and no two rows in one place
msa_status check_norm_out(const msa_tensor& t, const msa_norm_rope_dims* d, int64_t heads) {
  const msa_status s = check_tensor(t);
  if (s != MSA_OK) return s;
  return rows_apart(t, d->batch, d->n_tok, heads) ? MSA_OK : MSA_ERR_INVALID_ARG;
}
// tensors read through TMA maps, which have no stride of 0
msa_status check_mapped(const msa_tensor& t, int64_t batch, int64_t tok, int64_t heads) {
  const msa_status s = check_tensor(t);
  if (s != MSA_OK) return s;
  return rows_apart(t, batch, tok, heads) ? MSA_OK : MSA_ERR_UNSUPPORTED;
}

// check_tensor for strides in elements of `bytes` bytes
msa_status check_rows(const msa_tensor& t, int bytes) {
  const msa_status s = check_tensor(t);
  if (s == MSA_OK || bytes == 2 || s != MSA_ERR_ALIGNMENT) return s;
  const int64_t e = 16 / bytes;
  if (!aligned16(t.ptr) || t.s_batch % e || t.s_tok % e || t.s_head % e) return MSA_ERR_ALIGNMENT;
  return MSA_OK;
}

msa::NormRopeArgs norm_rope_args(const msa_norm_rope_dims* d, const float* w_q, const float* w_k,
                                 const float* table, int64_t n_pos, const int64_t* positions,
                                 int32_t* dev_err) {
  msa::NormRopeArgs a;
  std::memset(&a, 0, sizeof(a));
  a.w[0] = w_q;
  a.w[1] = w_k;
  a.table = table;
  a.positions = positions;
  a.n_pos = n_pos;
  a.pos0 = d->pos0;
  a.batch = d->batch;
  a.n_tok = d->n_tok;
  a.heads[0] = d->h_q;
  a.heads[1] = d->h_k;
  a.rot = d->rot;
  a.eps = d->eps;
  a.page_size = 1;
  a.err = dev_err;
  return a;
}
void set_src(msa::NormRopeArgs& a, int k, const msa_tensor& t) {
  a.src[k] = reinterpret_cast<const __nv_bfloat16*>(t.ptr);
  a.ss_b[k] = t.s_batch;
  a.ss_t[k] = t.s_tok;
  a.ss_h[k] = t.s_head;
}
void set_dst(msa::NormRopeArgs& a, int k, void* p, int64_t sb, int64_t st, int64_t sh) {
  a.dst[k] = reinterpret_cast<__nv_bfloat16*>(p);
  a.ds_b[k] = sb;
  a.ds_t[k] = st;
  a.ds_h[k] = sh;
}
void set_dst(msa::NormRopeArgs& a, int k, const msa_tensor& t) {
  set_dst(a, k, const_cast<void*>(t.ptr), t.s_batch, t.s_tok, t.s_head);
}

// 5-D bf16 view of a paged cache tensor: {64 columns, page_size tokens, 2 panels,
// heads, pages}; box {64, rows, 2, 1, 1} lands as [panel][rows][128 B]
msa_status make_map_pages(CUtensorMap* map, const void* ptr, const msa_paged_kv* c,
                          uint32_t rows) {
  auto fn = encode_fn();
  if (fn == nullptr) return MSA_ERR_CUDA;
  cuuint64_t dims[5] = {64, (cuuint64_t)c->page_size, 2, (cuuint64_t)c->h_kv,
                        (cuuint64_t)c->n_pages};
  cuuint64_t strides[4] = {(cuuint64_t)c->s_tok * 2, 128, (cuuint64_t)c->s_head * 2,
                           (cuuint64_t)c->s_page * 2};
  for (int i = 0; i < 4; ++i)
    if (strides[i] == 0) strides[i] = 16;      // a dimension of extent 1 still needs a stride
  cuuint32_t box[5] = {64, rows, 2, 1, 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(ptr), dims,
                  strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? MSA_OK : MSA_ERR_CUDA;
}

msa::WindowArgs window_args(const msa_dims* d, int64_t window, int64_t n_sink,
                            const int32_t* kv_len, int32_t* dev_err) {
  msa::WindowArgs a;
  std::memset(&a, 0, sizeof(a));
  a.batch = d->batch;
  a.n_q = d->n_q;
  a.n_kv = d->n_kv;
  a.q_pos0 = d->q_pos0;
  a.window = window;
  a.sink = msa::min64(n_sink, d->n_kv);
  a.G = d->h_kv;
  a.R = d->h_q / d->h_kv;
  a.scale = d->scale;
  a.kv_len = kv_len;
  a.err = dev_err;
  return a;
}

// q-shaped [B, n_q, H, 128] tiles: 128 / R queries x R heads, 64 columns a box
msa_status make_map_rows(CUtensorMap* map, const msa_dims* d, const msa_tensor& t) {
  const int32_t R = d->h_q / d->h_kv;
  return make_map(map, t.ptr, MSA_HEAD_DIM, d->h_q, d->n_q, d->batch, t.s_head, t.s_tok,
                  t.s_batch, (uint32_t)R, (uint32_t)(MSA_BLOCK_TOKENS / R));
}
// k, v [B, h_kv, n_kv, 128]: `keys` keys, 64 columns a box
msa_status make_map_keys(CUtensorMap* map, const msa_dims* d, const msa_tensor& t,
                         uint32_t keys) {
  return make_map(map, t.ptr, MSA_HEAD_DIM, d->n_kv, d->h_kv, d->batch, t.s_tok, t.s_head,
                  t.s_batch, keys, 1);
}

msa_status check_window(const msa_dims* d, int64_t window, int64_t n_sink,
                        const int32_t* kv_len) {
  const msa_status s = check_dims(d);
  if (s != MSA_OK) return s;
  if (window < 0 || n_sink < 0) return MSA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(kv_len) & 3u) != 0) return MSA_ERR_ALIGNMENT;
  return MSA_OK;
}

}  // namespace

extern "C" {

msa_status msa_qk_norm_rope(const msa_norm_rope_dims* d, msa_tensor q, msa_tensor k,
                            const float* w_q, const float* w_k, const float* table,
                            int64_t n_pos, const int64_t* positions, msa_tensor q_out,
                            msa_tensor k_out, int32_t* dev_err, void* stream) {
  msa_status s = check_norm_rope(d, w_q, w_k, table, n_pos, positions);
  if (s != MSA_OK) return s;
  if (d->h_q > 0 && ((s = check_tensor(q)) != MSA_OK ||
                     (s = check_norm_out(q_out, d, d->h_q)) != MSA_OK))
    return s;
  if (d->h_k > 0 && ((s = check_tensor(k)) != MSA_OK ||
                     (s = check_norm_out(k_out, d, d->h_k)) != MSA_OK))
    return s;
  msa::NormRopeArgs a = norm_rope_args(d, w_q, w_k, table, n_pos, positions, dev_err);
  set_src(a, 0, q);
  set_src(a, 1, k);
  set_dst(a, 0, q_out);
  set_dst(a, 1, k_out);
  return from_cuda(msa::launch_norm_rope(a, d->d, d->interleaved != 0, false,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

msa_status msa_qk_norm_rope_paged(const msa_norm_rope_dims* d, msa_tensor q, msa_tensor k,
                                  msa_tensor v, const float* w_q, const float* w_k,
                                  const float* table, int64_t n_pos, const int64_t* positions,
                                  msa_tensor q_out, const msa_paged_kv* cache, int32_t* dev_err,
                                  void* stream) {
  msa_status s = check_norm_rope(d, w_q, w_k, table, n_pos, positions);
  if (s != MSA_OK) return s;
  if (d->d != MSA_HEAD_DIM) return MSA_ERR_UNSUPPORTED;
  if ((s = check_paged(cache)) != MSA_OK) return s;
  if (d->h_k != cache->h_kv) return MSA_ERR_INVALID_ARG;
  if (d->h_q > 0 && ((s = check_tensor(q)) != MSA_OK ||
                     (s = check_norm_out(q_out, d, d->h_q)) != MSA_OK))
    return s;
  if ((s = check_tensor(k)) != MSA_OK) return s;
  if ((s = check_tensor(v)) != MSA_OK) return s;
  msa::NormRopeArgs a = norm_rope_args(d, w_q, w_k, table, n_pos, positions, dev_err);
  set_src(a, 0, q);
  set_src(a, 1, k);
  set_src(a, 2, v);
  set_dst(a, 0, q_out);
  set_dst(a, 1, cache->k, cache->s_page, cache->s_tok, cache->s_head);
  set_dst(a, 2, cache->v, cache->s_page, cache->s_tok, cache->s_head);
  a.heads[2] = d->h_k;
  a.block_table = cache->block_table;
  a.table_stride = cache->table_stride;
  a.n_pages = cache->n_pages;
  a.page_size = cache->page_size;
  return from_cuda(msa::launch_norm_rope(a, d->d, d->interleaved != 0, true,
                                         reinterpret_cast<cudaStream_t>(stream)));
}

size_t msa_qk_norm_rope_bwd_workspace(const msa_norm_rope_dims* d) {
  if (d == nullptr || (d->d != 64 && d->d != 128)) return 0;
  return msa::norm_rope_bwd_workspace(d->d);
}

msa_status msa_qk_norm_rope_bwd(const msa_norm_rope_dims* d, msa_tensor q, msa_tensor k,
                                const float* w_q, const float* w_k, const float* table,
                                int64_t n_pos, const int64_t* positions, msa_tensor d_q,
                                msa_tensor d_k, int32_t dy_fp32, msa_tensor dx_q,
                                msa_tensor dx_k, float* dw_q, float* dw_k, void* ws,
                                size_t ws_bytes, int32_t* dev_err, void* stream) {
  msa_status s = check_norm_rope(d, w_q, w_k, table, n_pos, positions);
  if (s != MSA_OK) return s;
  if (dy_fp32 != 0 && dy_fp32 != 1) return MSA_ERR_INVALID_ARG;
  if (d->h_q > 0 && ((s = check_tensor(q)) != MSA_OK ||
                     (s = check_norm_out(dx_q, d, d->h_q)) != MSA_OK))
    return s;
  if (d->h_k > 0 && ((s = check_tensor(k)) != MSA_OK ||
                     (s = check_norm_out(dx_k, d, d->h_k)) != MSA_OK))
    return s;
  if (d->h_q > 0 && (s = check_rows(d_q, dy_fp32 ? 4 : 2)) != MSA_OK) return s;
  if (d->h_k > 0 && (s = check_rows(d_k, dy_fp32 ? 4 : 2)) != MSA_OK) return s;
  if (ws == nullptr) return MSA_ERR_INVALID_ARG;
  if (!aligned16(ws)) return MSA_ERR_ALIGNMENT;
  if (ws_bytes < msa_qk_norm_rope_bwd_workspace(d)) return MSA_ERR_WORKSPACE_TOO_SMALL;
  msa::NormRopeBwdArgs p;
  std::memset(&p, 0, sizeof(p));
  p.f = norm_rope_args(d, w_q, w_k, table, n_pos, positions, dev_err);
  set_src(p.f, 0, q);
  set_src(p.f, 1, k);
  set_dst(p.f, 0, dx_q);
  set_dst(p.f, 1, dx_k);
  const msa_tensor* dy[2] = {&d_q, &d_k};
  for (int i = 0; i < 2; ++i) {
    p.dy[i] = dy[i]->ptr;
    p.ys_b[i] = dy[i]->s_batch;
    p.ys_t[i] = dy[i]->s_tok;
    p.ys_h[i] = dy[i]->s_head;
  }
  p.part = reinterpret_cast<float*>(ws);
  return from_cuda(msa::launch_norm_rope_bwd(p, d->d, d->interleaved != 0, dy_fp32 != 0, dw_q,
                                             dw_k, reinterpret_cast<cudaStream_t>(stream)));
}

size_t msa_paged_decode_attn_workspace(const msa_dims* d) {
  if (check_dims(d) != MSA_OK) return 0;
  return msa::paged_decode_workspace(d->batch, d->h_q / d->h_kv);
}

msa_status msa_paged_decode_attn(const msa_dims* d, int64_t window, int64_t n_sink, msa_tensor q,
                                 const msa_paged_kv* cache, void* out, float* lse, void* ws,
                                 size_t ws_bytes, int32_t* dev_err, void* stream) {
  msa_status s = check_dims(d);
  if (s != MSA_OK) return s;
  if (d->n_q != 1 || window < 0 || n_sink < 0) return MSA_ERR_INVALID_ARG;
  if ((s = check_tensor(q)) != MSA_OK) return s;
  if ((s = check_paged(cache)) != MSA_OK) return s;
  if (cache->seq_lens == nullptr || cache->h_kv != d->h_kv) return MSA_ERR_INVALID_ARG;
  if (cache->table_stride < (d->n_kv + cache->page_size - 1) / cache->page_size)
    return MSA_ERR_INVALID_ARG;
  if (out == nullptr || lse == nullptr || ws == nullptr) return MSA_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(ws) || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return MSA_ERR_ALIGNMENT;
  if (ws_bytes < msa_paged_decode_attn_workspace(d)) return MSA_ERR_WORKSPACE_TOO_SMALL;
  const int32_t tile = msa::paged_decode_tile();
  if (d->batch > msa::paged_decode_max_batch() ||
      d->batch * d->h_kv * (d->n_kv / tile + 2) > 0x7FFFFFFF)
    return MSA_ERR_UNSUPPORTED;
  CUtensorMap tk, tv;
  const uint32_t rows = (uint32_t)(cache->page_size < tile ? cache->page_size : tile);
  if ((s = make_map_pages(&tk, cache->k, cache, rows)) != MSA_OK) return s;
  if ((s = make_map_pages(&tv, cache->v, cache, rows)) != MSA_OK) return s;
  msa::PagedDecodeArgs a;
  std::memset(&a, 0, sizeof(a));
  a.q = reinterpret_cast<const __nv_bfloat16*>(q.ptr);
  a.qs_b = q.s_batch;
  a.qs_h = q.s_head;
  a.block_table = cache->block_table;
  a.seq_lens = cache->seq_lens;
  a.table_stride = cache->table_stride;
  a.n_pages = cache->n_pages;
  a.cap = (int32_t)d->n_kv;
  a.page_size = cache->page_size;
  while ((1 << a.page_shift) < a.page_size) ++a.page_shift;
  a.batch = (int32_t)d->batch;
  a.G = d->h_kv;
  a.R = d->h_q / d->h_kv;
  a.window = window == 0 ? a.cap : (int32_t)msa::min64(window, d->n_kv);
  a.sink = (int32_t)msa::min64(n_sink, d->n_kv);
  a.scale = d->scale;
  a.out = reinterpret_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.err = dev_err;
  return from_cuda(
      msa::launch_paged_decode(tk, tv, a, ws, reinterpret_cast<cudaStream_t>(stream)));
}

msa_status msa_window_attn_fwd(const msa_dims* d, int64_t window, int64_t n_sink, msa_tensor q,
                               msa_tensor k, msa_tensor v, const int32_t* kv_len, void* out,
                               void* out_rest, float* lse, int32_t* dev_err, void* stream) {
  msa_status s = check_window(d, window, n_sink, kv_len);
  if (s != MSA_OK) return s;
  if ((s = check_mapped(q, d->batch, d->n_q, d->h_q)) != MSA_OK) return s;
  for (const msa_tensor* t : {&k, &v})
    if ((s = check_mapped(*t, d->batch, d->n_kv, d->h_kv)) != MSA_OK) return s;
  if (out == nullptr || lse == nullptr) return MSA_ERR_INVALID_ARG;
  if (!aligned32(out) || !aligned16(out_rest) || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return MSA_ERR_ALIGNMENT;
  CUtensorMap tq, tk, tv, tk32, tv32;
  if ((s = make_map_rows(&tq, d, q)) != MSA_OK) return s;
  if ((s = make_map_keys(&tk, d, k, 128)) != MSA_OK) return s;
  if ((s = make_map_keys(&tv, d, v, 128)) != MSA_OK) return s;
  if ((s = make_map_keys(&tk32, d, k, 32)) != MSA_OK) return s;
  if ((s = make_map_keys(&tv32, d, v, 32)) != MSA_OK) return s;
  msa::WindowArgs a = window_args(d, window, n_sink, kv_len, dev_err);
  a.out = reinterpret_cast<__nv_bfloat16*>(out);
  a.rest = reinterpret_cast<int8_t*>(out_rest);
  a.lse = lse;
  return from_cuda(msa::launch_window_attn_fwd(tq, tk, tv, tk32, tv32, a,
                                               reinterpret_cast<cudaStream_t>(stream)));
}

size_t msa_window_attn_bwd_workspace(const msa_dims* d, int64_t window, int64_t n_sink) {
  if (check_window(d, window, n_sink, nullptr) != MSA_OK) return 0;
  return msa::window_attn_bwd_workspace(window_args(d, window, n_sink, nullptr, nullptr));
}

msa_status msa_window_attn_bwd(const msa_dims* d, int64_t window, int64_t n_sink, msa_tensor q,
                               msa_tensor k, msa_tensor v, msa_tensor o,
                               const void* o_rest, msa_tensor d_o, const float* lse,
                               const int32_t* kv_len, void* dq, void* dk,
                               void* dv, void* ws, size_t ws_bytes, int32_t* dev_err,
                               void* stream) {
  msa_status s = check_window(d, window, n_sink, kv_len);
  if (s != MSA_OK) return s;
  for (const msa_tensor* t : {&q, &d_o})
    if ((s = check_mapped(*t, d->batch, d->n_q, d->h_q)) != MSA_OK) return s;
  for (const msa_tensor* t : {&k, &v})
    if ((s = check_mapped(*t, d->batch, d->n_kv, d->h_kv)) != MSA_OK) return s;
  if ((s = check_tensor(o)) != MSA_OK) return s;
  if (lse == nullptr || dq == nullptr || dk == nullptr || dv == nullptr || ws == nullptr)
    return MSA_ERR_INVALID_ARG;
  if (!aligned32(dq) || !aligned32(dk) || !aligned32(dv) || !aligned32(ws) || !aligned16(o_rest) ||
      (reinterpret_cast<uintptr_t>(lse) & 3u))
    return MSA_ERR_ALIGNMENT;
  const size_t need = msa_window_attn_bwd_workspace(d, window, n_sink);
  if (need == 0) return MSA_ERR_UNSUPPORTED;
  if (ws_bytes < need) return MSA_ERR_WORKSPACE_TOO_SMALL;
  CUtensorMap tq, tdo, tk, tv, tk32, tv32;
  if ((s = make_map_rows(&tq, d, q)) != MSA_OK) return s;
  if ((s = make_map_rows(&tdo, d, d_o)) != MSA_OK) return s;
  if ((s = make_map_keys(&tk, d, k, 128)) != MSA_OK) return s;
  if ((s = make_map_keys(&tv, d, v, 128)) != MSA_OK) return s;
  if ((s = make_map_keys(&tk32, d, k, 32)) != MSA_OK) return s;
  if ((s = make_map_keys(&tv32, d, v, 32)) != MSA_OK) return s;
  msa::WindowArgs a = window_args(d, window, n_sink, kv_len, dev_err);
  a.o = reinterpret_cast<const __nv_bfloat16*>(o.ptr);
  a.os_b = o.s_batch;
  a.os_t = o.s_tok;
  a.os_h = o.s_head;
  a.d_o = reinterpret_cast<const __nv_bfloat16*>(d_o.ptr);
  a.ds_b = d_o.s_batch;
  a.ds_t = d_o.s_tok;
  a.ds_h = d_o.s_head;
  a.rest = const_cast<int8_t*>(reinterpret_cast<const int8_t*>(o_rest));
  a.lse = const_cast<float*>(lse);
  a.dq = reinterpret_cast<__nv_bfloat16*>(dq);
  a.dk = reinterpret_cast<__nv_bfloat16*>(dk);
  a.dv = reinterpret_cast<__nv_bfloat16*>(dv);
  return from_cuda(msa::launch_window_attn_bwd(tq, tdo, tk, tv, tk32, tv32, a, ws,
                                               reinterpret_cast<cudaStream_t>(stream)));
}

uint64_t msa_debug_set_attn_wait_limit_ns(uint64_t ns) {
  if (ns == 0) ns = msa::kWaitLimitNs;
  if (ns > msa::kWaitLimitNs) ns = msa::kWaitLimitNs;
  return msa::set_attn_wait_limit(ns);
}

const char* msa_status_string(msa_status s) {
  switch (s) {
    case MSA_OK: return "MSA_OK";
    case MSA_ERR_INVALID_ARG: return "MSA_ERR_INVALID_ARG";
    case MSA_ERR_UNSUPPORTED: return "MSA_ERR_UNSUPPORTED";
    case MSA_ERR_ALIGNMENT: return "MSA_ERR_ALIGNMENT";
    case MSA_ERR_WORKSPACE_TOO_SMALL: return "MSA_ERR_WORKSPACE_TOO_SMALL";
    case MSA_ERR_CUDA: return "MSA_ERR_CUDA";
    case MSA_ERR_SCRATCH_LIMIT: return "MSA_ERR_SCRATCH_LIMIT";
  }
  return "MSA_ERR_UNKNOWN";
}

}  // extern "C"
