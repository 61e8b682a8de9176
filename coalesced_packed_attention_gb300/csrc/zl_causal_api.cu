// C-ABI entry points of the causal attention: argument checks, TMA tensor maps, launches.
#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <mutex>

#include "zl_causal.h"
#include "zl_internal.h"

using namespace zl;

namespace {

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

PFN_cuTensorMapEncodeTiled_v12000 tiled_encode() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// Keys or values [tokens, key heads, d] with a token stride: boxes of 128 tokens x 64 channels of one head;
// coordinates (channel, head, token).
bool kv_map(CUtensorMap* m, const void* base, int64_t tokens, int64_t stride, int32_t heads, int32_t d) {
  auto fn = tiled_encode();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
  cuuint32_t box[3] = {64, 1, 128}, step[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Query rows packed by key head: [tokens, key heads, group, d], boxes of 128 / group tokens x group heads x 64
// channels; coordinates (channel, head in group, key head, token).
bool row_map(CUtensorMap* m, const void* base, int64_t tokens, int64_t stride, int32_t kv_heads, int32_t group, int32_t d) {
  auto fn = tiled_encode();
  if (!fn) return false;
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)group, (cuuint64_t)kv_heads, (cuuint64_t)tokens};
  cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)group * d * 2, (cuuint64_t)stride * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)group, 1, (cuuint32_t)tokens_per_block(group)}, step[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A plan that can be launched, with the device it was built on current.
bool ready(const zl_causal_plan* p) {
  if (!p || p->host_only || !p->tables) return false;
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == p->device;
}

// ~0.5 s at 2 GHz; short for the test hook
long long spin_limit(const zl_causal_plan* p) { return p->test_withhold ? 20000000LL : 1000000000LL; }

// exp2(scale log2(e) s): a scale of zero or below has another maximum, and a subnormal one is flushed
bool scale_ok(float scale) { return std::isnormal(scale) && scale > 0.f && std::isnormal(scale * 1.44269504f); }

bool stride_ok(int64_t stride, int32_t heads, int32_t d) {
  return stride >= (int64_t)heads * d && stride < ((int64_t)1 << 38);
}

zl_status check_inputs(const zl_causal_plan* p, const void* q, int64_t qs, const void* k, int64_t ks, const void* v,
                       int64_t vs, float scale) {
  const int32_t d = p->head_dim;
  if (!scale_ok(scale)) return ZL_ERR_INVALID_ARG;
  if (p->q_tokens > 0 && (!q || !stride_ok(qs, p->n_q_heads, d))) return ZL_ERR_INVALID_ARG;
  if (p->kv_tokens > 0 && (!k || !v || !stride_ok(ks, p->n_kv_heads, d) || !stride_ok(vs, p->n_kv_heads, d)))
    return ZL_ERR_INVALID_ARG;
  if (!on16(q) || !on16(k) || !on16(v) || qs % 8 || ks % 8 || vs % 8) return ZL_ERR_ALIGN;
  return ZL_OK;
}

}  // namespace

extern "C" zl_status zl_causal_attn_fwd(const zl_causal_plan* p, const void* q, int64_t q_stride, const void* k,
                                        int64_t k_stride, const void* v, int64_t v_stride, void* o, float* lse,
                                        void* workspace, float scale, void* stream) {
  NvtxRange range("zl_causal_attn_fwd");
  if (!ready(p)) return ZL_ERR_INVALID_ARG;
  zl_status s = check_inputs(p, q, q_stride, k, k_stride, v, v_stride, scale);
  if (s != ZL_OK) return s;
  if (p->fwd_tiles.empty()) return ZL_OK;  // no query rows
  if (!o || !lse || (p->fwd_bytes > 0 && !workspace)) return ZL_ERR_INVALID_ARG;
  if (!on16(o) || !on16(lse) || !on16(workspace)) return ZL_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  CUtensorMap tq, tk, tv;
  if (!row_map(&tq, q, p->q_tokens, q_stride, p->n_kv_heads, p->group, p->head_dim)) return ZL_ERR_CUDA;
  // without a key row no tile loads keys: any valid map will do
  if (p->kv_tokens == 0) tk = tv = tq;
  else if (!kv_map(&tk, k, p->kv_tokens, k_stride, p->n_kv_heads, p->head_dim) ||
           !kv_map(&tv, v, p->kv_tokens, v_stride, p->n_kv_heads, p->head_dim))
    return ZL_ERR_CUDA;
  CausalFwdParams fp;
  fp.tiles = p->d_fwd_tiles;
  fp.tile_ptr = p->d_fwd_ptr;
  fp.status = p->d_status;
  fp.wait_limit = spin_limit(p);
  fp.withhold_load = p->test_withhold ? 1 : 0;
  fp.n_q_heads = p->n_q_heads;
  fp.group = p->group;
  fp.o = static_cast<__nv_bfloat16*>(o);
  fp.lse = lse;
  fp.part_o = static_cast<float*>(workspace);
  fp.part_lse = fp.part_o + (int64_t)p->slots * 256 * p->head_dim;
  fp.scale_log2 = scale * 1.44269504088896340736f;
  if ((s = hold_tables(p, st)) != ZL_OK) return s;
  if (launch_causal_fwd(p->head_dim, tq, tk, tv, fp, (int)p->fwd_ptr.size() - 1, p->fwd_short, st) != cudaSuccess) return ZL_ERR_CUDA;
  if (p->merges.empty()) return ZL_OK;
  CausalMergeParams mp;
  mp.groups = p->d_merges;
  mp.n_groups = (int32_t)p->merges.size();
  mp.rows = p->merge_rows;
  mp.n_q_heads = p->n_q_heads;
  mp.group = p->group;
  mp.part_o = fp.part_o;
  mp.part_lse = fp.part_lse;
  mp.o = fp.o;
  mp.lse = lse;
  return launch_causal_merge(p->head_dim, mp, st) == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
}

extern "C" zl_status zl_causal_attn_bwd(const zl_causal_plan* p, const void* q, int64_t q_stride, const void* k,
                                        int64_t k_stride, const void* v, int64_t v_stride, const void* o,
                                        const void* d_o, const float* lse, void* dq, int64_t dq_stride, void* dk,
                                        int64_t dk_stride, void* dv, int64_t dv_stride, void* workspace, float scale,
                                        void* stream) {
  NvtxRange range("zl_causal_attn_bwd");
  if (!ready(p) || p->shared_keys || p->forward_only) return ZL_ERR_INVALID_ARG;
  zl_status s = check_inputs(p, q, q_stride, k, k_stride, v, v_stride, scale);
  if (s != ZL_OK) return s;
  const int32_t d = p->head_dim;
  if (p->q_tokens > 0 && (!o || !d_o || !lse || !dq || !stride_ok(dq_stride, p->n_q_heads, d) || !workspace))
    return ZL_ERR_INVALID_ARG;
  if (p->kv_tokens > 0 &&
      (!dk || !dv || !stride_ok(dk_stride, p->n_kv_heads, d) || !stride_ok(dv_stride, p->n_kv_heads, d)))
    return ZL_ERR_INVALID_ARG;
  if (!on16(o) || !on16(d_o) || !on16(lse) || !on16(dq) || !on16(dk) || !on16(dv) || !on16(workspace) || dq_stride % 8 ||
      dk_stride % 8 || dv_stride % 8)
    return ZL_ERR_ALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  float* row_d = static_cast<float*>(workspace);
  const int64_t rows = p->q_tokens * p->n_q_heads;
  float* acc = row_d + (rows * 4 + 255) / 256 * 64;
  float* part = acc + p->acc_blocks * 128 * d;
  if ((s = hold_tables(p, st)) != ZL_OK) return s;
  if (rows > 0 && launch_causal_bwd_pre(d, static_cast<const __nv_bfloat16*>(o), static_cast<const __nv_bfloat16*>(d_o), row_d,
                                        rows, acc, p->acc_blocks * 128 * d, p->num_sms, st) != cudaSuccess)
    return ZL_ERR_CUDA;
  if (!p->bwd_tiles.empty()) {
    CUtensorMap tq, tk, tv, tdo;
    if (!kv_map(&tk, k, p->kv_tokens, k_stride, p->n_kv_heads, d) || !kv_map(&tv, v, p->kv_tokens, v_stride, p->n_kv_heads, d))
      return ZL_ERR_CUDA;
    if (rows == 0) tq = tdo = tk;  // no query row: no tile loads one
    else if (!row_map(&tq, q, p->q_tokens, q_stride, p->n_kv_heads, p->group, d) ||
             !row_map(&tdo, d_o, p->q_tokens, (int64_t)p->n_q_heads * d, p->n_kv_heads, p->group, d))
      return ZL_ERR_CUDA;
    CausalBwdParams bp;
    bp.tiles = p->d_bwd_tiles;
    bp.tile_ptr = p->d_bwd_ptr;
    bp.status = p->d_status;
    bp.wait_limit = spin_limit(p);
    bp.withhold_load = p->test_withhold ? 1 : 0;
    bp.n_q_heads = p->n_q_heads;
    bp.n_kv_heads = p->n_kv_heads;
    bp.group = p->group;
    bp.lse = lse;
    bp.row_d = row_d;
    bp.acc = acc;
    bp.part = part;
    bp.dk = static_cast<__nv_bfloat16*>(dk);
    bp.dv = static_cast<__nv_bfloat16*>(dv);
    bp.dk_stride = dk_stride;
    bp.dv_stride = dv_stride;
    bp.scale = scale;
    bp.scale_log2 = scale * 1.44269504088896340736f;
    if (launch_causal_bwd(d, tq, tk, tv, tdo, bp, (int)p->bwd_ptr.size() - 1, p->bwd_short, st) != cudaSuccess) return ZL_ERR_CUDA;
  }
  CausalFinishParams fp;
  fp.seqs = p->d_seqs;
  fp.merges = p->d_bwd_merges;
  fp.n_seqs = (int32_t)p->seqs.size();
  fp.n_merges = (int32_t)p->bwd_merges.size();
  fp.n_q_heads = p->n_q_heads;
  fp.n_kv_heads = p->n_kv_heads;
  fp.acc_blocks = p->acc_blocks;
  fp.acc = acc;
  fp.part = part;
  fp.dq = static_cast<__nv_bfloat16*>(dq);
  fp.dk = static_cast<__nv_bfloat16*>(dk);
  fp.dv = static_cast<__nv_bfloat16*>(dv);
  fp.dq_stride = dq_stride;
  fp.dk_stride = dk_stride;
  fp.dv_stride = dv_stride;
  fp.scale = scale;
  return launch_causal_finish(d, fp, p->num_sms, st) == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
}

extern "C" zl_status zl_causal_get_device_status(const zl_causal_plan* p, void* stream, int32_t* device_status) {
  if (!ready(p) || !device_status) return ZL_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t v = 0;
  if (cudaMemcpyAsync(&v, p->d_status, sizeof(int32_t), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess || cudaMemsetAsync(p->d_status, 0, sizeof(int32_t), st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return ZL_ERR_CUDA;
  *device_status = v;
  return ZL_OK;
}
