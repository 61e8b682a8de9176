// Rotary positions of queries and keys, optionally behind an RMS norm of every head, forward
// and backward, one pass over the data each (sm_103a).
//
// Per head row x of d values at position t, with weights w:
//   n = x / sqrt(mean(x^2) + eps),  y = n w        (norm; without it y = x)
//   pair (a, b) of y with angle theta = t f:  (a cos - b sin, b cos + a sin) * amplitude
// and backward, with g the gradient of the result:
//   dy = the transposed rotation of g,  dw = sum over tokens and heads of dy n,
//   dx = (dn - n mean(dn n)) / sqrt(mean(x^2) + eps)  with dn = dy w.
//
// Bound: HBM, 4 bytes per value forward (6 backward with the norm); nothing is read twice and no
// statistic is kept between the passes (the backward has x in hand and forms the mean again).
// A row is held by d / 8 lanes, 16 bytes each, so a warp takes 2 (d = 128) or 4 (d = 64) heads of
// one token at a step and walks the token's query and key heads with the token's sines and
// cosines in registers.  The half layout's partner value sits rot/16 lanes away in the same row:
// the packed bf16 words are exchanged (4 shuffles for 8 values), and the weight of the partner is
// folded into its sine, so no normalised value has to be passed.
//
// Angles: a pair's frequency is a 64-bit fixed-point fraction of a turn per position, so
// position x frequency modulo 2^64 IS the fraction of the turn, exact at any position; its top 32
// bits go through sincospi.  (A float32 angle at position 10^6 is off by 0.03 rad.)
//
// Sums are fp32.  The weight gradients are summed per lane over the warp's tokens, per block in
// shared memory, and over blocks by a second launch, each in a fixed order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "zl_causal.h"
#include "zl_internal.h"
#include "zl_ptx.cuh"

namespace zl {

namespace {

constexpr int kRopeThreads = 256;

struct RopeTensor {
  const __nv_bfloat16* x;  // input (backward: the forward's input, norm only)
  const __nv_bfloat16* g;  // backward: gradient of the forward's result
  __nv_bfloat16* out;
  const float* w;
  int64_t x_stride, g_stride, out_stride;  // elements per token
  int32_t heads, steps;                    // steps of 32 / (d / 8) heads
};

struct RopeParams {
  RopeTensor t[2];  // queries, keys
  const int32_t* positions;
  const uint64_t* freq;
  float* partial;  // weight gradients per block, [blocks][2 d]
  int64_t n_tokens;
  int32_t rot, n_axes, axis1, axis2;  // first pair of the second and the third axis
  int32_t chunk;                      // steps of one token that one warp takes
  float eps, amplitude;
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 16 bytes of bf16 as eight floats
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  f[0] = bf_lo(v.x); f[1] = bf_hi(v.x); f[2] = bf_lo(v.y); f[3] = bf_hi(v.y);
  f[4] = bf_lo(v.z); f[5] = bf_hi(v.z); f[6] = bf_lo(v.w); f[7] = bf_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}
__device__ __forceinline__ uint4 load16(const __nv_bfloat16* p) { return *reinterpret_cast<const uint4*>(p); }

// the partner values of a lane's eight: of the partner lane (half) or the neighbour (interleaved)
template <bool kHalf>
__device__ __forceinline__ void partners(const uint4& v, const float (&f)[8], int plane, float (&p)[8]) {
  if constexpr (kHalf) {
    uint4 o;
    o.x = __shfl_sync(0xffffffffu, v.x, plane);
    o.y = __shfl_sync(0xffffffffu, v.y, plane);
    o.z = __shfl_sync(0xffffffffu, v.z, plane);
    o.w = __shfl_sync(0xffffffffu, v.w, plane);
    unpack8(o, p);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = f[i ^ 1];
  }
}

template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int s = kLanes / 2; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

template <int D, bool kHalf, bool kNorm, bool kBwd>
__global__ void __launch_bounds__(kRopeThreads) zl_qk_rope_kernel(const RopeParams p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes of a row, rows of a step
  constexpr int kUnroll = kBwd && kNorm ? 2 : 4;      // steps whose loads are in flight together
  constexpr bool kDw = kBwd && kNorm;
  const int lane = threadIdx.x & 31, sub = lane / kLanes, gl = lane % kLanes, e0 = gl * 8;
  const int nwarps = gridDim.x * (kRopeThreads / 32);
  const bool turns = e0 < p.rot;  // half: rot is a multiple of 16, so all eight values or none
  const int hop = p.rot / 16;
  const int plane = kHalf && turns ? (gl < hop ? lane + hop : lane - hop) : lane;
  const int pe0 = kHalf ? (plane % kLanes) * 8 : e0;  // first channel of the partner values
  const int s_begin = blockIdx.y * p.chunk;
  float acc[2][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[0][i] = acc[1][i] = 0.f;

  for (int64_t tok = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5); tok < p.n_tokens; tok += nwarps) {
    // out[i] = value[i] c[i] + partner[i] s[i], the sign of the sine included
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) { c[i] = 1.f; s[i] = 0.f; }
    if (p.rot > 0) {
      const int32_t* pt = p.positions + tok * p.n_axes;
      const int32_t t0 = __ldg(pt), t1 = p.n_axes > 1 ? __ldg(pt + 1) : 0, t2 = p.n_axes > 2 ? __ldg(pt + 2) : 0;
      auto turn = [&](int pair, float& cs, float& sn) {
        const int32_t t = pair < p.axis1 ? t0 : pair < p.axis2 ? t1 : t2;
        const uint64_t phase = (uint64_t)(int64_t)t * __ldg(p.freq + pair);
        // top 32 bits as a signed fraction of a turn; 2 pi r = pi (2 r)
        sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &sn, &cs);
        cs *= p.amplitude;
        sn *= p.amplitude;
      };
      if constexpr (kHalf) {
        if (turns) {
          const bool lower = gl < hop;
          const int pair0 = lower ? e0 : e0 - p.rot / 2;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            turn(pair0 + i, c[i], s[i]);
            s[i] = lower ? -s[i] : s[i];
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          if (e0 + i < p.rot) {
            turn((e0 + i) >> 1, c[i], s[i + 1]);
            c[i + 1] = c[i];
            s[i] = -s[i + 1];
          }
        }
      }
    }
    if constexpr (kBwd) {
#pragma unroll
      for (int i = 0; i < 8; ++i) s[i] = -s[i];  // the transpose turns back
    }
    int s0 = s_begin, s_left = p.chunk;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const RopeTensor& T = p.t[t];
      const int n = max(0, min(T.steps - s0, s_left));  // steps of this tensor in the chunk
      const int first = s0;
      s0 = max(0, s0 - T.steps);
      if (n <= 0) continue;
      s_left -= n;
      float a[8], b[8];  // forward: weights folded into cosine and sine; backward: a = weights
#pragma unroll
      for (int i = 0; i < 8; ++i) { a[i] = c[i]; b[i] = s[i]; }
      if constexpr (kNorm) {
        if (kBwd) {
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] = T.w ? __ldg(T.w + e0 + i) : 1.f;
        } else if (T.w) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            a[i] = c[i] * __ldg(T.w + e0 + i);
            b[i] = s[i] * __ldg(T.w + (kHalf ? pe0 + i : e0 + (i ^ 1)));
          }
        }
      }
      const __nv_bfloat16* xp = T.x + tok * T.x_stride + e0;
      const __nv_bfloat16* gp = T.g + tok * T.g_stride + e0;
      __nv_bfloat16* op = T.out + tok * T.out_stride + e0;
      for (int st = first; st < first + n; st += kUnroll) {
        uint4 vx[kUnroll], vg[kUnroll];
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int h = (st + u) * kRows + sub;
          vx[u] = vg[u] = make_uint4(0u, 0u, 0u, 0u);
          if (st + u < first + n && h < T.heads) {
            if constexpr (!kBwd || kNorm) vx[u] = load16(xp + (int64_t)h * D);
            if constexpr (kBwd) vg[u] = load16(gp + (int64_t)h * D);
          }
        }
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          const int h = (st + u) * kRows + sub;
          const bool ok = st + u < first + n && h < T.heads;
          float o[8];
          if constexpr (!kBwd) {
            float x[8], q[8];
            unpack8(vx[u], x);
            partners<kHalf>(vx[u], x, plane, q);
            float r = 1.f;
            if constexpr (kNorm) {
              float ss = 0.f;
#pragma unroll
              for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
              r = rsqrtf(fmaf(row_sum<kLanes>(ss), 1.f / D, p.eps));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              o[i] = fmaf(x[i], a[i], q[i] * b[i]);
              if constexpr (kNorm) o[i] *= r;
            }
          } else {
            float g[8], q[8], dy[8];
            unpack8(vg[u], g);
            partners<kHalf>(vg[u], g, plane, q);
#pragma unroll
            for (int i = 0; i < 8; ++i) dy[i] = fmaf(g[i], c[i], q[i] * s[i]);
            if constexpr (kNorm) {
              float x[8];
              unpack8(vx[u], x);
              float ss = 0.f, dot = 0.f;
#pragma unroll
              for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
              for (int i = 0; i < 8; ++i) dot = fmaf(dy[i] * a[i], x[i], dot);
              const float r = rsqrtf(fmaf(row_sum<kLanes>(ss), 1.f / D, p.eps));
              const float m = row_sum<kLanes>(dot) * (r * (1.f / D));  // mean(dn n)
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float nrm = x[i] * r;
                if (ok) acc[t][i] = fmaf(dy[i], nrm, acc[t][i]);
                o[i] = r * fmaf(-m, nrm, dy[i] * a[i]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) o[i] = dy[i];
            }
          }
          if (ok) *reinterpret_cast<uint4*>(op + (int64_t)h * D) = pack8(o);
        }
      }
    }
  }
  if constexpr (kDw) {
    if (p.partial) {
      __shared__ float red[kRopeThreads / 32 * kRows][2 * D];
      float* row = red[(threadIdx.x >> 5) * kRows + sub];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        row[e0 + i] = acc[0][i];
        row[D + e0 + i] = acc[1][i];
      }
      __syncthreads();
      if (threadIdx.x < 2 * D) {
        float v = 0.f;
        for (int r = 0; r < kRopeThreads / 32 * kRows; ++r) v += red[r][threadIdx.x];
        p.partial[((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (2 * D) + threadIdx.x] = v;
      }
    }
  }
}

// Sum of the blocks' weight gradients: 32 columns a block, 32 slices of the rows, in order.
__global__ void __launch_bounds__(1024) zl_qk_rope_dw_kernel(const float* __restrict__ partial, int32_t rows, int32_t d,
                                                             float* __restrict__ dwq, float* __restrict__ dwk) {
  __shared__ float red[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + x;
  float v = 0.f;
#pragma unroll 4
  for (int r = y; r < rows; r += 32) v += __ldg(partial + (int64_t)r * (2 * d) + col);
  red[y][x] = v;
  __syncthreads();
  if (y == 0) {
    v = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) v += red[r][x];
    float* out = col < d ? dwq : dwk;
    if (out) out[col < d ? col : col - d] = v;
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

zl_status check_desc(const zl_qk_rope_desc* d) {
  if (!d) return ZL_ERR_INVALID_ARG;
  if (d->head_dim != 64 && d->head_dim != 128) return ZL_ERR_UNSUPPORTED;
  if (d->n_tokens < 0 || d->n_tokens > (int64_t)INT32_MAX || d->n_q_heads < 0 || d->n_kv_heads < 0 ||
      d->n_q_heads > 65536 || d->n_kv_heads > 65536 || (d->n_q_heads == 0 && d->n_kv_heads == 0))
    return ZL_ERR_INVALID_ARG;
  if ((d->norm != 0 && d->norm != 1) || (d->half_layout != 0 && d->half_layout != 1)) return ZL_ERR_INVALID_ARG;
  if (d->norm && !(d->eps >= 0.f && std::isfinite(d->eps))) return ZL_ERR_INVALID_ARG;
  if (d->rot_dim < 0 || d->rot_dim > d->head_dim || d->rot_dim % (d->half_layout ? 16 : 2)) return ZL_ERR_INVALID_ARG;
  if (d->rot_dim > 0) {
    if (d->n_axes < 1 || d->n_axes > 3 || !std::isfinite(d->amplitude)) return ZL_ERR_INVALID_ARG;
    int64_t pairs = 0;
    for (int a = 0; a < d->n_axes; ++a) {
      if (d->axis_pairs[a] < 0) return ZL_ERR_INVALID_ARG;
      pairs += d->axis_pairs[a];
    }
    if (pairs * 2 != d->rot_dim) return ZL_ERR_INVALID_ARG;
  }
  return ZL_OK;
}

// One of the two tensors' pointers: heads 0 wants none, any other count wants them aligned, with a
// token stride that holds its heads.
zl_status check_tensor(const void* p, int64_t stride, int32_t heads, int32_t d) {
  if (heads == 0) return ZL_OK;
  if (!p || stride < (int64_t)heads * d) return ZL_ERR_INVALID_ARG;
  if (!aligned16(p) || stride % 8) return ZL_ERR_ALIGN;
  return ZL_OK;
}

using RopeKernel = void (*)(const RopeParams);

template <int D, bool kBwd>
RopeKernel pick(bool half, bool norm) {
  if (half) return norm ? zl_qk_rope_kernel<D, true, true, kBwd> : zl_qk_rope_kernel<D, true, false, kBwd>;
  return norm ? zl_qk_rope_kernel<D, false, true, kBwd> : zl_qk_rope_kernel<D, false, false, kBwd>;
}

// Blocks that the weight gradients' workspace has rows for.
constexpr int kMaxDwBlocks = 2048;

cudaError_t launch_rope(const zl_qk_rope_desc& d, bool bwd, RopeParams& p, float* dwq, float* dwk,
                        cudaStream_t stream) {
  const int D = d.head_dim, rows = 256 / D;
  for (int t = 0; t < 2; ++t) {
    p.t[t].heads = t == 0 ? d.n_q_heads : d.n_kv_heads;
    p.t[t].steps = (p.t[t].heads + rows - 1) / rows;
  }
  p.n_tokens = d.n_tokens;
  p.rot = d.rot_dim;
  p.n_axes = d.rot_dim > 0 ? d.n_axes : 0;
  p.axis1 = p.n_axes > 1 ? d.axis_pairs[0] : INT32_MAX;
  p.axis2 = p.n_axes > 2 ? d.axis_pairs[0] + d.axis_pairs[1] : INT32_MAX;
  p.eps = d.eps;
  p.amplitude = d.amplitude;
  RopeKernel k = D == 128 ? (bwd ? pick<128, true>(d.half_layout, d.norm) : pick<128, false>(d.half_layout, d.norm))
                          : (bwd ? pick<64, true>(d.half_layout, d.norm) : pick<64, false>(d.half_layout, d.norm));
  int dev = 0, sms = 0, per_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k, kRopeThreads, 0);
  if (e != cudaSuccess) return e;
  if (per_sm < 1) per_sm = 1;
  // One wave of blocks, a warp per token; with fewer tokens than warps a token's heads are split
  // over several warps (each forms the token's sines again), down to kUnroll steps a warp.
  const int64_t warps = (int64_t)sms * per_sm * (kRopeThreads / 32);
  const int steps = p.t[0].steps + p.t[1].steps;
  int64_t chunks = d.n_tokens > 0 ? warps / d.n_tokens : 1;
  const int64_t most = (steps + 3) / 4;
  if (chunks > most) chunks = most;
  if (p.partial && chunks > kMaxDwBlocks) chunks = kMaxDwBlocks;
  if (chunks < 1) chunks = 1;
  p.chunk = (int)((steps + chunks - 1) / chunks);
  const int ny = (steps + p.chunk - 1) / p.chunk;
  int64_t nx = (d.n_tokens + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  const int64_t cap = ((int64_t)sms * per_sm + ny - 1) / ny;
  if (nx > cap) nx = cap;
  if (p.partial && nx * ny > kMaxDwBlocks) nx = kMaxDwBlocks / ny;
  if (nx < 1) nx = 1;
  k<<<dim3((unsigned)nx, (unsigned)ny), kRopeThreads, 0, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || !p.partial) return e;
  zl_qk_rope_dw_kernel<<<2 * D / 32, 1024, 0, stream>>>(p.partial, (int32_t)(nx * ny), D, dwq, dwk);
  return cudaGetLastError();
}

// The kernels are built for sm_103a alone.
zl_status check_device() {
  int dev = 0, major = 0, minor = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
    return ZL_ERR_CUDA;
  return major == 10 && minor == 3 ? ZL_OK : ZL_ERR_UNSUPPORTED;
}

}  // namespace

}  // namespace zl

using namespace zl;

extern "C" zl_status zl_rope_frequencies(const double* radians, int32_t n, uint64_t* out) {
  if (n < 0 || (n > 0 && (!radians || !out))) return ZL_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n; ++i)
    if (!std::isfinite(radians[i])) return ZL_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n; ++i) {
    const double turns = radians[i] * 0.15915494309189533577;  // 1 / (2 pi)
    const double frac = turns - std::floor(turns);             // whole turns of a whole position change nothing
    // 2^32 at a time: the product with 2^64 may round up to 2^64, which is no turn at all
    const double hi = std::floor(std::ldexp(frac, 32));
    const double lo = std::floor(std::ldexp(std::ldexp(frac, 32) - hi, 32));
    out[i] = ((uint64_t)hi << 32) + (uint64_t)lo;
  }
  return ZL_OK;
}

extern "C" zl_status zl_qk_rope_workspace(const zl_qk_rope_desc* d, int64_t* bytes) {
  const zl_status s = check_desc(d);
  if (s != ZL_OK) return s;
  if (!bytes) return ZL_ERR_INVALID_ARG;
  *bytes = (int64_t)kMaxDwBlocks * 2 * d->head_dim * (int64_t)sizeof(float);
  return ZL_OK;
}

extern "C" zl_status zl_qk_rope_fwd(const zl_qk_rope_desc* d, const void* q, int64_t q_stride, const void* k,
                                    int64_t k_stride, const float* q_weight, const float* k_weight,
                                    const int32_t* positions, const uint64_t* freq, void* q_out, int64_t q_out_stride,
                                    void* k_out, int64_t k_out_stride, void* stream) {
  NvtxRange range("zl_qk_rope_fwd");
  zl_status s = check_desc(d);
  if (s != ZL_OK) return s;
  if (!d->norm && (q_weight || k_weight)) return ZL_ERR_INVALID_ARG;
  if (d->n_tokens == 0) return ZL_OK;
  const int32_t D = d->head_dim;
  if ((s = check_tensor(q, q_stride, d->n_q_heads, D)) != ZL_OK || (s = check_tensor(k, k_stride, d->n_kv_heads, D)) != ZL_OK ||
      (s = check_tensor(q_out, q_out_stride, d->n_q_heads, D)) != ZL_OK ||
      (s = check_tensor(k_out, k_out_stride, d->n_kv_heads, D)) != ZL_OK)
    return s;
  if (d->rot_dim > 0 && (!positions || !freq)) return ZL_ERR_INVALID_ARG;
  if ((s = check_device()) != ZL_OK) return s;
  RopeParams p{};
  p.t[0] = {static_cast<const __nv_bfloat16*>(q), nullptr, static_cast<__nv_bfloat16*>(q_out), q_weight, q_stride, 0,
            q_out_stride, 0, 0};
  p.t[1] = {static_cast<const __nv_bfloat16*>(k), nullptr, static_cast<__nv_bfloat16*>(k_out), k_weight, k_stride, 0,
            k_out_stride, 0, 0};
  p.positions = positions;
  p.freq = freq;
  return launch_rope(*d, false, p, nullptr, nullptr, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
}

extern "C" zl_status zl_qk_rope_bwd(const zl_qk_rope_desc* d, const void* q, int64_t q_stride, const void* k,
                                    int64_t k_stride, const float* q_weight, const float* k_weight,
                                    const int32_t* positions, const uint64_t* freq, const void* dq_out,
                                    int64_t dq_out_stride, const void* dk_out, int64_t dk_out_stride, void* dq,
                                    int64_t dq_stride, void* dk, int64_t dk_stride, float* dq_weight, float* dk_weight,
                                    void* workspace, void* stream) {
  NvtxRange range("zl_qk_rope_bwd");
  zl_status s = check_desc(d);
  if (s != ZL_OK) return s;
  if (!d->norm && (q_weight || k_weight)) return ZL_ERR_INVALID_ARG;
  if ((dq_weight && !q_weight) || (dk_weight && !k_weight)) return ZL_ERR_INVALID_ARG;
  // a side without heads has no weights to give a gradient to
  if ((dq_weight && d->n_q_heads == 0) || (dk_weight && d->n_kv_heads == 0)) return ZL_ERR_INVALID_ARG;
  const bool dw = dq_weight || dk_weight;
  if (dw && !workspace) return ZL_ERR_INVALID_ARG;
  if (dw && !aligned16(workspace)) return ZL_ERR_ALIGN;
  const int32_t D = d->head_dim;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d->n_tokens == 0) {  // no rows: the weights' gradients are empty sums
    if ((dq_weight && cudaMemsetAsync(dq_weight, 0, sizeof(float) * D, st) != cudaSuccess) ||
        (dk_weight && cudaMemsetAsync(dk_weight, 0, sizeof(float) * D, st) != cudaSuccess))
      return ZL_ERR_CUDA;
    return ZL_OK;
  }
  if (d->norm && ((s = check_tensor(q, q_stride, d->n_q_heads, D)) != ZL_OK ||
                  (s = check_tensor(k, k_stride, d->n_kv_heads, D)) != ZL_OK))
    return s;
  if ((s = check_tensor(dq_out, dq_out_stride, d->n_q_heads, D)) != ZL_OK ||
      (s = check_tensor(dk_out, dk_out_stride, d->n_kv_heads, D)) != ZL_OK ||
      (s = check_tensor(dq, dq_stride, d->n_q_heads, D)) != ZL_OK || (s = check_tensor(dk, dk_stride, d->n_kv_heads, D)) != ZL_OK)
    return s;
  if (d->rot_dim > 0 && (!positions || !freq)) return ZL_ERR_INVALID_ARG;
  if ((s = check_device()) != ZL_OK) return s;
  RopeParams p{};
  p.t[0] = {static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(dq_out), static_cast<__nv_bfloat16*>(dq),
            q_weight, q_stride, dq_out_stride, dq_stride, 0, 0};
  p.t[1] = {static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(dk_out), static_cast<__nv_bfloat16*>(dk),
            k_weight, k_stride, dk_out_stride, dk_stride, 0, 0};
  p.positions = positions;
  p.freq = freq;
  p.partial = dw ? static_cast<float*>(workspace) : nullptr;
  return launch_rope(*d, true, p, dq_weight, dk_weight, st) == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
}
