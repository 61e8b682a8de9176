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
// Bound: HBM (49 144 tokens, d = 128: 32/8 heads forward 154.6 us, 6.5 TB/s; 20/20 heads gradient 249.4 us, 6.1
// TB/s), 4 bytes per value forward (6 backward with the norm); nothing is read twice and no
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
#include "zl_overlap.cuh"
#include "zl_ptx.cuh"

namespace zl {

namespace {

constexpr int kRopeThreads = 256;

struct RopeTensor {
  const __nv_bfloat16* x;  // input (backward: the forward's input, norm only)
  const __nv_bfloat16* g;  // backward: gradient of the forward's result
  __nv_bfloat16* out;
  const float* w;
  const uint8_t* rows;                     // backward: 0 where a token has no gradient; null: every token has one
  int64_t x_stride, g_stride, out_stride;  // elements per token
  int32_t heads, batches;                  // batches of rope_unroll steps of 32 / (d / 8) heads
};

struct RopeParams {
  RopeTensor t[2];  // queries, keys
  const int32_t* positions;
  const uint64_t* freq;
  float* partial;  // weight gradients per block, [blocks][2 d]; null: not wanted, or of the only block and so final:
  float *dwq, *dwk;
  int64_t n_tokens;
  int32_t rot, n_axes, axis1, axis2;  // first pair of the second and the third axis
  int32_t chunk;                      // batches of one token that one warp takes
  float eps, amplitude;
};

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 16 bytes of bf16 as four pairs of floats, which the two-wide fp32 operations take: they halve the instructions of
// the arithmetic (56 % of the issue slots went on it, one value at a time)
__device__ __forceinline__ void unpack8(const uint4& v, float2 (&f)[4]) {
  f[0] = make_float2(bf_lo(v.x), bf_hi(v.x));
  f[1] = make_float2(bf_lo(v.y), bf_hi(v.y));
  f[2] = make_float2(bf_lo(v.z), bf_hi(v.z));
  f[3] = make_float2(bf_lo(v.w), bf_hi(v.w));
}
__device__ __forceinline__ uint4 pack8(const float2 (&f)[4]) {
  return make_uint4(pack_bf16(f[0].x, f[0].y), pack_bf16(f[1].x, f[1].y), pack_bf16(f[2].x, f[2].y), pack_bf16(f[3].x, f[3].y));
}
__device__ __forceinline__ uint4 load16(const __nv_bfloat16* p) { return *reinterpret_cast<const uint4*>(p); }

// the partner values of a lane's eight: of the partner lane (half) or the neighbour (interleaved)
template <bool kHalf>
__device__ __forceinline__ void partners(const uint4& v, int plane, float2 (&p)[4]) {
  if constexpr (kHalf) {
    uint4 o;
    o.x = __shfl_sync(0xffffffffu, v.x, plane);
    o.y = __shfl_sync(0xffffffffu, v.y, plane);
    o.z = __shfl_sync(0xffffffffu, v.z, plane);
    o.w = __shfl_sync(0xffffffffu, v.w, plane);
    unpack8(o, p);
  } else {
    p[0] = make_float2(bf_hi(v.x), bf_lo(v.x));
    p[1] = make_float2(bf_hi(v.y), bf_lo(v.y));
    p[2] = make_float2(bf_hi(v.z), bf_lo(v.z));
    p[3] = make_float2(bf_hi(v.w), bf_lo(v.w));
  }
}

// The words of `yes` whose pairs turn (the half layout: all of a lane's or none), of `no` the others: channels past the
// rotated ones have no partner and pass through as they are, where a product with a sine of 0 would make NaN of an
// Inf, their own or their neighbour's.
template <bool kHalf>
__device__ __forceinline__ uint4 where_turning(int e0, int rot, const uint4& yes, const uint4& no) {
  constexpr int kStep = kHalf ? 0 : 2;
  return make_uint4(e0 < rot ? yes.x : no.x, e0 + kStep < rot ? yes.y : no.y, e0 + 2 * kStep < rot ? yes.z : no.z,
                    e0 + 3 * kStep < rot ? yes.w : no.w);
}

template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int s = kLanes / 2; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// A warp's unit is a batch of kUnroll steps of one tensor of one token; the loads of the next batch (of the next
// token after the last) are issued before the current one is computed, so 16-byte loads are in flight through
// the sines, the sums and the stores alike.
template <bool kBwd, bool kNorm>
constexpr int rope_unroll() {
  return kBwd && kNorm ? 2 : 4;
}

// kPlain: every channel is rotated (rot = d) and every token has a gradient.  The selects that let the other channels
// through and the look at a token's byte cost 2 to 4 % of a launch (49 144 tokens, 20/20 heads: gradient 257 against
// 250 us), so they are compiled for the calls that have such channels or bytes alone.
template <int D, bool kHalf, bool kNorm, bool kBwd, bool kPlain>
__global__ void __launch_bounds__(kRopeThreads, 2) zl_qk_rope_kernel(const RopeParams p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes of a row, rows of a step
  constexpr int kUnroll = rope_unroll<kBwd, kNorm>();
  constexpr bool kDw = kBwd && kNorm;
  constexpr bool kHasX = !kBwd || kNorm;
  __shared__ __align__(16) float red[kDw ? kRopeThreads / 32 * kRows : 1][2 * D];  // weights, then (kDw) the weights' gradients
  const int lane = threadIdx.x & 31, sub = lane / kLanes, gl = lane % kLanes, e0 = gl * 8;
  const int64_t nwarps = (int64_t)gridDim.x * (kRopeThreads / 32);
  const bool turns = e0 < p.rot;  // half: rot is a multiple of 16, so all eight values or none
  const int hop = p.rot / 16;
  const bool lower = gl < hop;
  const int plane = kHalf && turns ? (lower ? lane + hop : lane - hop) : lane;
  const int pe0 = kHalf ? (plane % kLanes) * 8 : e0;  // first channel of the partner values
  let_next_start();
  wait_for_previous();
  // the pairs whose sines this lane forms, and the lane that forms the first of those that it uses
  const int pairs = p.rot / 2, my_pair = 2 * lane;
  const int src = (kHalf ? (lower ? e0 : e0 - pairs) : e0 / 2) / 2;
  const uint64_t f0 = my_pair < pairs ? p.freq[my_pair] : 0, f1 = my_pair + 1 < pairs ? p.freq[my_pair + 1] : 0;
  auto axis_of = [&](int pair) { return pair < p.axis1 ? 0 : pair < p.axis2 ? 1 : 2; };
  const int ax0 = my_pair < pairs ? axis_of(my_pair) : 0, ax1 = my_pair + 1 < pairs ? axis_of(my_pair + 1) : 0;

  if constexpr (kNorm) {
    if (threadIdx.x < 2 * D) {
      const float* w = threadIdx.x < D ? p.t[0].w : p.t[1].w;
      red[0][threadIdx.x] = w ? w[threadIdx.x % D] : 1.f;
    }
    __syncthreads();
  }
  const int nb0 = p.t[0].batches;
  const int b_begin = blockIdx.y * p.chunk, b_end = min(b_begin + p.chunk, nb0 + p.t[1].batches);
  float2 acc0[4], acc1[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc0[i] = acc1[i] = make_float2(0.f, 0.f);

  struct Batch {
    uint4 x[kUnroll], g[kUnroll];
  };
  auto fetch = [&](int64_t tok, int bi, Batch& v) {
    const RopeTensor& T = p.t[bi >= nb0];
    const int h0 = (bi >= nb0 ? bi - nb0 : bi) * (kUnroll * kRows) + sub;
    const __nv_bfloat16* xp = T.x + tok * T.x_stride + (int64_t)h0 * D + e0;
    const __nv_bfloat16* gp = T.g + tok * T.g_stride + (int64_t)h0 * D + e0;
    int heads = T.heads;
    if constexpr (kBwd && !kPlain) {
      if (T.rows != nullptr && T.rows[tok] == 0) heads = 0;
    }
    // What is not loaded has g = 0 and x = 1, whose norm is finite whatever eps is: it adds 0 to the weights' gradients,
    // and a token without a gradient gets 0.  (Plain calls take x = 0, which needs no register, and r = 0 below: gradient
    // of 49 144 tokens, 20/20 heads, 250 against 254 us.)
    constexpr uint32_t kFill = kPlain ? 0u : 0x3f803f80u;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const bool in = h0 + u * kRows < heads;
      if constexpr (kHasX) v.x[u] = in ? load16(xp + u * kRows * D) : make_uint4(kFill, kFill, kFill, kFill);
      if constexpr (kBwd) v.g[u] = in ? load16(gp + u * kRows * D) : make_uint4(0u, 0u, 0u, 0u);
    }
  };

  int64_t tok = (int64_t)blockIdx.x * (kRopeThreads / 32) + (threadIdx.x >> 5);
  Batch cur;
  if (tok < p.n_tokens) fetch(tok, b_begin, cur);
  for (; tok < p.n_tokens; tok += nwarps) {
    // out[i] = value[i] c[i] + partner[i] s[i], the sign of the sine included
    float c[8], s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) { c[i] = 1.f; s[i] = 0.f; }
    if (p.rot > 0) {
      const int32_t* pt = p.positions + tok * p.n_axes;
      float cs[2], sn[2];
      auto turn = [&](uint64_t f, int axis, float& co, float& si) {
        const uint64_t phase = (uint64_t)(int64_t)pt[axis] * f;
        // top 32 bits as a signed fraction of a turn; 2 pi r = pi (2 r)
        sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &si, &co);
        co *= p.amplitude;
        si *= p.amplitude;
      };
      turn(f0, ax0, cs[0], sn[0]);
      turn(f1, ax1, cs[1], sn[1]);
      // 2 pairs a lane, so the pairs from 2 src on sit in lanes src, src + 1, ...
      if constexpr (kHalf) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float co = __shfl_sync(0xffffffffu, cs[i & 1], src + i / 2), si = __shfl_sync(0xffffffffu, sn[i & 1], src + i / 2);
          if (turns) {
            c[i] = co;
            s[i] = lower != kBwd ? -si : si;  // backward turns back
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          const float co = __shfl_sync(0xffffffffu, cs[(i / 2) & 1], src + i / 4);
          const float si = __shfl_sync(0xffffffffu, sn[(i / 2) & 1], src + i / 4);
          if (e0 + i < p.rot) {
            c[i] = c[i + 1] = co;
            s[i] = kBwd ? si : -si;
            s[i + 1] = -s[i];
          }
        }
      }
    }
    float2 a[4], b[4];  // forward: cosine and sine, the weights folded in; backward: the weights, and in cs2, sn2 both
    float2 cs2[4], sn2[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cs2[i] = make_float2(c[2 * i], c[2 * i + 1]);
      sn2[i] = make_float2(s[2 * i], s[2 * i + 1]);
    }
    for (int bi = b_begin; bi < b_end; ++bi) {
      Batch nxt;
      if (bi + 1 < b_end) fetch(tok, bi + 1, nxt);
      else if (tok + nwarps < p.n_tokens) fetch(tok + nwarps, b_begin, nxt);
      const int t = bi >= nb0;
      const RopeTensor& T = p.t[t];
      if (bi == b_begin || bi == nb0) {
        if constexpr (kNorm) {
          const float* w = red[0] + t * D;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 own = make_float2(w[e0 + 2 * i], w[e0 + 2 * i + 1]);
            if constexpr (kBwd) {
              a[i] = own;
            } else {
              const float2 other = kHalf ? make_float2(w[pe0 + 2 * i], w[pe0 + 2 * i + 1]) : make_float2(own.y, own.x);
              a[i] = mul2(cs2[i], own);
              b[i] = mul2(sn2[i], other);
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) { a[i] = cs2[i]; b[i] = sn2[i]; }
        }
      }
      const int h0 = (t ? bi - nb0 : bi) * (kUnroll * kRows) + sub;
      __nv_bfloat16* op = T.out + tok * T.out_stride + (int64_t)h0 * D + e0;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const bool ok = h0 + u * kRows < T.heads;
        float2 o[4];
        auto partner_values = [&](const uint4& v, float2 (&q)[4]) {
          partners<kHalf>(v, plane, q);
          if constexpr (kNorm && !kPlain) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (e0 + (kHalf ? 0 : 2 * i) >= p.rot) q[i] = make_float2(0.f, 0.f);
          }
        };
        if constexpr (!kBwd) {
          float2 x[4], q[4];
          unpack8(cur.x[u], x);
          partner_values(cur.x[u], q);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = fma2(x[i], a[i], mul2(q[i], b[i]));
          if constexpr (kNorm) {
            float2 ss = mul2(x[0], x[0]);
#pragma unroll
            for (int i = 1; i < 4; ++i) ss = fma2(x[i], x[i], ss);
            const float r = rsqrtf(fmaf(row_sum<kLanes>(ss.x + ss.y), 1.f / D, p.eps));
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = mul2(o[i], make_float2(r, r));
          }
        } else {
          float2 g[4], q[4], dy[4];
          unpack8(cur.g[u], g);
          partner_values(cur.g[u], q);
#pragma unroll
          for (int i = 0; i < 4; ++i) dy[i] = fma2(g[i], cs2[i], mul2(q[i], sn2[i]));
          if constexpr (kNorm) {
            float2 x[4], dn[4];
            unpack8(cur.x[u], x);
#pragma unroll
            for (int i = 0; i < 4; ++i) dn[i] = mul2(dy[i], a[i]);
            float2 ss = mul2(x[0], x[0]), dot = mul2(dn[0], x[0]);
#pragma unroll
            for (int i = 1; i < 4; ++i) {
              ss = fma2(x[i], x[i], ss);
              dot = fma2(dn[i], x[i], dot);
            }
            float r = rsqrtf(fmaf(row_sum<kLanes>(ss.x + ss.y), 1.f / D, p.eps));
            if constexpr (kPlain) r = ok ? r : 0.f;  // a lane without a head adds nothing, whatever eps makes of its zeros
            const float m = row_sum<kLanes>(dot.x + dot.y) * (r * (1.f / D));  // mean(dn n)
            const float2 r2 = make_float2(r, r), nm2 = make_float2(-m, -m);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              x[i] = mul2(x[i], r2);
              o[i] = mul2(r2, fma2(nm2, x[i], dn[i]));
            }
            if (t == 0) {
#pragma unroll
              for (int i = 0; i < 4; ++i) acc0[i] = fma2(dy[i], x[i], acc0[i]);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) acc1[i] = fma2(dy[i], x[i], acc1[i]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = dy[i];
          }
        }
        if (ok) {
          if constexpr (kNorm || kPlain) *reinterpret_cast<uint4*>(op + u * kRows * D) = pack8(o);
          else *reinterpret_cast<uint4*>(op + u * kRows * D) = where_turning<kHalf>(e0, p.rot, pack8(o), kBwd ? cur.g[u] : cur.x[u]);
        }
      }
      cur = nxt;
    }
  }
  if constexpr (kDw) {
    if (p.partial || p.dwq || p.dwk) {
      __syncthreads();  // the weights in red[0] have been read
      float* row = red[(threadIdx.x >> 5) * kRows + sub];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        *reinterpret_cast<float2*>(row + e0 + 2 * i) = acc0[i];
        *reinterpret_cast<float2*>(row + D + e0 + 2 * i) = acc1[i];
      }
      __syncthreads();
      if (threadIdx.x < 2 * D) {
        float v = 0.f;
        for (int r = 0; r < kRopeThreads / 32 * kRows; ++r) v += red[r][threadIdx.x];
        if (p.partial) p.partial[((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (2 * D) + threadIdx.x] = v;
        else if (threadIdx.x < D) { if (p.dwq) p.dwq[threadIdx.x] = v; }
        else if (p.dwk) p.dwk[threadIdx.x - D] = v;
      }
    }
  }
}

// Sum of the blocks' weight gradients: 32 columns a block, 32 slices of the rows, in order.
__global__ void __launch_bounds__(1024) zl_qk_rope_dw_kernel(const float* partial, int32_t rows, int32_t d, float* dwq, float* dwk) {
  __shared__ float red[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + x;
  let_next_start();
  wait_for_previous();
  float v = 0.f;
#pragma unroll 4
  for (int r = y; r < rows; r += 32) v += partial[(int64_t)r * (2 * d) + col];
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

bool aligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
bool aligned16(const void* p) { return aligned(p, 16); }

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

// An output may lie where its input does, row for row; at another stride it would overwrite rows not yet read.
bool same_rows(const void* in, int64_t in_stride, const void* out, int64_t out_stride, int64_t n) {
  return in != out || in_stride == out_stride || n <= 1;
}

// One of the two tensors' pointers: heads 0 wants none, any other count wants them aligned, with a
// token stride that holds its heads.
zl_status check_tensor(const void* p, int64_t stride, int32_t heads, int32_t d) {
  if (heads == 0) return ZL_OK;
  if (!p || stride < (int64_t)heads * d) return ZL_ERR_INVALID_ARG;
  if (!aligned16(p) || stride % 8) return ZL_ERR_ALIGN;
  return ZL_OK;
}

// What is read number by number: weights, positions, frequencies.
bool numbers_aligned(const float* qw, const float* kw, const int32_t* positions, const uint64_t* freq) {
  return aligned(qw, sizeof(float)) && aligned(kw, sizeof(float)) && aligned(positions, sizeof(int32_t)) &&
         aligned(freq, sizeof(uint64_t));
}

using RopeKernel = void (*)(const RopeParams);

template <int D, bool kBwd, bool kPlain>
RopeKernel pick(bool half, bool norm) {
  if (half) return norm ? zl_qk_rope_kernel<D, true, true, kBwd, kPlain> : zl_qk_rope_kernel<D, true, false, kBwd, kPlain>;
  return norm ? zl_qk_rope_kernel<D, false, true, kBwd, kPlain> : zl_qk_rope_kernel<D, false, false, kBwd, kPlain>;
}
template <int D>
RopeKernel pick(bool half, bool norm, bool bwd, bool plain) {
  if (bwd) return plain ? pick<D, true, true>(half, norm) : pick<D, true, false>(half, norm);
  return plain ? pick<D, false, true>(half, norm) : pick<D, false, false>(half, norm);
}

// Blocks that the weight gradients' workspace has rows for.
constexpr int kMaxDwBlocks = 2048;

cudaError_t launch_rope(const zl_qk_rope_desc& d, bool bwd, int sms, RopeParams& p, float* dwq, float* dwk,
                        cudaStream_t stream) {
  const int D = d.head_dim;
  const int per_batch = (bwd && d.norm ? rope_unroll<true, true>() : rope_unroll<false, true>()) * (256 / D);  // heads
  for (int t = 0; t < 2; ++t) {
    p.t[t].heads = t == 0 ? d.n_q_heads : d.n_kv_heads;
    p.t[t].batches = (p.t[t].heads + per_batch - 1) / per_batch;
  }
  p.n_tokens = d.n_tokens;
  p.rot = d.rot_dim;
  p.n_axes = d.rot_dim > 0 ? d.n_axes : 0;
  p.axis1 = p.n_axes > 1 ? d.axis_pairs[0] : INT32_MAX;
  p.axis2 = p.n_axes > 2 ? d.axis_pairs[0] + d.axis_pairs[1] : INT32_MAX;
  p.eps = d.eps;
  p.amplitude = d.amplitude;
  const bool plain = d.rot_dim == D && !p.t[0].rows && !p.t[1].rows;
  const RopeKernel k = D == 128 ? pick<128>(d.half_layout, d.norm, bwd, plain) : pick<64>(d.half_layout, d.norm, bwd, plain);
  static PerDeviceInt resident[32];  // blocks per SM of each variant
  int per_sm = 0;
  cudaError_t e = resident[(D == 128) * 16 + plain * 8 + bwd * 4 + d.half_layout * 2 + d.norm].get(&per_sm, [&](int, int* v) {
    const cudaError_t r = cudaOccupancyMaxActiveBlocksPerMultiprocessor(v, k, kRopeThreads, 0);
    if (*v < 1) *v = 1;
    return r;
  });
  if (e != cudaSuccess) return e;
  // One wave of blocks, a warp per token; with fewer tokens than warps a token's heads are split over several
  // warps (each forms the token's sines again), down to one batch a warp.
  const int64_t warps = (int64_t)sms * per_sm * (kRopeThreads / 32);
  const int batches = p.t[0].batches + p.t[1].batches;
  int64_t chunks = warps / d.n_tokens;
  // weight gradients of a block's worth of tokens: one block and no second launch (3 us against 2 + 2)
  if (p.partial && d.n_tokens <= kRopeThreads / 32) {
    chunks = 1;
    p.partial = nullptr;
    p.dwq = dwq;
    p.dwk = dwk;
  }
  if (chunks > batches) chunks = batches;
  if (p.partial && chunks > kMaxDwBlocks) chunks = kMaxDwBlocks;
  if (chunks < 1) chunks = 1;
  p.chunk = (int)((batches + chunks - 1) / chunks);
  const int ny = (batches + p.chunk - 1) / p.chunk;
  int64_t nx = (d.n_tokens + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  const int64_t cap = ((int64_t)sms * per_sm + ny - 1) / ny;
  if (nx > cap) nx = cap;
  if (p.partial && nx * ny > kMaxDwBlocks) nx = kMaxDwBlocks / ny;
  if (nx < 1) nx = 1;
  e = launch_overlapped(k, dim3((unsigned)nx, (unsigned)ny), kRopeThreads, 0, stream, p);
  if (e != cudaSuccess || !p.partial) return e;
  return launch_overlapped(zl_qk_rope_dw_kernel, 2 * D / 32, 1024, 0, stream, p.partial, (int32_t)(nx * ny), D, dwq, dwk);
}

// SM count of the current device; the kernels are built for sm_103a alone.
zl_status check_device(int* sms) {
  static PerDeviceInt count;
  const cudaError_t e = count.get(sms, [](int dev, int* v) {
    int major = 0, minor = 0;
    cudaError_t r = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    if (r == cudaSuccess) r = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    if (r == cudaSuccess) r = cudaDeviceGetAttribute(v, cudaDevAttrMultiProcessorCount, dev);
    if (major != 10 || minor != 3) *v = -1;
    return r;
  });
  return e != cudaSuccess ? ZL_ERR_CUDA : *sms > 0 ? ZL_OK : ZL_ERR_UNSUPPORTED;
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
  if ((d->n_q_heads > 0 && !same_rows(q, q_stride, q_out, q_out_stride, d->n_tokens)) ||
      (d->n_kv_heads > 0 && !same_rows(k, k_stride, k_out, k_out_stride, d->n_tokens)))
    return ZL_ERR_INVALID_ARG;
  if (d->rot_dim > 0 && (!positions || !freq)) return ZL_ERR_INVALID_ARG;
  if (!numbers_aligned(q_weight, k_weight, positions, freq)) return ZL_ERR_ALIGN;
  int sms = 0;
  if ((s = check_device(&sms)) != ZL_OK) return s;
  RopeParams p{};
  p.t[0] = {static_cast<const __nv_bfloat16*>(q), nullptr, static_cast<__nv_bfloat16*>(q_out), q_weight, nullptr, q_stride, 0,
            q_out_stride, 0, 0};
  p.t[1] = {static_cast<const __nv_bfloat16*>(k), nullptr, static_cast<__nv_bfloat16*>(k_out), k_weight, nullptr, k_stride, 0,
            k_out_stride, 0, 0};
  p.positions = positions;
  p.freq = freq;
  return launch_rope(*d, false, sms, p, nullptr, nullptr, static_cast<cudaStream_t>(stream)) == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
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
  if ((d->n_q_heads > 0 && !same_rows(dq_out, dq_out_stride, dq, dq_stride, d->n_tokens)) ||
      (d->n_kv_heads > 0 && !same_rows(dk_out, dk_out_stride, dk, dk_stride, d->n_tokens)))
    return ZL_ERR_INVALID_ARG;
  if (d->rot_dim > 0 && (!positions || !freq)) return ZL_ERR_INVALID_ARG;
  if (!numbers_aligned(q_weight, k_weight, positions, freq) || !numbers_aligned(dq_weight, dk_weight, nullptr, nullptr))
    return ZL_ERR_ALIGN;
  int sms = 0;
  if ((s = check_device(&sms)) != ZL_OK) return s;
  RopeParams p{};
  p.t[0] = {static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(dq_out), static_cast<__nv_bfloat16*>(dq),
            q_weight, d->q_rows, q_stride, dq_out_stride, dq_stride, 0, 0};
  p.t[1] = {static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(dk_out), static_cast<__nv_bfloat16*>(dk),
            k_weight, d->k_rows, k_stride, dk_out_stride, dk_stride, 0, 0};
  p.positions = positions;
  p.freq = freq;
  p.partial = dw ? static_cast<float*>(workspace) : nullptr;
  return launch_rope(*d, true, sms, p, dq_weight, dk_weight, st) == cudaSuccess ? ZL_OK : ZL_ERR_CUDA;
}
