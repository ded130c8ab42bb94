// Per-head RMS norm of queries and keys with the rotary position embedding in
// the same pass: what stands between the projections and the attention (the
// path's inputs are rotated queries and keys).  For a head vector x of D
// features, weights w and the token's angles a_i:
//   y = w * x / sqrt(mean(x^2) + eps),
//   (y_a, y_b) -> (y_a cos a_i - y_b sin a_i, y_b cos a_i + y_a sin a_i)
// over the first `rot` features, paired (i, i + rot / 2) or (2 i, 2 i + 1).
// Backward, with xh = x / sqrt(mean(x^2) + eps) and dz the upstream gradient
// turned back by -a_i:
//   dw = sum over rows dz * xh,   dx = (dz w - xh mean(dz w xh)) / sqrt(...).
//
// Bound: HBM -- every value is read once and written once (2 + 2 bytes per
// feature forward).  A row lives in D / 8 lanes, 16 bytes each, so one load, a
// few shuffles (sum of squares; the partner feature, which for pairs (i, i +
// rot / 2) is always whole lanes away because rot is a multiple of 16) and
// one store do the work in registers.  The D / 8 lanes keep one token and walk
// `hc` of its heads: the token's cosines and sines (fp32, the size of two bf16
// rows) are read once per hc heads, kept in registers.  Everything is computed
// in fp32 and rounded to bf16 once, at the store.
#include "common.cuh"
#include "layer_args.cuh"

namespace msa {

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
  const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                    pack_bf16x2(x[6], x[7]));
}

// cosines and sines of the lane's 8 features: pairs (i, i + rot / 2): one per
// feature; adjacent pairs: entries 0..3, one per pair.  Lanes past rot keep 1, 0.
template <bool kInter>
__device__ __forceinline__ void load_angles(const float* __restrict__ row, int rot, int ln,
                                            float (&c)[8], float (&s)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i] = 1.f;
    s[i] = 0.f;
  }
  const int half = rot >> 1;
  if (8 * ln >= rot) return;
  if (kInter) {
    const float4 c0 = __ldg(reinterpret_cast<const float4*>(row + 4 * ln));
    const float4 s0 = __ldg(reinterpret_cast<const float4*>(row + half + 4 * ln));
    c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w;
    s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w;
  } else {
    const int i0 = 8 * ln < half ? 8 * ln : 8 * ln - half;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float4 c0 = __ldg(reinterpret_cast<const float4*>(row + i0) + j);
      const float4 s0 = __ldg(reinterpret_cast<const float4*>(row + half + i0) + j);
      c[4 * j] = c0.x; c[4 * j + 1] = c0.y; c[4 * j + 2] = c0.z; c[4 * j + 3] = c0.w;
      s[4 * j] = s0.x; s[4 * j + 1] = s0.y; s[4 * j + 2] = s0.z; s[4 * j + 3] = s0.w;
    }
  }
}

// turns y by the angles (sgn 1) or back (sgn -1); every lane of the warp calls it
template <bool kInter, int kLanes>
__device__ __forceinline__ void rotate8(float (&y)[8], const float (&c)[8], const float (&s)[8],
                                        int rot, int ln, float sgn) {
  if (kInter) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = y[2 * i], b = y[2 * i + 1], sn = sgn * s[i];
      y[2 * i] = a * c[i] - b * sn;
      y[2 * i + 1] = b * c[i] + a * sn;
    }
  } else {
    const int hl = rot >> 4;                       // lanes of one half
    const bool first = ln < hl;
    const int peer = 8 * ln < rot ? (first ? ln + hl : ln - hl) : ln;
    const float f = first ? -sgn : sgn;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = __shfl_sync(0xffffffffu, y[i], peer, kLanes);
      y[i] = y[i] * c[i] + f * o * s[i];
    }
  }
}

template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// position of token (b, i): -1 when the row is to be left alone (a negative
// position marks padding; one past the table is reported)
__device__ __forceinline__ int64_t token_pos(const NormRopeArgs& a, int64_t bt, int64_t i) {
  if (a.positions == nullptr) return a.pos0 + i;
  const int64_t p = __ldg(a.positions + bt);
  if (p >= a.n_pos) {
    report(a.err, MSA_DEVERR_BAD_POSITION);
    return -1;
  }
  return p;
}

constexpr int kNrThreads = 256;
constexpr int kNrUnroll = 4;       // rows in flight per lane

template <int kD, bool kInter, bool kPaged>
__global__ void __launch_bounds__(kNrThreads)
    norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int kLanes = kD / 8;
  const int ln = threadIdx.x % kLanes;
  const int64_t item = (int64_t)blockIdx.x * (kNrThreads / kLanes) + threadIdx.x / kLanes;
  const bool in = item < a.n_items;                 // lanes past the end still join the shuffles
  const int32_t per_tok = a.chunks[0] + a.chunks[1] + a.chunks[2];
  const int64_t bt = in ? item / per_tok : 0;
  int32_t ch = in ? (int32_t)(item - bt * per_tok) : 0;
  int kind = 0;
  if (ch >= a.chunks[0]) {
    ch -= a.chunks[0];
    kind = 1;
    if (ch >= a.chunks[1]) {
      ch -= a.chunks[1];
      kind = 2;
    }
  }
  const int64_t b = bt / a.n_tok, i = bt - b * a.n_tok;
  const int64_t pos = in ? token_pos(a, bt, i) : -1;
  bool live = pos >= 0;
  const int h0 = ch * a.hc, h1 = min(h0 + a.hc, a.heads[kind]);
  __nv_bfloat16* dst = nullptr;
  if (live) {
    dst = a.dst[kind] + 8 * ln;
    if (kPaged && kind > 0) {
      const int64_t pi = pos / a.page_size;
      const int64_t pg =
          pi < a.table_stride ? (int64_t)__ldg(a.block_table + b * a.table_stride + pi) : -1;
      if (pg < 0 || pg >= a.n_pages) {
        report(a.err, MSA_DEVERR_BAD_PAGE);
        live = false;
      }
      dst += pg * a.ds_b[kind] + (pos - pi * a.page_size) * a.ds_t[kind];
    } else {
      dst += b * a.ds_b[kind] + i * a.ds_t[kind];
    }
  }
  const __nv_bfloat16* src = a.src[kind] + b * a.ss_b[kind] + i * a.ss_t[kind] + 8 * ln;
  float c[8], s[8], w[8];
  const bool norm = !kPaged || kind < 2;
  load_angles<kInter>(a.table + (live ? pos : 0) * a.rot, live && norm ? a.rot : 0, ln, c, s);
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = 1.f;
  if (norm && a.w[kind] != nullptr) {
    const float4 w0 = __ldg(reinterpret_cast<const float4*>(a.w[kind] + 8 * ln));
    const float4 w1 = __ldg(reinterpret_cast<const float4*>(a.w[kind] + 8 * ln) + 1);
    w[0] = w0.x; w[1] = w0.y; w[2] = w0.z; w[3] = w0.w;
    w[4] = w1.x; w[5] = w1.y; w[6] = w1.z; w[7] = w1.w;
  }
  for (int hb = 0; hb < a.hc; hb += kNrUnroll) {
    uint4 v[kNrUnroll];
#pragma unroll
    for (int u = 0; u < kNrUnroll; ++u) {
      const int h = h0 + hb + u;
      v[u] = make_uint4(0, 0, 0, 0);
      if (live && h < h1) v[u] = *reinterpret_cast<const uint4*>(src + h * a.ss_h[kind]);
    }
#pragma unroll
    for (int u = 0; u < kNrUnroll; ++u) {
      const int h = h0 + hb + u;
      float x[8];
      unpack8(v[u], x);
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss += x[j] * x[j];
      ss = row_sum<kLanes>(ss);
      const float r = rsqrtf(ss * (1.f / kD) + a.eps);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = x[j] * r * w[j];
      rotate8<kInter, kLanes>(x, c, s, a.rot, ln, 1.f);
      if (live && h < h1)
        *reinterpret_cast<uint4*>(dst + h * a.ds_h[kind]) = norm ? pack8(x) : v[u];
    }
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
template <bool kF32>
__device__ __forceinline__ void load_dy(const void* p, int64_t off, uint4 (&v)[2]) {
  if (kF32) {
    v[0] = *reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(p) + off);
    v[1] = *reinterpret_cast<const uint4*>(reinterpret_cast<const float*>(p) + off + 4);
  } else {
    v[0] = *reinterpret_cast<const uint4*>(reinterpret_cast<const __nv_bfloat16*>(p) + off);
  }
}
template <bool kF32>
__device__ __forceinline__ void unpack_dy(const uint4 (&v)[2], float (&y)[8]) {
  if (kF32) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      y[4 * j] = u2f(v[j].x); y[4 * j + 1] = u2f(v[j].y);
      y[4 * j + 2] = u2f(v[j].z); y[4 * j + 3] = u2f(v[j].w);
    }
  } else {
    unpack8(v[0], y);
  }
}

// Persistent blocks: the lanes of a row keep their 8 features' weight-gradient
// sums in fp32 registers over all the rows they meet, then the block's rows
// are added in a fixed order and leave as one partial row; a second kernel adds
// the blocks in a fixed order.  No atomics: the same bits every run.
template <int kD, bool kInter, bool kF32>
__global__ void __launch_bounds__(kNrThreads)
    norm_rope_bwd_kernel(const __grid_constant__ NormRopeBwdArgs p) {
  constexpr int kLanes = kD / 8, kGroups = kNrThreads / kLanes, kU = 2;
  const NormRopeArgs& a = p.f;
  __shared__ float red[kGroups][kD + 4];
  const int ln = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
  const int32_t per_tok = a.chunks[0] + a.chunks[1];
  float dw[2][8];
#pragma unroll
  for (int j = 0; j < 8; ++j) dw[0][j] = dw[1][j] = 0.f;
  const int64_t step = (int64_t)gridDim.x * kGroups;
  // every group runs the same number of rounds, so the shuffles stay whole
  const int64_t rounds = (a.n_items + step - 1) / step;
  for (int64_t rd = 0; rd < rounds; ++rd) {
    const int64_t item = rd * step + (int64_t)blockIdx.x * kGroups + grp;
    const bool in = item < a.n_items;
    const int64_t bt = in ? item / per_tok : 0;
    int32_t ch = in ? (int32_t)(item - bt * per_tok) : 0;
    const int kind = ch >= a.chunks[0] ? 1 : 0;
    if (kind) ch -= a.chunks[0];
    const int64_t b = bt / a.n_tok, i = bt - b * a.n_tok;
    const int64_t pos = in ? token_pos(a, bt, i) : -1;
    const bool live = pos >= 0;
    const int h0 = ch * a.hc, h1 = min(h0 + a.hc, a.heads[kind]);
    const __nv_bfloat16* src = a.src[kind] + b * a.ss_b[kind] + i * a.ss_t[kind] + 8 * ln;
    __nv_bfloat16* dst = a.dst[kind] + b * a.ds_b[kind] + i * a.ds_t[kind] + 8 * ln;
    const int64_t yo = b * p.ys_b[kind] + i * p.ys_t[kind] + 8 * ln;
    float c[8], s[8], w[8];
    load_angles<kInter>(a.table + (live ? pos : 0) * a.rot, live ? a.rot : 0, ln, c, s);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 1.f;
    if (a.w[kind] != nullptr) {
      const float4 w0 = __ldg(reinterpret_cast<const float4*>(a.w[kind] + 8 * ln));
      const float4 w1 = __ldg(reinterpret_cast<const float4*>(a.w[kind] + 8 * ln) + 1);
      w[0] = w0.x; w[1] = w0.y; w[2] = w0.z; w[3] = w0.w;
      w[4] = w1.x; w[5] = w1.y; w[6] = w1.z; w[7] = w1.w;
    }
    float g[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = 0.f;
    for (int hb = 0; hb < a.hc; hb += kU) {
      uint4 xv[kU], yv[kU][2];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int h = h0 + hb + u;
        xv[u] = yv[u][0] = yv[u][1] = make_uint4(0, 0, 0, 0);
        if (live && h < h1) {
          xv[u] = *reinterpret_cast<const uint4*>(src + h * a.ss_h[kind]);
          load_dy<kF32>(p.dy[kind], yo + h * p.ys_h[kind], yv[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int h = h0 + hb + u;
        float x[8], y[8];
        unpack8(xv[u], x);
        unpack_dy<kF32>(yv[u], y);
        rotate8<kInter, kLanes>(y, c, s, a.rot, ln, -1.f);
        float ss = 0.f, sy = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          ss += x[j] * x[j];
          sy += x[j] * y[j] * w[j];
        }
        ss = row_sum<kLanes>(ss);
        sy = row_sum<kLanes>(sy);
        // absent rows (zeros) add nothing, with eps = 0 too (there r is infinite)
        const float r = live && h < h1 ? rsqrtf(ss * (1.f / kD) + a.eps) : 0.f;
        const float m = sy * r * (1.f / kD);         // mean(dz w xh)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float xh = x[j] * r;
          g[j] += y[j] * xh;
          x[j] = r * (y[j] * w[j] - xh * m);
        }
        if (live && h < h1) *reinterpret_cast<uint4*>(dst + h * a.ds_h[kind]) = pack8(x);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dw[0][j] += kind ? 0.f : g[j];
      dw[1][j] += kind ? g[j] : 0.f;
    }
  }
  for (int k = 0; k < 2; ++k) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) red[grp][8 * ln + j] = dw[k][j];
    __syncthreads();
    if (threadIdx.x < kD) {
      float t = 0.f;
#pragma unroll 8
      for (int r = 0; r < kGroups; ++r) t += red[r][threadIdx.x];
      p.part[((int64_t)blockIdx.x * 2 + k) * kD + threadIdx.x] = t;
    }
  }
}

// dw = sum over the blocks' partial rows: 32 columns x 32 row slices a block
__global__ void __launch_bounds__(1024)
    norm_rope_dw_kernel(const float* __restrict__ part, int32_t n_blocks, int32_t d,
                        float* __restrict__ dw_q, float* __restrict__ dw_k) {
  __shared__ float red[32][33];
  const int lane = threadIdx.x & 31, sl = threadIdx.x >> 5;
  const int col = blockIdx.x * 32 + lane;                    // 0 .. 2 d - 1
  float t = 0.f;
#pragma unroll 4
  for (int r = sl; r < n_blocks; r += 32) t += part[(int64_t)r * 2 * d + col];
  red[sl][lane] = t;
  __syncthreads();
  if (sl == 0) {
    float v = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) v += red[r][lane];
    float* out = col < d ? dw_q : dw_k;
    if (out != nullptr) out[col < d ? col : col - d] = v;
  }
}

template <int kD>
static void pick_fwd(const NormRopeArgs& a, bool inter, bool paged, unsigned grid,
                     cudaStream_t st) {
  if (paged) {
    if (inter) norm_rope_kernel<kD, true, true><<<grid, kNrThreads, 0, st>>>(a);
    else norm_rope_kernel<kD, false, true><<<grid, kNrThreads, 0, st>>>(a);
  } else {
    if (inter) norm_rope_kernel<kD, true, false><<<grid, kNrThreads, 0, st>>>(a);
    else norm_rope_kernel<kD, false, false><<<grid, kNrThreads, 0, st>>>(a);
  }
}

static void split_heads(NormRopeArgs& a, int kinds, int hc) {
  a.hc = hc;
  int64_t per_tok = 0;
  for (int k = 0; k < 3; ++k) {
    a.chunks[k] = k < kinds ? (a.heads[k] + hc - 1) / hc : 0;
    per_tok += a.chunks[k];
  }
  a.n_items = a.batch * a.n_tok * per_tok;
}

cudaError_t launch_norm_rope(NormRopeArgs a, int32_t d, bool inter, bool paged,
                             cudaStream_t st) {
  const int kinds = paged ? 3 : 2, groups = kNrThreads / (d / 8);
  // eight heads per token's angles when that still fills the GPU; two when it
  // does not, so that a decode step spreads over more SMs
  split_heads(a, kinds, 8);
  if (a.n_items < (int64_t)148 * 4 * groups) split_heads(a, kinds, 2);
  const int64_t grid = (a.n_items + groups - 1) / groups;
  if (grid == 0) return cudaSuccess;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  if (d == 128) pick_fwd<128>(a, inter, paged, (unsigned)grid, st);
  else pick_fwd<64>(a, inter, paged, (unsigned)grid, st);
  return cudaGetLastError();
}

constexpr int kNrBwdBlocks = 148 * 4;     // partial rows at most (the workspace's size)

size_t norm_rope_bwd_workspace(int32_t d) { return (size_t)kNrBwdBlocks * 2 * d * sizeof(float); }

template <int kD>
static void pick_bwd(const NormRopeBwdArgs& p, bool inter, bool f32, unsigned grid,
                     cudaStream_t st) {
  if (f32) {
    if (inter) norm_rope_bwd_kernel<kD, true, true><<<grid, kNrThreads, 0, st>>>(p);
    else norm_rope_bwd_kernel<kD, false, true><<<grid, kNrThreads, 0, st>>>(p);
  } else {
    if (inter) norm_rope_bwd_kernel<kD, true, false><<<grid, kNrThreads, 0, st>>>(p);
    else norm_rope_bwd_kernel<kD, false, false><<<grid, kNrThreads, 0, st>>>(p);
  }
}

cudaError_t launch_norm_rope_bwd(NormRopeBwdArgs p, int32_t d, bool inter, bool f32, float* dw_q,
                                 float* dw_k, cudaStream_t st) {
  const int groups = kNrThreads / (d / 8);
  split_heads(p.f, 2, 8);
  if (p.f.n_items < (int64_t)kNrBwdBlocks * groups) split_heads(p.f, 2, 2);
  const unsigned grid = (unsigned)min64((p.f.n_items + groups - 1) / groups, kNrBwdBlocks);
  if (d == 128) pick_bwd<128>(p, inter, f32, grid, st);
  else pick_bwd<64>(p, inter, f32, grid, st);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  norm_rope_dw_kernel<<<2 * d / 32, 1024, 0, st>>>(p.part, (int32_t)grid, d, dw_q, dw_k);
  return cudaGetLastError();
}

}  // namespace msa
