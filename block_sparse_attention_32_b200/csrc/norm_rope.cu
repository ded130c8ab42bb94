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
// feature forward, 4 + 2 or 6 + 2 backward).  A row lives in D / 8 lanes of 8
// features each (backward: D / 16 of 16).  For pairs (i, i + rot / 2) a lane takes
// features 4 l .. 4 l + 3 of both halves (two 8-byte loads), so that both partners of
// every pair are its own and the rotation needs no exchange; the features behind rot
// go to the lanes left over.  Only the sum of squares (and, backward, one more sum)
// crosses lanes.  A row's lanes keep one token and walk `hc` of its heads: the token's
// cosines and sines (fp32, the size of two bf16 rows) are read once per hc heads
// and kept in registers.  Everything is computed in fp32 and rounded to bf16 once,
// at the store.
// Measured: forward, 32768 tokens x (32 + 8) heads of 128: the kernel alone 110 us, 688
// MB, 6.2 TB/s (0.95 of the copy rate), a call after another 117 to 124.  Backward, 16384 x (64 + 8), bf16 gradients: 160 us, 915
// MB, 5.7 TB/s (0.87; the shuffles, unpacking and the two sums a row keep it from the
// rest).  64 tokens of a decode step into their pages: 5 us, a launch and a latency.
#include "common.cuh"
#include "layer_args.cuh"

namespace msa {

// A lane's 8 features as four packed fp32 pairs, arranged so that the partners of
// pair (0, 1 | 2, 3) sit in v[0] and v[2] (v[1] and v[3]), whatever the pairing.
struct Row8 {
  uint64_t v[4];
};
__device__ __forceinline__ uint64_t dup_f32x2(float x) {
  return pack_f32x2(__float_as_uint(x), __float_as_uint(x));
}
__device__ __forceinline__ float sum_f32x2(uint64_t x) {
  float a, b;
  unpack_f32x2(x, a, b);
  return a + b;
}
__device__ __forceinline__ uint64_t neg_f32x2(uint64_t x) { return x ^ 0x8000000080000000ull; }

template <bool kInter>
__device__ __forceinline__ void unpack8(const uint4& u, Row8& x) {
  constexpr uint32_t kHi = 0xFFFF0000u;
  if (kInter) {                       // a word holds both partners of a pair
    x.v[0] = pack_f32x2(u.x << 16, u.y << 16);
    x.v[2] = pack_f32x2(u.x & kHi, u.y & kHi);
    x.v[1] = pack_f32x2(u.z << 16, u.w << 16);
    x.v[3] = pack_f32x2(u.z & kHi, u.w & kHi);
  } else {
    x.v[0] = pack_f32x2(u.x << 16, u.x & kHi);
    x.v[1] = pack_f32x2(u.y << 16, u.y & kHi);
    x.v[2] = pack_f32x2(u.z << 16, u.z & kHi);
    x.v[3] = pack_f32x2(u.w << 16, u.w & kHi);
  }
}
// the same as plain floats: partners at j and j + 4
template <bool kInter>
__device__ __forceinline__ void floats8(const uint4& u, float (&x)[8]) {
  Row8 r;
  unpack8<kInter>(u, r);
#pragma unroll
  for (int j = 0; j < 4; ++j) unpack_f32x2(r.v[j], x[2 * j], x[2 * j + 1]);
}
template <bool kInter>
__device__ __forceinline__ uint4 words8(const float (&f)[8]) {
  if (kInter)
    return make_uint4(pack_bf16x2(f[0], f[4]), pack_bf16x2(f[1], f[5]), pack_bf16x2(f[2], f[6]),
                      pack_bf16x2(f[3], f[7]));
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
template <bool kInter>
__device__ __forceinline__ uint4 pack8(const Row8& x) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack_f32x2(x.v[i], f[2 * i], f[2 * i + 1]);
  return words8<kInter>(f);
}
// two runs of four fp32 values (o0.., o1..)
template <bool kInter>
__device__ __forceinline__ void arrange8(const float4& a, const float4& b, Row8& x) {
  auto pk = [](float lo, float hi) {
    return pack_f32x2(__float_as_uint(lo), __float_as_uint(hi));
  };
  if (kInter) {
    x.v[0] = pk(a.x, a.z);
    x.v[2] = pk(a.y, a.w);
    x.v[1] = pk(b.x, b.z);
    x.v[3] = pk(b.y, b.w);
  } else {
    x.v[0] = pk(a.x, a.y);
    x.v[1] = pk(a.z, a.w);
    x.v[2] = pk(b.x, b.y);
    x.v[3] = pk(b.z, b.w);
  }
}

// offsets of a lane's two runs of 4 features; `turns`: they are rotated
struct LanePos {
  int o0, o1, ang;     // ang: first of its 4 angles
  bool turns;
};
template <bool kInter>
__device__ __forceinline__ LanePos lane_pos(int ln, int rot) {
  LanePos p;
  if (kInter) {
    p.o0 = 8 * ln;
    p.o1 = 8 * ln + 4;
    p.ang = 4 * ln;
    p.turns = 8 * ln < rot;
  } else {
    const int half = rot >> 1;
    p.turns = 4 * ln < half;
    p.ang = 4 * ln;
    // rot is a multiple of 16, so the lanes behind rot / 8 hold whole runs of 8
    p.o0 = p.turns ? 4 * ln : 8 * ln;
    p.o1 = p.turns ? half + 4 * ln : 8 * ln + 4;
  }
  return p;
}
template <bool kInter>
__device__ __forceinline__ uint4 load_row(const __nv_bfloat16* p, const LanePos& l) {
  if (kInter) return *reinterpret_cast<const uint4*>(p + l.o0);
  const uint2 a = *reinterpret_cast<const uint2*>(p + l.o0);
  const uint2 b = *reinterpret_cast<const uint2*>(p + l.o1);
  return make_uint4(a.x, a.y, b.x, b.y);
}
template <bool kInter>
__device__ __forceinline__ void store_row(__nv_bfloat16* p, const LanePos& l, const uint4& v) {
  if (kInter) {
    *reinterpret_cast<uint4*>(p + l.o0) = v;
  } else {
    *reinterpret_cast<uint2*>(p + l.o0) = make_uint2(v.x, v.y);
    *reinterpret_cast<uint2*>(p + l.o1) = make_uint2(v.z, v.w);
  }
}

// cosines and sines of the lane's 4 pairs (1, 0 where nothing turns)
struct Angles {
  uint64_t c[2], s[2];
};
__device__ __forceinline__ void load_angles(const float* __restrict__ row, int rot,
                                            const LanePos& l, bool want, Angles& a) {
  a.c[0] = a.c[1] = dup_f32x2(1.f);
  a.s[0] = a.s[1] = 0ull;
  if (want && l.turns) {
    const ulonglong2 c = __ldg(reinterpret_cast<const ulonglong2*>(row + l.ang));
    const ulonglong2 s = __ldg(reinterpret_cast<const ulonglong2*>(row + (rot >> 1) + l.ang));
    a.c[0] = c.x;
    a.c[1] = c.y;
    a.s[0] = s.x;
    a.s[1] = s.y;
  }
}
template <bool kInter>
__device__ __forceinline__ void load_weights(const float* __restrict__ w, const LanePos& l,
                                             Row8& v) {
  float4 a = make_float4(1.f, 1.f, 1.f, 1.f), b = a;
  if (w != nullptr) {
    a = __ldg(reinterpret_cast<const float4*>(w + l.o0));
    b = __ldg(reinterpret_cast<const float4*>(w + l.o1));
  }
  arrange8<kInter>(a, b, v);
}

// turns y by the angles (kSign 1) or back (-1)
template <int kSign>
__device__ __forceinline__ void rotate8(Row8& y, const Angles& a) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint64_t p = y.v[i], q = y.v[i + 2];
    const uint64_t sp = kSign > 0 ? a.s[i] : neg_f32x2(a.s[i]), sm = neg_f32x2(sp);
    y.v[i] = fma_f32x2(q, sm, mul_f32x2(p, a.c[i]));
    y.v[i + 2] = fma_f32x2(p, sp, mul_f32x2(q, a.c[i]));
  }
}
__device__ __forceinline__ float dot8(const Row8& a, const Row8& b) {
  const uint64_t s0 = fma_f32x2(a.v[1], b.v[1], mul_f32x2(a.v[0], b.v[0]));
  const uint64_t s1 = fma_f32x2(a.v[3], b.v[3], mul_f32x2(a.v[2], b.v[2]));
  return sum_f32x2(add_f32x2(s0, s1));
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

constexpr int kNrThreads = 128;    // forward
constexpr int kNrBwdThreads = 256;
constexpr int kNrHeads = 8;        // heads of a token per item; all loaded before the first is used

template <int kD, bool kInter, bool kPaged>
__global__ void __launch_bounds__(kNrThreads)
    norm_rope_kernel(const __grid_constant__ NormRopeArgs a) {
  constexpr int kLanes = kD / 8;
  const int ln = threadIdx.x % kLanes;
  const LanePos lp = lane_pos<kInter>(ln, a.rot);
  const uint32_t item = blockIdx.x * (kNrThreads / kLanes) + threadIdx.x / kLanes;
  const bool in = item < a.n_items;                 // lanes past the end still join the shuffles
  const uint32_t per_tok = a.chunks[0] + a.chunks[1] + a.chunks[2];
  const uint32_t bt = in ? item / per_tok : 0;
  int32_t ch = in ? (int32_t)(item - bt * per_tok) : 0;
  int kind = 0;
  if (ch >= a.chunks[0]) {
    ch -= a.chunks[0];
    kind = 1;
    if (kPaged && ch >= a.chunks[1]) {
      ch -= a.chunks[1];
      kind = 2;
    }
  }
  const uint32_t b = bt / (uint32_t)a.n_tok, i = bt - b * (uint32_t)a.n_tok;
  const int h0 = ch * a.hc, h1 = min(h0 + a.hc, a.heads[kind]);
  const __nv_bfloat16* src =
      a.src[kind] + b * a.ss_b[kind] + i * a.ss_t[kind] + h0 * a.ss_h[kind];
  const int64_t pos = in ? token_pos(a, bt, i) : -1;
  bool live = pos >= 0;
  uint4 v[kNrHeads];
#pragma unroll
  for (int u = 0; u < kNrHeads; ++u) {
    v[u] = make_uint4(0, 0, 0, 0);
    if (live && h0 + u < h1) v[u] = load_row<kInter>(src + u * a.ss_h[kind], lp);
  }
  __nv_bfloat16* dst = nullptr;
  if (live) {
    dst = a.dst[kind] + h0 * a.ds_h[kind];
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
  Angles ang;
  Row8 wp;
  const bool norm = !kPaged || kind < 2;
  load_angles(a.table + (live ? pos : 0) * a.rot, a.rot, lp, live && norm, ang);
  load_weights<kInter>(norm ? a.w[kPaged ? min(kind, 1) : kind] : nullptr, lp, wp);
  // plain fp32 from here on: with packed pairs as in the backward the compiler needs more
  // registers and moves (32768 tokens, 40 heads: 131 us, 113 like this)
  float c[4], sn[4], w[8];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    unpack_f32x2(ang.c[j], c[2 * j], c[2 * j + 1]);
    unpack_f32x2(ang.s[j], sn[2 * j], sn[2 * j + 1]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) unpack_f32x2(wp.v[j], w[2 * j], w[2 * j + 1]);
#pragma unroll
  for (int u = 0; u < kNrHeads; ++u) {
    if (u >= a.hc) break;                           // the same for every lane
    float x[8];
    floats8<kInter>(v[u], x);
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss += x[j] * x[j];
    ss = row_sum<kLanes>(ss);
    const float r = rsqrtf(ss * (1.f / kD) + a.eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = x[j] * r * w[j];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float p = x[j], q = x[j + 4];
      x[j] = p * c[j] - q * sn[j];
      x[j + 4] = q * c[j] + p * sn[j];
    }
    if (live && h0 + u < h1)
      store_row<kInter>(dst + u * a.ds_h[kind], lp, norm ? words8<kInter>(x) : v[u]);
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------
// Backward lanes hold 16 features, two runs of 8 (D / 16 lanes a row): the sums'
// shuffles, the square root and the addresses of a row, half of the forward's kind of
// work, are shared by twice the features.  v[j] and v[j + 4] hold partners.
struct Row16 {
  uint64_t v[8];
};
template <bool kInter>
__device__ __forceinline__ LanePos lane_pos16(int ln, int rot) {
  LanePos p;
  p.ang = 8 * ln;
  if (kInter) {
    p.turns = 16 * ln < rot;
    p.o0 = 16 * ln;
    p.o1 = 16 * ln + 8;
  } else {
    const int half = rot >> 1;          // a multiple of 8
    p.turns = 8 * ln < half;
    p.o0 = p.turns ? 8 * ln : 16 * ln;
    p.o1 = p.turns ? half + 8 * ln : 16 * ln + 8;
  }
  return p;
}
template <bool kInter>
__device__ __forceinline__ void unpack16(const uint4& a, const uint4& b, Row16& x) {
  Row8 r0, r1;
  unpack8<kInter>(a, r0);               // runs of 8: (0, 1 | 2, 3) partners, or plain pairs
  unpack8<kInter>(b, r1);
  if (kInter) {
    x.v[0] = r0.v[0]; x.v[1] = r0.v[1]; x.v[2] = r1.v[0]; x.v[3] = r1.v[1];
    x.v[4] = r0.v[2]; x.v[5] = r0.v[3]; x.v[6] = r1.v[2]; x.v[7] = r1.v[3];
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x.v[j] = r0.v[j];
      x.v[4 + j] = r1.v[j];
    }
  }
}
template <bool kInter>
__device__ __forceinline__ void pack16(const Row16& x, uint4& a, uint4& b) {
  Row8 r0, r1;
  if (kInter) {
    r0.v[0] = x.v[0]; r0.v[1] = x.v[1]; r1.v[0] = x.v[2]; r1.v[1] = x.v[3];
    r0.v[2] = x.v[4]; r0.v[3] = x.v[5]; r1.v[2] = x.v[6]; r1.v[3] = x.v[7];
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r0.v[j] = x.v[j];
      r1.v[j] = x.v[4 + j];
    }
  }
  a = pack8<kInter>(r0);
  b = pack8<kInter>(r1);
}
// two runs of eight fp32 values
template <bool kInter>
__device__ __forceinline__ void arrange16(const uint4 (&u)[4], Row16& x) {
  Row8 r0, r1;
  auto f = [](const uint4& q) { return make_float4(u2f(q.x), u2f(q.y), u2f(q.z), u2f(q.w)); };
  arrange8<kInter>(f(u[0]), f(u[1]), r0);
  arrange8<kInter>(f(u[2]), f(u[3]), r1);
  if (kInter) {
    x.v[0] = r0.v[0]; x.v[1] = r0.v[1]; x.v[2] = r1.v[0]; x.v[3] = r1.v[1];
    x.v[4] = r0.v[2]; x.v[5] = r0.v[3]; x.v[6] = r1.v[2]; x.v[7] = r1.v[3];
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x.v[j] = r0.v[j];
      x.v[4 + j] = r1.v[j];
    }
  }
}
// feature of element e (0, 1) of v[j]
template <bool kInter>
__device__ __forceinline__ int feature16(const LanePos& l, int j, int e) {
  if (!kInter) return (j < 4 ? l.o0 : l.o1) + 2 * (j & 3) + e;
  const int i = 2 * (j & 3) + e;        // pair of the lane
  return l.o0 + 2 * i + (j >> 2);
}

template <bool kF32>
struct Grad16 {                         // a lane's upstream gradient as loaded
  uint4 u[kF32 ? 4 : 2];
};
template <bool kF32>
__device__ __forceinline__ void load_dy(const void* p, int64_t off, const LanePos& l,
                                        Grad16<kF32>& v) {
  if (kF32) {
    const float* y = reinterpret_cast<const float*>(p) + off;
    v.u[0] = *reinterpret_cast<const uint4*>(y + l.o0);
    v.u[1] = *reinterpret_cast<const uint4*>(y + l.o0 + 4);
    v.u[kF32 ? 2 : 0] = *reinterpret_cast<const uint4*>(y + l.o1);
    v.u[kF32 ? 3 : 1] = *reinterpret_cast<const uint4*>(y + l.o1 + 4);
  } else {
    const __nv_bfloat16* y = reinterpret_cast<const __nv_bfloat16*>(p) + off;
    v.u[0] = *reinterpret_cast<const uint4*>(y + l.o0);
    v.u[1] = *reinterpret_cast<const uint4*>(y + l.o1);
  }
}
__device__ __forceinline__ float dot16(const Row16& a, const Row16& b) {
  uint64_t s0 = mul_f32x2(a.v[0], b.v[0]), s1 = mul_f32x2(a.v[1], b.v[1]);
#pragma unroll
  for (int j = 2; j < 8; j += 2) {
    s0 = fma_f32x2(a.v[j], b.v[j], s0);
    s1 = fma_f32x2(a.v[j + 1], b.v[j + 1], s1);
  }
  return sum_f32x2(add_f32x2(s0, s1));
}

// Persistent blocks over the items, all of the queries' before the keys': the
// lanes of a row keep their 16 features' weight-gradient sums in fp32 registers
// over all the rows they meet, then the block's rows are added in a fixed order
// and leave as one partial row; a second kernel adds the blocks in a fixed
// order.  No atomics: the same bits every run.
template <int kD, bool kInter, bool kF32>
__global__ void __launch_bounds__(kNrBwdThreads, 2)
    norm_rope_bwd_kernel(const __grid_constant__ NormRopeBwdArgs p) {
  constexpr int kLanes = kD / 16, kGroups = kNrBwdThreads / kLanes, kU = kF32 ? 1 : 2;  // rows
  const NormRopeArgs& a = p.f;
  __shared__ float red[kGroups][kD + 4];            // the queries' sums, then the keys'
  grid_launch_dependents();
  const int ln = threadIdx.x % kLanes, grp = threadIdx.x / kLanes;
  const LanePos lp = lane_pos16<kInter>(ln, a.rot);
  Row16 g, w;
  auto weights = [&](const float* wp) {
    uint4 u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      u[j] = make_uint4(0x3f800000u, 0x3f800000u, 0x3f800000u, 0x3f800000u);
      if (wp != nullptr)
        u[j] = __ldg(reinterpret_cast<const uint4*>(wp + (j < 2 ? lp.o0 : lp.o1) + 4 * (j & 1)));
    }
    arrange16<kInter>(u, w);
  };
  auto put = [&](const Row16& x) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float t[2];
      unpack_f32x2(x.v[j], t[0], t[1]);
      red[grp][feature16<kInter>(lp, j, 0)] = t[0];
      red[grp][feature16<kInter>(lp, j, 1)] = t[1];
    }
  };
#pragma unroll
  for (int j = 0; j < 8; ++j) g.v[j] = 0ull;
  int cur = 0;                                      // kind that g belongs to
  weights(a.w[0]);
  const uint32_t n_items = (uint32_t)a.n_items;
  const uint32_t nq = (uint32_t)(a.batch * a.n_tok) * a.chunks[0];
  const uint32_t step = gridDim.x * kGroups;
  // every group runs the same number of rounds, so the shuffles stay whole
  const uint32_t rounds = (n_items + step - 1) / step;
  for (uint32_t rd = 0; rd < rounds; ++rd) {
    const uint32_t item = rd * step + blockIdx.x * kGroups + grp;
    const bool in = item < n_items;
    const int kind = in && item >= nq ? 1 : 0;
    const uint32_t it = in ? (kind ? item - nq : item) : 0;
    const uint32_t per = max(a.chunks[kind], 1);
    const uint32_t bt = it / per;
    const int32_t ch = (int32_t)(it - bt * per);
    const uint32_t b = bt / (uint32_t)a.n_tok, i = bt - b * (uint32_t)a.n_tok;
    if (in && kind != cur) {
      cur = kind;
      put(g);
#pragma unroll
      for (int j = 0; j < 8; ++j) g.v[j] = 0ull;
      weights(a.w[1]);
    }
    const int64_t pos = in ? token_pos(a, bt, i) : -1;
    const bool live = pos >= 0;
    const int h0 = ch * a.hc, n_h = live ? min(a.hc, a.heads[kind] - h0) : 0;
    const __nv_bfloat16* src =
        a.src[kind] + b * a.ss_b[kind] + i * a.ss_t[kind] + h0 * a.ss_h[kind];
    __nv_bfloat16* dst = a.dst[kind] + b * a.ds_b[kind] + i * a.ds_t[kind] + h0 * a.ds_h[kind];
    const int64_t yo = b * p.ys_b[kind] + i * p.ys_t[kind] + h0 * p.ys_h[kind];
    uint64_t c[4], sn[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c[j] = dup_f32x2(1.f);
      sn[j] = 0ull;
    }
    if (live && lp.turns) {
      const float* row = a.table + pos * a.rot + lp.ang;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const ulonglong2 u = __ldg(reinterpret_cast<const ulonglong2*>(row) + j);
        const ulonglong2 v = __ldg(reinterpret_cast<const ulonglong2*>(row + (a.rot >> 1)) + j);
        c[2 * j] = u.x; c[2 * j + 1] = u.y;
        sn[2 * j] = v.x; sn[2 * j + 1] = v.y;
      }
    }
    for (int hb = 0; hb < a.hc; hb += kU) {
      uint4 xv[kU][2];
      Grad16<kF32> yv[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        xv[u][0] = xv[u][1] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < (kF32 ? 4 : 2); ++j) yv[u].u[j] = make_uint4(0, 0, 0, 0);
        if (hb + u < n_h) {
          const __nv_bfloat16* x = src + (hb + u) * a.ss_h[kind];
          xv[u][0] = *reinterpret_cast<const uint4*>(x + lp.o0);
          xv[u][1] = *reinterpret_cast<const uint4*>(x + lp.o1);
          load_dy<kF32>(p.dy[kind], yo + (hb + u) * p.ys_h[kind], lp, yv[u]);
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        Row16 x, y;
        unpack16<kInter>(xv[u][0], xv[u][1], x);
        if (kF32) {
          const uint4 q[4] = {yv[u].u[0], yv[u].u[1], yv[u].u[kF32 ? 2 : 0], yv[u].u[kF32 ? 3 : 1]};
          arrange16<kInter>(q, y);
        } else {
          unpack16<kInter>(yv[u].u[0], yv[u].u[1], y);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {               // turned back
          const uint64_t q = y.v[j], r = y.v[j + 4];
          y.v[j] = fma_f32x2(r, sn[j], mul_f32x2(q, c[j]));
          y.v[j + 4] = fma_f32x2(q, neg_f32x2(sn[j]), mul_f32x2(r, c[j]));
        }
        float ss = dot16(x, x);
        Row16 yw;
#pragma unroll
        for (int j = 0; j < 8; ++j) yw.v[j] = mul_f32x2(y.v[j], w.v[j]);
        float sy = dot16(x, yw);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) {
          ss += __shfl_xor_sync(0xffffffffu, ss, o);
          sy += __shfl_xor_sync(0xffffffffu, sy, o);
        }
        // absent rows (zeros) add nothing, with eps = 0 too (there r is infinite)
        const float r = hb + u < n_h ? rsqrtf(ss * (1.f / kD) + a.eps) : 0.f;
        // dx = r (dz w) - x r^3 mean(dz w x)
        const float m = sy * r * (1.f / kD);
        const uint64_t r2 = dup_f32x2(r), f2 = dup_f32x2(-r * r * m);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          g.v[j] = fma_f32x2(y.v[j], mul_f32x2(x.v[j], r2), g.v[j]);
          x.v[j] = fma_f32x2(x.v[j], f2, mul_f32x2(yw.v[j], r2));
        }
        if (hb + u < n_h) {
          uint4 o0, o1;
          pack16<kInter>(x, o0, o1);
          __nv_bfloat16* d = dst + (hb + u) * a.ds_h[kind];
          *reinterpret_cast<uint4*>(d + lp.o0) = o0;
          *reinterpret_cast<uint4*>(d + lp.o1) = o1;
        }
      }
    }
  }
  // queries: what was put away at the change of kind, or what is at hand
  for (int k = 0; k < 2; ++k) {
    if (k == 0) {
      if (cur == 0) put(g);
    } else {
      if (cur == 0)
#pragma unroll
        for (int j = 0; j < 8; ++j) g.v[j] = 0ull;
      put(g);
    }
    __syncthreads();
    if (threadIdx.x < kD) {
      float t = 0.f;
#pragma unroll 8
      for (int r = 0; r < kGroups; ++r) t += red[r][threadIdx.x];
      p.part[((int64_t)blockIdx.x * 2 + k) * kD + threadIdx.x] = t;
    }
    __syncthreads();
  }
}

// dw = sum over the blocks' partial rows: 32 columns x 32 row slices a block
__global__ void __launch_bounds__(1024)
    norm_rope_dw_kernel(const float* part, int32_t n_blocks, int32_t d,
                        float* dw_q, float* dw_k) {
  __shared__ float red[32][33];
  grid_wait();
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
  // eight heads per token's angles when that still fills the GPU (2048 tokens x 40
  // heads: 14.4 us, with two 20.5); two when it does not, so that a decode step spreads
  // over more SMs (64 tokens: 6.2 us, with eight 8.2)
  split_heads(a, kinds, kNrHeads);
  if (a.n_items < (int64_t)148 * 4 * groups) split_heads(a, kinds, 2);
  if (a.n_items > 0x7FFFFF00) return cudaErrorInvalidValue;
  const int64_t grid = (a.n_items + groups - 1) / groups;
  if (d == 128) pick_fwd<128>(a, inter, paged, (unsigned)grid, st);
  else pick_fwd<64>(a, inter, paged, (unsigned)grid, st);
  return cudaGetLastError();
}

constexpr int kNrBwdBlocks = 148 * 2;     // the blocks that fit at once; the workspace's rows

size_t norm_rope_bwd_workspace(int32_t d) { return (size_t)kNrBwdBlocks * 2 * d * sizeof(float); }

template <int kD>
static void pick_bwd(const NormRopeBwdArgs& p, bool inter, bool f32, unsigned grid,
                     cudaStream_t st) {
  if (f32) {
    if (inter) norm_rope_bwd_kernel<kD, true, true><<<grid, kNrBwdThreads, 0, st>>>(p);
    else norm_rope_bwd_kernel<kD, false, true><<<grid, kNrBwdThreads, 0, st>>>(p);
  } else {
    if (inter) norm_rope_bwd_kernel<kD, true, false><<<grid, kNrBwdThreads, 0, st>>>(p);
    else norm_rope_bwd_kernel<kD, false, false><<<grid, kNrBwdThreads, 0, st>>>(p);
  }
}

cudaError_t launch_norm_rope_bwd(NormRopeBwdArgs p, int32_t d, bool inter, bool f32, float* dw_q,
                                 float* dw_k, cudaStream_t st) {
  const int groups = kNrBwdThreads / (d / 16);
  // eight heads or two, as forward, by the blocks that stay (64 tokens x 40 heads: 10.3
  // us with two, 14.4 with eight; 2048: 24.6 and 28; 16384 x 72: eight is the faster)
  split_heads(p.f, 2, 8);
  if (p.f.n_items < (int64_t)kNrBwdBlocks * groups * 4) split_heads(p.f, 2, 2);
  if (p.f.n_items > 0x7FFFFF00) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)min64((p.f.n_items + groups - 1) / groups, kNrBwdBlocks);
  if (d == 128) pick_bwd<128>(p, inter, f32, grid, st);
  else pick_bwd<64>(p, inter, f32, grid, st);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_dependent(norm_rope_dw_kernel, 2 * d / 32, 1024, 0, st, p.part, (int32_t)grid, d,
                          dw_q, dw_k);
}

}  // namespace msa
