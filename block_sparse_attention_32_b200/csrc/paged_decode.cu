// Attention of one new token per sequence over a paged key-value cache, split
// over the cache's length and joined.  For sequence b of L tokens (the new
// one is token L - 1, already in the cache) and head h of group g, over the
// tokens J = {j < L : window = 0 or L - 1 - j < window or j < sink}:
//   o = sum_{j in J} softmax_{j in J}(scale q.k_j) v_j,  lse = ln sum e^{scale q.k_j}.
//
// Bound: HBM, on the visible tokens' K and V (512 bytes per token and KV head,
// read once); R <= 16 query heads share each of them, 4 R flops a byte.  So the
// design keeps as many K/V bytes in flight as fit and splits them evenly:
//   * the tokens are cut into 32-token tiles (8 KB of K, 8 KB of V), and the
//     tiles of all (sequence, group) items, one after the other, are dealt to
//     all warps of the GPU in equal contiguous runs, whatever the sequences'
//     lengths are.  The lengths are read on the device, so a captured call
//     follows them;
//   * every warp is on its own: it streams its run through its own ring of TMA
//     stages (no block-wide barrier anywhere in the loop), finds the pages in
//     the block table 32 tiles ahead, and keeps one running softmax in
//     registers.  S = Q K^T and O = P V are warp tiles (mma.sync m16n8k16, the
//     heads of the group as the 16 rows), so P goes from accumulator to operand
//     in registers; a 128-row tensor-memory tile would be 1/8 to 1/128 full;
//   * an item that lies inside one warp's run is finished there; one that
//     crosses runs leaves a piece (m, l, acc) per run -- at most two per warp,
//     so the workspace does not depend on the lengths -- and a second kernel
//     joins the pieces in a fixed order (the same bits every run).
// Pages end inside tiles, tiles inside windows: tokens that are not visible
// are masked by a select on S, and their V rows are zeroed in shared memory, so
// whatever the cache holds there (NaN too) stays out.  Pages that hold no
// visible token are not touched: their table entries may be anything.
// P is rounded to bf16 for the P V product (relative 2^-9 a weight, averaged
// over the keys); l sums the fp32 weights.
#include "common.cuh"
#include "layer_args.cuh"

namespace msa {

constexpr int kPdWarps = 6;
constexpr int kPdStages = 2;                        // per warp
constexpr int kPdTile = 32;                         // tokens
constexpr int kPdStageBytes = 2 * kPdTile * 256;    // K, V
constexpr int kPdThreads = 32 * kPdWarps;
constexpr int kPdMaxBatch = 4096;
constexpr int kPdOffPrefix = kPdWarps * kPdStages * kPdStageBytes;
constexpr int kPdOffBar = kPdOffPrefix + (kPdMaxBatch + 4) * 4;
constexpr int kPdOffMisc = kPdOffBar + kPdWarps * kPdStages * 8;
constexpr int kPdSmemBytes = 1024 + kPdOffMisc + 64 + kPdWarps * 8;
static_assert(kPdSmemBytes <= 232448, "shared memory per block");
constexpr int kPdMinTiles = 2;                      // tiles a warp at least takes
constexpr int kPdMaxBlocks = 148;                   // blocks at most (the workspace's size)

// the visible tokens of a sequence as tiles: nst tiles of sinks (when they do
// not run into the window's), then tiles first .. first + nt - nst - 1
struct SeqTiles {
  int32_t L, lo, nst, first, nt;
};
__device__ __forceinline__ SeqTiles seq_tiles(const PagedDecodeArgs& a, int32_t len) {
  SeqTiles t;
  t.L = len < 0 ? 0 : (int32_t)min64(len, a.cap);
  t.lo = a.window > 0 ? (int32_t)max64(0, (int64_t)t.L - a.window) : 0;
  t.first = t.lo / kPdTile;
  t.nst = (int32_t)((min64(a.sink, t.lo) + kPdTile - 1) / kPdTile);
  if (t.nst >= t.first) {          // one run from the first token on
    t.first = t.nst > 0 ? 0 : t.first;
    t.nst = 0;
  }
  t.nt = t.nst + (t.L + kPdTile - 1) / kPdTile - t.first;
  return t;
}

// walks the tiles of a warp's run: item = (b, g), tile j of its sequence
struct PdCursor {
  int32_t b, g, j;
  SeqTiles t;
};
__device__ __forceinline__ void pd_seek(PdCursor& c, const PagedDecodeArgs& a,
                                        const int32_t* prefix, int64_t x) {
  int32_t lo = 0, hi = a.batch;                     // last b with G * prefix[b] <= x, nt > 0
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if ((int64_t)prefix[mid] * a.G <= x) lo = mid; else hi = mid;
  }
  c.b = lo;
  c.t = seq_tiles(a, __ldg(a.seq_lens + lo));
  const int64_t r = x - (int64_t)prefix[lo] * a.G;
  c.g = (int32_t)(r / c.t.nt);
  c.j = (int32_t)(r - (int64_t)c.g * c.t.nt);
}
__device__ __forceinline__ void pd_next(PdCursor& c, const PagedDecodeArgs& a) {
  if (++c.j < c.t.nt) return;
  c.j = 0;
  if (++c.g < a.G) return;
  c.g = 0;
  do {
    if (++c.b >= a.batch) return;
    c.t = seq_tiles(a, __ldg(a.seq_lens + c.b));
  } while (c.t.nt == 0);
}
__device__ __forceinline__ int32_t pd_token(const SeqTiles& t, int32_t j) {
  return kPdTile * (j < t.nst ? j : t.first + j - t.nst);
}

// the run of worker w among nw over `total` tiles, and the worker of tile x
__device__ __forceinline__ int64_t pd_start(int64_t w, int64_t nw, int64_t total) {
  return w * total / nw;
}
__device__ __forceinline__ int64_t pd_worker(int64_t x, int64_t nw, int64_t total) {
  return ((x + 1) * nw - 1) / total;
}
__device__ __forceinline__ int64_t pd_workers(int64_t all, int64_t total) {
  return max64(1, min64(all, (total + kPdMinTiles - 1) / kPdMinTiles));
}

__global__ void __launch_bounds__(kPdThreads, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ PagedDecodeArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  int32_t* prefix = reinterpret_cast<int32_t*>(base + kPdOffPrefix);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* full = reinterpret_cast<uint64_t*>(base + kPdOffBar) + warp * kPdStages;
  int32_t* wsum = reinterpret_cast<int32_t*>(base + kPdOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(wsum + 8);
  // pages of a stage's two 16-token halves that could not be read (bits 0, 1)
  int32_t* badbits = wsum + 9 + warp * kPdStages;
  static_assert(kPdStages * kPdWarps * 4 + 36 <= 64 + kPdWarps * 8, "misc area");

  if (tid == 0) {
    *abort_flag = 0;
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  if (lane == 0)
    for (int s = 0; s < kPdStages; ++s) mbar_init(full + s, 1);
  fence_mbarrier_init();
  // tiles before each sequence: every thread takes a contiguous share
  {
    const int per = (a.batch + kPdThreads - 1) / kPdThreads;
    const int b0 = min(tid * per, a.batch), b1 = min(b0 + per, a.batch);
    int32_t s = 0;
    for (int b = b0; b < b1; ++b) {
      const int32_t len = __ldg(a.seq_lens + b);
      if (blockIdx.x == 0 && (len < 0 || len > a.cap)) report(a.err, MSA_DEVERR_BAD_LENGTH);
      s += seq_tiles(a, len).nt;
    }
    int32_t inc = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int32_t off = inc - s;
    for (int w = 0; w < warp; ++w) off += wsum[w];
    for (int b = b0; b < b1; ++b) {
      prefix[b] = off;
      if (blockIdx.x == 0) a.prefix[b] = off;
      off += seq_tiles(a, __ldg(a.seq_lens + b)).nt;
    }
    if (b1 == a.batch && (b0 < b1 || tid == 0)) {
      prefix[a.batch] = off;
      if (blockIdx.x == 0) a.prefix[a.batch] = off;
    }
  }
  __syncthreads();

  const int64_t total = (int64_t)prefix[a.batch] * a.G;
  const int64_t nw = pd_workers((int64_t)gridDim.x * kPdWarps, total);
  const int64_t w = (int64_t)warp * gridDim.x + blockIdx.x;     // neighbours on other SMs
  if (w >= nw || total == 0) return;
  const int64_t x0 = pd_start(w, nw, total), x1 = pd_start(w + 1, nw, total);
  if (x0 >= x1) return;

  uint8_t* ring = base + warp * kPdStages * kPdStageBytes;
  const int box = min(a.page_size, kPdTile), nsub = kPdTile / box;
  const uint32_t sub_bytes = (uint32_t)box * 256;
  PdCursor ic, cc;                         // issue and compute cursors
  pd_seek(ic, a, prefix, x0);
  cc = ic;
  int64_t xi = x0;                         // next tile to issue
  // pages of the 32 tiles from pg_x on: lane l holds those of tile pg_x + l
  int64_t pg_x = x0;
  int32_t pg[2];
  auto load_pages = [&]() {
    PdCursor c = ic;
    const int64_t n = min64(32, x1 - pg_x);
    int32_t b = 0, tok = 0;
    bool need0 = false, need1 = false;
    for (int64_t k = 0; k < n; ++k) {      // walk the cursor, keep this lane's tile
      if (k == lane) {
        b = c.b;
        tok = pd_token(c.t, c.j);
        auto need = [&](int32_t t0) {
          return t0 < c.t.L && (t0 + box > c.t.lo || t0 < a.sink);
        };
        need0 = need(tok);
        need1 = nsub > 1 && need(tok + box);
      }
      if (k + 1 < n) pd_next(c, a);
    }
    auto page = [&](int32_t t0) {
      const int64_t pi = t0 / a.page_size;
      if (pi >= a.table_stride) return -1;
      const int32_t p = __ldg(a.block_table + b * a.table_stride + pi);
      return p >= 0 && p < a.n_pages ? p : -1;
    };
    pg[0] = need0 ? page(tok) : -2;        // -2: nothing visible, not touched
    pg[1] = need1 ? page(tok + box) : -2;
    if (pg[0] == -1 || pg[1] == -1) report(a.err, MSA_DEVERR_BAD_PAGE);
  };
  load_pages();
  // lane 0 brings tile xi into stage s
  auto issue = [&](int s) {
    if (xi >= x1) return;
    if (xi - pg_x >= 32) {
      pg_x = xi;
      load_pages();
    }
    const int src = (int)(xi - pg_x);
    const int32_t p0 = __shfl_sync(0xffffffffu, pg[0], src);
    const int32_t p1 = __shfl_sync(0xffffffffu, pg[1], src);
    if (lane == 0) {
      const int32_t tok = pd_token(ic.t, ic.j);
      const int32_t r0 = tok % a.page_size;
      uint8_t* st = ring + s * kPdStageBytes;
      badbits[s] = (p0 == -1 ? 1 : 0) | (p1 == -1 ? 2 : 0);
      const uint32_t n = (p0 >= 0 ? 1u : 0u) + (p1 >= 0 ? 1u : 0u);
      if (n == 0) mbar_arrive(full + s);
      else mbar_arrive_expect_tx(full + s, n * 2 * sub_bytes);
      if (p0 >= 0) {
        tma_load_5d(st, &tm_k, full + s, 0, r0, 0, ic.g, p0);
        tma_load_5d(st + kPdTile * 256, &tm_v, full + s, 0, r0, 0, ic.g, p0);
      }
      if (p1 >= 0) {
        tma_load_5d(st + sub_bytes, &tm_k, full + s, 0, 0, 0, ic.g, p1);
        tma_load_5d(st + kPdTile * 256 + sub_bytes, &tm_v, full + s, 0, 0, 0, ic.g, p1);
      }
    }
    ++xi;
    if (xi < x1) pd_next(ic, a);
  };
  for (int s = 0; s < kPdStages; ++s) issue(s);

  const int gq = lane >> 2, tq = lane & 3;
  const float scale_log2 = a.scale * 1.4426950408889634f;
  uint32_t qf[8][4];
  float o[16][4], m[2], l[2];
  int32_t seg_j0 = 0;                     // first tile of the item in this run
  bool fresh = true, ok = true;
  int64_t n = 0;
  for (int64_t x = x0; ok && x < x1; ++x, ++n) {
    if (fresh) {                          // a new item: its queries, an empty state
      fresh = false;
      seg_j0 = cc.j;
      const __nv_bfloat16* q0 = a.q + cc.b * a.qs_b + (int64_t)(cc.g * a.R + gq) * a.qs_h + 2 * tq;
      const bool v0 = gq < a.R, v1 = gq + 8 < a.R;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const __nv_bfloat16* p = q0 + 16 * ks;
        qf[ks][0] = v0 ? __ldg(reinterpret_cast<const uint32_t*>(p)) : 0u;
        qf[ks][1] = v1 ? __ldg(reinterpret_cast<const uint32_t*>(p + 8 * a.qs_h)) : 0u;
        qf[ks][2] = v0 ? __ldg(reinterpret_cast<const uint32_t*>(p + 8)) : 0u;
        qf[ks][3] = v1 ? __ldg(reinterpret_cast<const uint32_t*>(p + 8 * a.qs_h + 8)) : 0u;
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      m[0] = m[1] = -INFINITY;
      l[0] = l[1] = 0.f;
    }
    const int s = (int)(n % kPdStages);
    ok = mbar_wait(full + s, (uint32_t)((n / kPdStages) & 1), abort_flag, a.err);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    uint8_t* st = ring + s * kPdStageBytes;
    const uint32_t k_s = smem_u32(st), v_s = k_s + kPdTile * 256;
    const int32_t tok = pd_token(cc.t, cc.j);
    const int32_t bad = badbits[s];
    auto visible = [&](int r) {           // row r of the tile
      const int32_t t = tok + r;
      return t < cc.t.L && (t >= cc.t.lo || t < a.sink) && !((bad >> (r >= box ? 1 : 0)) & 1);
    };
    const uint32_t vis = __ballot_sync(0xffffffffu, visible(lane));
    if (vis != 0xffffffffu) {             // clear the V rows nobody may see
      for (int r = 0; r < kPdTile; ++r) {
        if ((vis >> r) & 1) continue;
        uint8_t* row = st + kPdTile * 256 + (r / box) * sub_bytes + (r % box) * 128;
        *reinterpret_cast<uint2*>(row + (lane >> 4) * (box * 128) + (lane & 15) * 8) =
            make_uint2(0, 0);
      }
      fence_proxy_async_smem();           // before the stage's next TMA write
      __syncwarp();
    }
    // S = Q K^T: heads (gq, gq + 8) x keys 8 nt + (2 tq, 2 tq + 1)
    float sc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
#pragma unroll
    for (int kp = 0; kp < 2; ++kp) {      // keys 16 kp .. + 15
      const int kr = 16 * kp + (lane & 7) + ((lane >> 4) << 3);
      const uint32_t row = k_s + (kr / box) * sub_bytes + (kr % box) * 128;
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const int ch = 2 * (ks & 3) + ((lane >> 3) & 1);
        uint32_t b0, b1, b2, b3;
        ldmatrix_x4(row + (ks >> 2) * (box * 128) + ((ch ^ (kr & 7)) << 4), b0, b1, b2, b3);
        mma_bf16_16816(sc[2 * kp], qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], b0, b1);
        mma_bf16_16816(sc[2 * kp + 1], qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], b2, b3);
      }
    }
    float mx[2] = {m[0], m[1]};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = 8 * i + 2 * tq;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sc[i][e] = (vis >> (c + (e & 1))) & 1 ? sc[i][e] * scale_log2 : -INFINITY;
        mx[e >> 1] = fmaxf(mx[e >> 1], sc[i][e]);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
    }
    if (__any_sync(0xffffffffu, mx[0] != m[0] || mx[1] != m[1])) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        // -inf - -inf (nothing visible yet) must give a factor, not NaN
        const float f = mx[r] == -INFINITY ? 1.f : ex2_approx(m[r] - mx[r]);
        l[r] *= f;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          o[i][2 * r] *= f;
          o[i][2 * r + 1] *= f;
        }
        m[r] = mx[r];
      }
    }
    const float z0 = m[0] == -INFINITY ? 0.f : m[0], z1 = m[1] == -INFINITY ? 0.f : m[1];
    uint32_t pf[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float p0 = ex2_approx(sc[i][0] - z0), p1 = ex2_approx(sc[i][1] - z0);
      const float p2 = ex2_approx(sc[i][2] - z1), p3 = ex2_approx(sc[i][3] - z1);
      l[0] += p0 + p1;
      l[1] += p2 + p3;
      pf[i][0] = pack_bf16x2(p0, p1);
      pf[i][1] = pack_bf16x2(p2, p3);
    }
    // O += P V: heads x dims 8 nt + (2 tq, 2 tq + 1)
#pragma unroll
    for (int kp = 0; kp < 2; ++kp) {
      const int kr = 16 * kp + (lane & 15);
      const uint32_t row = v_s + (kr / box) * sub_bytes + (kr % box) * 128;
#pragma unroll
      for (int dp = 0; dp < 8; ++dp) {    // dims 16 dp .. + 15
        const int ch = 2 * (dp & 3) + (lane >> 4);
        uint32_t b0, b1, b2, b3;
        ldmatrix_x4_trans(row + (dp >> 2) * (box * 128) + ((ch ^ (kr & 7)) << 4), b0, b1, b2, b3);
        mma_bf16_16816(o[2 * dp], pf[2 * kp][0], pf[2 * kp][1], pf[2 * kp + 1][0],
                       pf[2 * kp + 1][1], b0, b1);
        mma_bf16_16816(o[2 * dp + 1], pf[2 * kp][0], pf[2 * kp][1], pf[2 * kp + 1][0],
                       pf[2 * kp + 1][1], b2, b3);
      }
    }
    __syncwarp();                         // the stage has been read
    issue(s);

    const bool item_ends = cc.j + 1 == cc.t.nt;
    if (item_ends || x + 1 == x1) {       // the item's last tile here: out, or a piece
      float lt[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        lt[r] = l[r] + __shfl_xor_sync(0xffffffffu, l[r], 1);
        lt[r] += __shfl_xor_sync(0xffffffffu, lt[r], 2);
      }
      const bool whole = seg_j0 == 0 && item_ends;
      const int slot = seg_j0 == 0 ? 1 : 0;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int hr = gq + 8 * r;
        if (hr >= a.R) continue;
        if (whole) {
          const int64_t row = (int64_t)cc.b * a.G * a.R + cc.g * a.R + hr;
          const float inv = lt[r] == 0.f ? 0.f : 1.f / lt[r];
          uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + row * kHeadDim);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            dst[4 * i + tq] = pack_bf16x2(o[i][2 * r] * inv, o[i][2 * r + 1] * inv);
          if (tq == 0)
            a.lse[row] = lt[r] == 0.f ? -INFINITY : m[r] * 0.6931471805599453f + logf(lt[r]);
        } else {
          const int64_t row = (w * 2 + slot) * a.R + hr;
          float* dst = a.part_acc + row * kHeadDim + 2 * tq;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            *reinterpret_cast<float2*>(dst + 8 * i) = make_float2(o[i][2 * r], o[i][2 * r + 1]);
          if (tq == 0)
            *reinterpret_cast<float2*>(a.part_ml + row * 2) = make_float2(m[r], lt[r]);
        }
      }
      fresh = true;
    }
    if (x + 1 < x1) pd_next(cc, a);
  }
  // no copy may still be writing shared memory when the block exits
  const int64_t issued = xi - x0;
  if (!ok && lane == 0)
    for (int64_t k = n; k < issued; ++k)
      mbar_drain(full + k % kPdStages, (uint32_t)((k / kPdStages) & 1), a.err);
}

// Joins an item's pieces in the order of the workers' runs, and writes the rows
// of empty sequences (o = 0, lse = -inf).  One block per (sequence, head): each
// of 4 warps takes every fourth piece, a lane 4 dims.
__global__ void __launch_bounds__(128)
    paged_join_kernel(const __grid_constant__ PagedDecodeArgs a, int64_t all_workers) {
  __shared__ float4 sacc[4][32];
  __shared__ float sl[4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int H = a.G * a.R;
  const int b = blockIdx.x / H, h = blockIdx.x - b * H, g = h / a.R, r = h - g * a.R;
  const int64_t row = (int64_t)b * H + h;
  const int32_t p0 = a.prefix[b], nt = a.prefix[b + 1] - p0;
  if (nt == 0) {
    a.out[row * kHeadDim + threadIdx.x] = __float2bfloat16_rn(0.f);
    if (threadIdx.x == 0) a.lse[row] = -INFINITY;
    return;
  }
  const int64_t total = (int64_t)a.prefix[a.batch] * a.G;
  const int64_t nw = pd_workers(all_workers, total);
  const int64_t x = (int64_t)p0 * a.G + (int64_t)g * nt;
  const int64_t w0 = pd_worker(x, nw, total), w1 = pd_worker(x + nt - 1, nw, total);
  if (w0 == w1) return;                    // finished by its one worker
  // the first piece is its worker's last item (slot 1), the others continue one (slot 0)
  auto prow = [&](int64_t k) { return (2 * k + (k == w0 ? 1 : 0)) * a.R + r; };
  float M = -INFINITY;
  for (int64_t k = w0 + lane; k <= w1; k += 32) M = fmaxf(M, a.part_ml[prow(k) * 2]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float z = M == -INFINITY ? 0.f : M;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float L = 0.f;
#pragma unroll 4
  for (int64_t k = w0 + warp; k <= w1; k += 4) {
    const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + prow(k) * 2);
    const float4 v = *reinterpret_cast<const float4*>(a.part_acc + prow(k) * kHeadDim + 4 * lane);
    const float f = ex2_approx(ml.x - z);
    L += f * ml.y;
    acc.x += f * v.x;
    acc.y += f * v.y;
    acc.z += f * v.z;
    acc.w += f * v.w;
  }
  sacc[warp][lane] = acc;
  if (lane == 0) sl[warp] = L;
  __syncthreads();
  if (warp == 0) {
    float4 t = sacc[0][lane];
    float Ls = sl[0];
#pragma unroll
    for (int k = 1; k < 4; ++k) {
      const float4 u = sacc[k][lane];
      t.x += u.x;
      t.y += u.y;
      t.z += u.z;
      t.w += u.w;
      Ls += sl[k];
    }
    const float inv = Ls == 0.f ? 0.f : 1.f / Ls;
    uint2 pk = make_uint2(pack_bf16x2(t.x * inv, t.y * inv), pack_bf16x2(t.z * inv, t.w * inv));
    *reinterpret_cast<uint2*>(a.out + row * kHeadDim + 4 * lane) = pk;
    if (lane == 0) a.lse[row] = Ls == 0.f ? -INFINITY : M * 0.6931471805599453f + logf(Ls);
  }
}

size_t paged_decode_workspace(int64_t batch, int32_t R) {
  const size_t pre = ((size_t)(batch + 1) * 4 + 15) / 16 * 16;
  return pre + (size_t)kPdMaxBlocks * kPdWarps * 2 * R * (2 + kHeadDim) * sizeof(float);
}

int64_t paged_decode_max_batch() { return kPdMaxBatch; }
int32_t paged_decode_tile() { return kPdTile; }

cudaError_t launch_paged_decode(const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                PagedDecodeArgs a, void* ws, cudaStream_t st) {
  static KernelSetup setup;
  int sms = 0;
  cudaError_t e = kernel_setup(setup, reinterpret_cast<const void*>(paged_decode_kernel), kPdSmemBytes, 0, &sms);
  if (e != cudaSuccess) return e;
  const int grid = sms < kPdMaxBlocks ? sms : kPdMaxBlocks;
  const int64_t workers = (int64_t)grid * kPdWarps;
  uint8_t* p = static_cast<uint8_t*>(ws);
  a.prefix = reinterpret_cast<int32_t*>(p);
  p += ((size_t)(a.batch + 1) * 4 + 15) / 16 * 16;
  a.part_acc = reinterpret_cast<float*>(p);
  a.part_ml = a.part_acc + (size_t)kPdMaxBlocks * kPdWarps * 2 * a.R * kHeadDim;
  paged_decode_kernel<<<grid, kPdThreads, kPdSmemBytes, st>>>(tm_k, tm_v, a);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int64_t rows = (int64_t)a.batch * a.G * a.R;
  paged_join_kernel<<<(unsigned)rows, 128, 0, st>>>(a, workers);
  return cudaGetLastError();
}

}  // namespace msa
