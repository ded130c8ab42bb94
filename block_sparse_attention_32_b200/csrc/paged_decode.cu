// Attention of one new token per sequence over a paged key-value cache, split
// over the cache's length and joined.  For sequence b of L tokens (the new
// one is token L - 1, already in the cache) and head h of group g, over the
// tokens J = {j < L : window = 0 or L - 1 - j < window or j < sink}:
//   o = sum_{j in J} softmax_{j in J}(scale q.k_j) v_j,  lse = ln sum e^{scale q.k_j}.
//
// Bound: HBM, on the visible tokens' K and V (512 bytes per token and KV head,
// read once); R <= 16 query heads share each of them, R flops a byte.  So the
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
// P is rounded to bf16 for the P V product (at most 2^-8 of a weight, averaged
// over the keys); l sums the fp32 weights.
// Measured: 64 sequences of 500 to 32768 tokens, 64 / 8 heads: 297 us with the
// join, 1.88 GB, 6.3 TB/s (0.97 of the copy rate).  One of 4093 tokens: 12.3 us, of
// which the reads are 2.6: a launch, three dependent memory latencies (lengths,
// table, tiles) and the join.  Windows of 4096, 37 sequences, 32 / 2 heads: 26.7 us; the
// kernel alone 18.5, of which the reads are 8.1, the join alone 8.3 (the same with pages of
// 16 and of 64): 3.7 tiles a warp, no more than start and end of its ring.
#include "common.cuh"
#include "layer_args.cuh"

namespace msa {

constexpr int kPdWarps = 6;
constexpr int kPdStages = 2;                        // per warp
constexpr int kPdTile = 32;                         // tokens
constexpr int kPdStageBytes = 2 * kPdTile * 256;    // K, V
constexpr int kPdThreads = 32 * kPdWarps;
constexpr int kPdMaxBatch = 4096;
// shared memory: the stages, barriers, small things, then the lengths and the tiles
// before each sequence (sized by the batch)
constexpr int kPdOffBar = kPdWarps * kPdStages * kPdStageBytes;
constexpr int kPdOffMisc = kPdOffBar + kPdWarps * kPdStages * 8;
constexpr int kPdOffLens = kPdOffMisc + 128;
constexpr int pd_smem_bytes(int batch) { return 1024 + kPdOffLens + (2 * batch + 1) * 4; }
static_assert(pd_smem_bytes(kPdMaxBatch) <= 232448, "shared memory per block");
constexpr int kPdMinTiles = 2;                      // tiles a warp at least takes
constexpr int kPdMaxBlocks = 148;                   // blocks at most (the workspace's size)

// the visible tokens of a sequence as tiles: nst tiles of sinks (when they do
// not run into the window's), then tiles first .. first + nt - nst - 1
struct SeqTiles {
  int32_t L, lo, nst, first, nt;
};
__device__ __forceinline__ SeqTiles seq_tiles(const PagedDecodeArgs& a, int32_t len) {
  SeqTiles t;
  t.L = max(0, min(len, a.cap));
  t.lo = max(0, t.L - a.window);
  t.first = t.lo / kPdTile;
  t.nst = (min(a.sink, t.lo) + kPdTile - 1) / kPdTile;
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
                                        const int32_t* prefix, const int32_t* lens, int32_t x) {
  int32_t lo = 0, hi = a.batch;                     // last b with G * prefix[b] <= x, nt > 0
  while (hi - lo > 1) {
    const int32_t mid = (lo + hi) >> 1;
    if (prefix[mid] * a.G <= x) lo = mid; else hi = mid;
  }
  c.b = lo;
  c.t = seq_tiles(a, lens[lo]);
  const uint32_t r = (uint32_t)(x - prefix[lo] * a.G);
  c.g = (int32_t)(r / (uint32_t)c.t.nt);
  c.j = (int32_t)(r - (uint32_t)(c.g * c.t.nt));
}
__device__ __forceinline__ void pd_next(PdCursor& c, const PagedDecodeArgs& a,
                                        const int32_t* lens) {
  if (++c.j < c.t.nt) return;
  c.j = 0;
  if (++c.g < a.G) return;
  c.g = 0;
  do {
    if (++c.b >= a.batch) return;
    c.t = seq_tiles(a, lens[c.b]);
  } while (c.t.nt == 0);
}
__device__ __forceinline__ int32_t pd_token(const SeqTiles& t, int32_t j) {
  return kPdTile * (j < t.nst ? j : t.first + j - t.nst);
}

// how `total` tiles (< 2^31, checked by the host) are dealt: nw workers, the first
// `more` of them with one tile more than the others
struct PdDeal {
  uint32_t total, nw, base, more;
  __device__ __forceinline__ PdDeal(uint32_t total_, uint32_t all) : total(total_) {
    nw = max(1u, min(all, (total + kPdMinTiles - 1) / kPdMinTiles));
    base = total / nw;
    more = total - base * nw;
  }
  __device__ __forceinline__ uint32_t start(uint32_t w) const { return w * base + min(w, more); }
  __device__ __forceinline__ uint32_t worker(uint32_t x) const {       // of tile x
    const uint32_t cut = more * (base + 1);
    return x < cut ? x / (base + 1) : more + (x - cut) / base;
  }
};

// kBox: tokens of a TMA box, min(page, 32).  A lane's accumulator rows are heads gq and
// gq + 8, for R <= 8 too (leaving the second out gained nothing: 33 us either way for
// 4 sequences of some 5000 tokens)
template <int kBox>
__global__ void __launch_bounds__(kPdThreads, 1)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ PagedDecodeArgs a) {
  extern __shared__ uint8_t smem_raw[];
  // (an offset, so that the compiler still knows the address space)
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  int32_t* lens = reinterpret_cast<int32_t*>(base + kPdOffLens);
  int32_t* prefix = lens + a.batch;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint64_t* full = reinterpret_cast<uint64_t*>(base + kPdOffBar) + warp * kPdStages;
  int32_t* wsum = reinterpret_cast<int32_t*>(base + kPdOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(wsum + 8);
  // pages of a stage's two 16-token halves that could not be read (bits 0, 1)
  int32_t* badbits = wsum + 9 + warp * kPdStages;
  static_assert(kPdStages * kPdWarps * 4 + 36 <= 128, "misc area");

  grid_launch_dependents();                // the join's blocks may take their places

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
      lens[b] = len;
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
      off += seq_tiles(a, lens[b]).nt;
    }
    if (b1 == a.batch && (b0 < b1 || tid == 0)) {
      prefix[a.batch] = off;
      if (blockIdx.x == 0) a.prefix[a.batch] = off;
    }
  }
  __syncthreads();

  const PdDeal deal((uint32_t)prefix[a.batch] * (uint32_t)a.G, gridDim.x * kPdWarps);
  const uint32_t w = warp * gridDim.x + blockIdx.x;             // neighbours on other SMs
  if (w >= deal.nw || deal.total == 0) return;
  const int32_t x0 = (int32_t)deal.start(w), x1 = (int32_t)deal.start(w + 1);

  uint8_t* ring = base + warp * kPdStages * kPdStageBytes;
  constexpr int kSub = kPdTile / kBox;     // boxes of a tile
  constexpr uint32_t kSubBytes = kBox * 256;
  PdCursor ic, cc;                         // issue and compute cursors
  pd_seek(ic, a, prefix, lens, x0);
  cc = ic;
  int32_t xi = x0;                         // next tile to issue
  // pages of the 32 tiles from pg_x on: lane l holds those of tile pg_x + l
  int32_t pg_x = x0;
  int32_t pg[2];
  auto load_pages = [&]() {
    pg[0] = pg[1] = -2;                    // -2: nothing visible, not touched
    if (lane < x1 - pg_x) {
      PdCursor c = ic;
      c.j += lane;
      if (c.j >= c.t.nt) pd_seek(c, a, prefix, lens, pg_x + lane);
      const int32_t tok = pd_token(c.t, c.j);
#pragma unroll
      for (int k = 0; k < kSub; ++k) {
        const int32_t t0 = tok + k * kBox;
        if (t0 >= c.t.L || (t0 + kBox <= c.t.lo && t0 >= a.sink)) continue;
        const int32_t pi = t0 >> a.page_shift;
        int32_t p = -1;
        if (pi < a.table_stride) p = __ldg(a.block_table + c.b * a.table_stride + pi);
        pg[k] = p >= 0 && p < a.n_pages ? p : -1;
        if (pg[k] == -1) report(a.err, MSA_DEVERR_BAD_PAGE);
      }
    }
    __syncwarp();
  };
  load_pages();
  // lane 0 brings tile xi into stage s
  auto issue = [&](int s) {
    if (xi >= x1) return;
    if (xi - pg_x >= 32) {
      pg_x = xi;
      load_pages();
    }
    const int src = xi - pg_x;
    const int32_t p0 = __shfl_sync(0xffffffffu, pg[0], src);
    const int32_t p1 = __shfl_sync(0xffffffffu, pg[1], src);
    if (lane == 0) {
      const int32_t tok = pd_token(ic.t, ic.j);
      const int32_t r0 = tok & ((1 << a.page_shift) - 1);
      uint8_t* st = ring + s * kPdStageBytes;
      badbits[s] = (p0 == -1 ? 1 : 0) | (p1 == -1 ? 2 : 0);
      const uint32_t n = (p0 >= 0 ? 1u : 0u) + (p1 >= 0 ? 1u : 0u);
      if (n == 0) mbar_arrive(full + s);
      else mbar_arrive_expect_tx(full + s, n * 2 * kSubBytes);
      if (p0 >= 0) {
        tma_load_5d(st, &tm_k, full + s, 0, r0, 0, ic.g, p0);
        tma_load_5d(st + kPdTile * 256, &tm_v, full + s, 0, r0, 0, ic.g, p0);
      }
      if (p1 >= 0) {
        tma_load_5d(st + kSubBytes, &tm_k, full + s, 0, 0, 0, ic.g, p1);
        tma_load_5d(st + kPdTile * 256 + kSubBytes, &tm_v, full + s, 0, 0, 0, ic.g, p1);
      }
    }
    ++xi;
    if (xi < x1) pd_next(ic, a, lens);
  };
  for (int s = 0; s < kPdStages; ++s) issue(s);

  const int gq = lane >> 2, tq = lane & 3;
  const float scale_log2 = a.scale * 1.4426950408889634f;
  // ldmatrix rows of this lane: K (keys 16 kp + (lane & 7) + 8 (lane >> 4), chunks
  // 2 ks + ((lane >> 3) & 1)), V (keys 16 kp + (lane & 15), chunks 2 dp + (lane >> 4))
  const int krow = (lane & 7) + ((lane >> 4) << 3), vrow = lane & 15;
  const uint32_t ring_s = smem_u32(ring);
  uint32_t koff[4], voff[4];               // of chunk pair c in a panel
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    koff[c] = krow * 128 + (((2 * c + ((lane >> 3) & 1)) ^ (krow & 7)) << 4);
    voff[c] = kPdTile * 256 + vrow * 128 + (((2 * c + (lane >> 4)) ^ (vrow & 7)) << 4);
  }
  uint32_t qf[8][4];
  float o[16][4], m[2], l[2];
  int32_t seg_j0 = 0;                     // first tile of the item in this run
  bool fresh = true, ok = true;
  uint32_t n = 0;
  for (int32_t x = x0; x < x1; ++x, ++n) {
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
    const uint32_t st = ring_s + s * kPdStageBytes;
    const int32_t tok = pd_token(cc.t, cc.j);
    const int32_t bad = badbits[s];
    uint32_t vis = 0xffffffffu;
    if (bad != 0 || tok + kPdTile > cc.t.L || (tok < cc.t.lo && tok + kPdTile > a.sink)) {
      const int32_t t = tok + lane;
      vis = __ballot_sync(0xffffffffu, t < cc.t.L && (t >= cc.t.lo || t < a.sink) &&
                                           !((bad >> (lane / kBox)) & 1));
      // clear the V rows nobody may see: a row per lane, chunks in an order that
      // keeps the lanes on different banks
      if (!((vis >> lane) & 1)) {
        uint8_t* row = ring + s * kPdStageBytes + kPdTile * 256 + (lane / kBox) * kSubBytes +
                       (lane % kBox) * 128;
#pragma unroll
        for (int c = 0; c < 16; ++c)
          *reinterpret_cast<uint4*>(row + (c >> 3) * (kBox * 128) + (((c + lane) & 7) << 4)) =
              make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();           // before the stage's next TMA write
      __syncwarp();
    }
    // S = Q K^T: heads (gq, gq + 8) x keys 8 nt + (2 tq, 2 tq + 1)
    float sc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
#pragma unroll
      for (int kp = 0; kp < 2; ++kp) {      // keys 16 kp .. + 15
        const uint32_t row = st + koff[ks & 3] + (ks >> 2) * (kBox * 128) +
                             (kBox == 32 ? kp * 2048u : kp * kSubBytes);
        uint32_t b0, b1, b2, b3;
        ldmatrix_x4(row, b0, b1, b2, b3);
        mma_bf16_16816(sc[2 * kp], qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], b0, b1);
        mma_bf16_16816(sc[2 * kp + 1], qf[ks][0], qf[ks][1], qf[ks][2], qf[ks][3], b2, b3);
      }
    }
    if (vis != 0xffffffffu) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!((vis >> (8 * i + 2 * tq + (e & 1))) & 1)) sc[i][e] = -INFINITY;
    }
    float mx[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mx[r] = fmaxf(sc[0][2 * r], sc[0][2 * r + 1]);
#pragma unroll
      for (int i = 1; i < 4; ++i) mx[r] = fmax3f(mx[r], sc[i][2 * r], sc[i][2 * r + 1]);
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
      mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
      mx[r] = fmaxf(m[r], mx[r] * scale_log2);
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
    uint32_t pf[4][2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const float z = m[r] == -INFINITY ? 0.f : -m[r];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p0 = ex2_approx(fmaf(sc[i][2 * r], scale_log2, z));
        const float p1 = ex2_approx(fmaf(sc[i][2 * r + 1], scale_log2, z));
        l[r] += p0 + p1;
        pf[i][r] = pack_bf16x2(p0, p1);
      }
    }
    // O += P V: heads x dims 8 nt + (2 tq, 2 tq + 1)
#pragma unroll
    for (int kp = 0; kp < 2; ++kp) {
#pragma unroll
      for (int dp = 0; dp < 8; ++dp) {    // dims 16 dp .. + 15
        const uint32_t row = st + voff[dp & 3] + (dp >> 2) * (kBox * 128) +
                             (kBox == 32 ? kp * 2048u : kp * kSubBytes);
        uint32_t b0, b1, b2, b3;
        ldmatrix_x4_trans(row, b0, b1, b2, b3);
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
      const bool whole = seg_j0 == 0 && item_ends;
      const int slot = seg_j0 == 0 ? 1 : 0;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float lt = l[r] + __shfl_xor_sync(0xffffffffu, l[r], 1);
        lt += __shfl_xor_sync(0xffffffffu, lt, 2);
        const int hr = gq + 8 * r;
        if (hr >= a.R) continue;
        if (whole) {
          const int64_t row = (int64_t)cc.b * a.G * a.R + cc.g * a.R + hr;
          const float inv = lt == 0.f ? 0.f : 1.f / lt;
          uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + row * kHeadDim);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            dst[4 * i + tq] = pack_bf16x2(o[i][2 * r] * inv, o[i][2 * r + 1] * inv);
          if (tq == 0)
            a.lse[row] = lt == 0.f ? -INFINITY : m[r] * 0.6931471805599453f + logf(lt);
        } else {
          const int64_t row = ((int64_t)w * 2 + slot) * a.R + hr;
          float* dst = a.part_acc + row * kHeadDim + 2 * tq;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            *reinterpret_cast<float2*>(dst + 8 * i) = make_float2(o[i][2 * r], o[i][2 * r + 1]);
          if (tq == 0) *reinterpret_cast<float2*>(a.part_ml + row * 2) = make_float2(m[r], lt);
        }
      }
      fresh = true;
    }
    if (x + 1 < x1) pd_next(cc, a, lens);
  }
  // no copy may still be writing shared memory when the block exits
  const uint32_t issued = (uint32_t)(xi - x0);
  if (!ok && lane == 0)
    for (uint32_t k = n; k < issued; ++k)
      mbar_drain(full + k % kPdStages, (uint32_t)((k / kPdStages) & 1), a.err);
}

// Joins an item's pieces in a fixed order, and writes the rows of empty
// sequences (o = 0, lse = -inf).  kSplit warps share a (sequence, head), each
// taking every kSplit-th piece, four on their way at a time, a lane 4 dims.  The
// blocks are in place before the pieces are complete (launched while the main
// kernel runs); nothing is read before grid_wait.
constexpr int kPdJoinWarps = 8;
template <int kSplit>
__global__ void __launch_bounds__(32 * kPdJoinWarps)
    paged_join_kernel(const __grid_constant__ PagedDecodeArgs a, uint32_t all_workers) {
  __shared__ float4 sacc[kSplit > 1 ? kPdJoinWarps : 1][32];
  __shared__ float2 sml[kPdJoinWarps];
  constexpr int kRowsBlock = kPdJoinWarps / kSplit;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t H = a.G * a.R, row = blockIdx.x * kRowsBlock + warp / kSplit;
  const uint32_t b = row / H, h = row - b * H, g = h / a.R, r = h - g * a.R;
  if (b >= a.batch) return;                // whole rows' warps (kSplit > 1: never)
  grid_wait();
  const int32_t p0 = a.prefix[b], nt = a.prefix[b + 1] - p0;
  float M = -INFINITY, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (nt > 0) {
    const PdDeal deal((uint32_t)a.prefix[a.batch] * (uint32_t)a.G, all_workers);
    const uint32_t x = (uint32_t)(p0 * a.G + g * nt);
    const uint32_t w0 = deal.worker(x), w1 = deal.worker(x + nt - 1);
    if (w0 == w1) return;                  // finished by its one worker
    for (uint32_t k0 = w0 + warp % kSplit; k0 <= w1; k0 += 4 * kSplit) {
      float2 ml[4];
      float4 v[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t k = k0 + u * kSplit;
        ml[u] = make_float2(-INFINITY, 0.f);
        v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k <= w1) {
          // the first piece is its worker's last item (slot 1), the others continue one (slot 0)
          const uint32_t p = (2 * k + (k == w0 ? 1 : 0)) * a.R + r;
          ml[u] = *reinterpret_cast<const float2*>(a.part_ml + p * 2);
          v[u] = *reinterpret_cast<const float4*>(a.part_acc + p * kHeadDim + 4 * lane);
        }
      }
      const float mx = fmaxf(fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)), M);
      const float z = mx == -INFINITY ? 0.f : mx, fo = ex2_approx(M - z);
      M = mx;
      L *= fo;
      acc = make_float4(acc.x * fo, acc.y * fo, acc.z * fo, acc.w * fo);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float f = ex2_approx(ml[u].x - z);
        L += f * ml[u].y;
        acc.x += f * v[u].x;
        acc.y += f * v[u].y;
        acc.z += f * v[u].z;
        acc.w += f * v[u].w;
      }
    }
  }
  if (kSplit > 1) {
    sacc[warp][lane] = acc;
    if (lane == 0) sml[warp] = make_float2(M, L);
    __syncthreads();
    if (warp != 0) return;
    M = -INFINITY;
#pragma unroll
    for (int k = 0; k < kSplit; ++k) M = fmaxf(M, sml[k].x);
    const float z = M == -INFINITY ? 0.f : M;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    L = 0.f;
#pragma unroll
    for (int k = 0; k < kSplit; ++k) {
      const float f = ex2_approx(sml[k].x - z);
      const float4 u = sacc[k][lane];
      acc.x += f * u.x;
      acc.y += f * u.y;
      acc.z += f * u.z;
      acc.w += f * u.w;
      L += f * sml[k].y;
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
  *reinterpret_cast<uint2*>(a.out + (int64_t)row * kHeadDim + 4 * lane) = make_uint2(
      pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (lane == 0) a.lse[row] = L == 0.f ? -INFINITY : M * 0.6931471805599453f + logf(L);
}

size_t paged_decode_workspace(int64_t batch, int32_t R) {
  const size_t pre = ((size_t)(batch + 1) * 4 + 15) / 16 * 16;
  return pre + (size_t)kPdMaxBlocks * kPdWarps * 2 * R * (2 + kHeadDim) * sizeof(float);
}

int64_t paged_decode_max_batch() { return kPdMaxBatch; }
int32_t paged_decode_tile() { return kPdTile; }

template <int kBox>
static cudaError_t launch_main(const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                               PagedDecodeArgs& a, uint32_t* workers, cudaStream_t st) {
  auto kernel = paged_decode_kernel<kBox>;
  static KernelSetup setup;
  int sms = 0;
  const cudaError_t e = kernel_setup(setup, reinterpret_cast<const void*>(kernel),
                                     pd_smem_bytes(kPdMaxBatch), 0, &sms);
  if (e != cudaSuccess) return e;
  const int grid = sms < kPdMaxBlocks ? sms : kPdMaxBlocks;
  *workers = (uint32_t)(grid * kPdWarps);
  kernel<<<grid, kPdThreads, pd_smem_bytes(a.batch), st>>>(tm_k, tm_v, a);
  return cudaGetLastError();
}

cudaError_t launch_paged_decode(const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                PagedDecodeArgs a, void* ws, cudaStream_t st) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  a.prefix = reinterpret_cast<int32_t*>(p);
  p += ((size_t)(a.batch + 1) * 4 + 15) / 16 * 16;
  a.part_acc = reinterpret_cast<float*>(p);
  a.part_ml = a.part_acc + (size_t)kPdMaxBlocks * kPdWarps * 2 * a.R * kHeadDim;
  uint32_t workers = 0;
  const bool small = a.page_size < kPdTile;
  const cudaError_t e = small ? launch_main<16>(tm_k, tm_v, a, &workers, st)
                              : launch_main<32>(tm_k, tm_v, a, &workers, st);
  if (e != cudaSuccess) return e;
  // a block for each row while all of them run at once (8 a SM; one sequence of 4093
  // tokens, L2 cold: 18 us, a warp for each 37), else a warp: there are few pieces a row
  // then (2048 sequences of up to 500 tokens, 64 heads: 215 us, a block for each 377)
  const unsigned rows = (unsigned)(a.batch * a.G * a.R);
  if (rows <= 8 * kPdMaxBlocks)
    return launch_dependent(paged_join_kernel<kPdJoinWarps>, rows, 32 * kPdJoinWarps, 0, st, a,
                            workers);
  return launch_dependent(paged_join_kernel<1>, (rows + kPdJoinWarps - 1) / kPdJoinWarps,
                          32 * kPdJoinWarps, 0, st, a, workers);
}

}  // namespace msa
