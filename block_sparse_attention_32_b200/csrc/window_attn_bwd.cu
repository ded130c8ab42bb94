// Backward of the window attention (window_attn.cu).  With p_ij = e^{scale q_i.k_j -
// lse_i} over the keys J(t_i) that query i sees, D_i = dO_i.o_i and
// dS_ij = p_ij (dO_i.v_j - D_i):
//   dq_i = scale sum_j dS_ij k_j,  dk_j = scale sum_i dS_ij q_i,  dv_j = sum_i p_ij dO_i,
// the last two over every query and every head of the group that sees key j.
//
// Bound: the tensor cores.  One pass over (query, key) tiles would need five
// products a tile but leaves one of dq and dk, dv to be added up across CTAs:
// dq pieces of every (row, key block) cost more HBM time (W / 128 pieces of 512
// bytes a row, written and read) than products, and atomics would make the bits
// depend on their order.  So each output gets its own walk, 4 + 3 products a
// tile pair, and every sum stays in TMEM in a fixed order:
//   dk, dv item  keys = the 128 accumulator rows, K and V stay; Q and dO tiles
//                stream: S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q
//   dq item      query rows stay (Q, dO); K and V tiles stream:
//                S = Q K^T, dP = dO V^T, dQ += dS K
// Both are "stay x stream" products of one shape, so ONE persistent kernel runs
// both kinds of item through the same roles, dealt by a counter: the short dq
// items fill the tail that the long dk, dv items leave.  Which CTA takes an item
// changes no result.
//   warps 0-15  P and dS, four warpgroups: thread = accumulator row x 32 columns (with
//               two warpgroups a tile's softmax took 3300 clocks, more than its
//               products: two warps a scheduler do not cover their latencies)
//   warp 16     scheduler and TMA;  warp 19  -lse, -D of the streamed rows
//   warp 17     issues S and dP;  warp 18  issues dV and dK or dQ (the issue of eight
//               MMAs takes as long as they do: one warp for all of them left the
//               tensor core waiting)
// TMEM: two tile buffers, dV, dK or dQ: 128 columns each.  A tile lives in one
// buffer: S(n), read into registers; dP(n) over it, made while the exponentials are
// at work; then P(n) and dS(n) (bf16) over that, the A operands of the sums.  Tiles
// alternate between the buffers, so the sums of n - 1 and S(n + 1) run beside the
// softmax of n.  (With one buffer for S and P, another for dP and dS, S(n + 1) had to
// wait for dV(n): 4300 clocks a tile.)  Per tile: dP(n), dK(n-1), dV(n-1), S(n+1).
// Q and dO (K and V) slots are freed apart: three for the first, which S needs early
// and dK keeps late, two for the second.
// Where rows see few keys or sequences are short, tiles come twice, for the high and the
// low parts of P and dS (wb_plan, wb_item).
// A key block that many queries see (sinks; no window) is cut into chunks of
// query tiles whose fp32 sums a last kernel adds in chunk order; few row tiles of many
// keys share those among several dq items, added the same way.
// Measured: 8192 tokens, 64 / 8 heads, W = 1024, S = 4: 860 us (0.905 TFLOP of visible
// pairs' products: 1.05 PFLOP/s, 0.64 of the burst rate) + 50 for D and the work list.
// The tensor pipe is busy 0.55 of its cycles.  With the softmax taken out (timed, wrong
// results) the products and their loads alone take 690 us, without the loads 625: a
// product of two shared-memory operands needs all 128 bytes a clock of the shared memory,
// which the loads and the broadcasts of lse and D share; the barriers alone, five a tile,
// 355.  The exponentials and the broadcasts are not what is waited for (without either:
// 845 of 860).  Two sets of warps taking alternate tiles need 64 columns a thread:
// spilled, or with half the warps 1.2 times slower.
#include <type_traits>

#include "common.cuh"
#include "layer_args.cuh"
#include "window_tiles.cuh"

namespace msa {

namespace {
constexpr int kWbThreads = 640;
constexpr int kWbCtl = 16;             // first control warp
// registers per thread: 96 at launch (65536 / 640 rounded down to the allocation
// unit; the launcher checks the compiled count)
constexpr int kWbRegsAtLaunch = 96, kWbRegsControl = 64, kWbRegsMath = 104;
static_assert(kWbRegsControl + 4 * kWbRegsMath == 5 * kWbRegsAtLaunch,
              "warpgroup register shares must add up to the launch allocation");
constexpr int kWbOffStay = 0;                          // K, V or Q, dO: 32 KB each
constexpr int kWbOffStream = 65536;                    // 3 slots for Q or K, 2 for dO or V
constexpr int kWbSlots = 5;
constexpr int kWbOffMeta = kWbOffStream + kWbSlots * 32768;   // slots: -lse log2 e [128], -D [128]
constexpr int kWbMeta = 2;
constexpr int kWbOffBar = kWbOffMeta + kWbMeta * 1024;
enum {
  XB_ITEM_FULL = 0, XB_ITEM_EMPTY = 2, XB_STAY_FULL = 4, XB_STAY_EMPTY, XB_STR_FULL = 6,
  XB_STR_EMPTY = XB_STR_FULL + kWbSlots, XB_DS_FULL = XB_STR_EMPTY + kWbSlots,
  XB_DONE = XB_DS_FULL + 2, XB_META_FULL = XB_DONE + 2,
  XB_META_EMPTY = XB_META_FULL + kWbMeta, XB_S_FULL = XB_META_EMPTY + kWbMeta, XB_S_READ,
  XB_DP_FULL, XB_ACC_FULL, XB_ACC_EMPTY, XB_DRAIN, XB_COUNT = XB_DRAIN + 2
};
constexpr int kWbOffMisc = kWbOffBar + XB_COUNT * 8;
constexpr int kWbOffItem = (kWbOffMisc + 16 + 15) / 16 * 16;    // two slots
constexpr int kWbItemBytes = 112;
constexpr int kWbSmemBytes = kWbOffItem + 2 * kWbItemBytes;
static_assert(kWbSmemBytes <= 232448, "shared memory per block");
constexpr int kWbItemReaders = 19;     // warps that read an item's number: all but the scheduler

struct WindowBwdArgs {
  WindowArgs w;
  const float* delta;       // [B, n_q, H]
  const int2* table;        // [n_cut]: (key block, chunk), the same for every (batch, group)
  const int32_t* pbase;     // [nblk]: first partial of a cut block, -1 for an uncut one
  int32_t* counter;
  float* part;              // [B * G, n_part, 2, 128, 128]: dV, dK sums of a chunk
  float* part_q;            // [n_dq, kq, 128, 128]: dQ sums of a row tile's shares of its keys
  int32_t chunk, nblk, n_cut, n_part, n_dkv, n_all, kq;
};

// query tiles (128 / R tokens) that see key block c: [first, first + count)
__host__ __device__ __forceinline__ void wb_query_tiles(const WindowArgs& a, int64_t c,
                                                        int32_t& first, int32_t& count) {
  const int64_t k0 = c * 128, tpt = 128 / a.R;
  const int64_t lo = max64(0, k0 - a.q_pos0);
  int64_t hi = a.n_q - 1;
  if (a.window > 0 && k0 >= a.sink)
    hi = min64(hi, k0 + 126 - a.q_pos0 + min64(a.window, int64_t(1) << 40));
  first = (int32_t)(lo / tpt);
  count = hi < lo ? 0 : (int32_t)(hi / tpt) - first + 1;
}
__host__ __device__ __forceinline__ int32_t wb_chunks(int32_t count, int32_t chunk) {
  return count <= chunk ? 1 : (count + chunk - 1) / chunk;
}

constexpr int64_t kWbTwiceKeys = 4;         // keys a row
constexpr int64_t kWbTwiceTerms = 2048;     // tile pairs of one (batch, group) x keys a row

struct WbPlan {
  int64_t nblk, n_cut, n_part, c_lo, c_hi, n_dkv, n_dq;   // c_lo .. c_hi: the cut blocks' range
  int32_t chunk, kq;         // kq: items that share a row tile's keys
  bool twice;
};
WbPlan wb_plan(const WindowArgs& a) {
  WbPlan p{};
  p.nblk = (a.n_kv + 127) / 128;
  int64_t total = 0;
  for (int64_t c = 0; c < p.nblk; ++c) {
    int32_t f, n;
    wb_query_tiles(a, c, f, n);
    total += n;
  }
  // Tiles twice: rounded to bf16, P and dS leave 2^-8 of each term in a gradient, as much as
  // the result's own rounding does.  Where terms cancel (sum_j dS_ij = 0: few keys a row) or
  // are few, that is neither small beside the sum nor averaged over many roundings (random
  // inputs, error over that of 32-bit sums rounded once: 1.43 where terms are many, 1.5 to 1.9
  // for rows of 2 to 4 keys and for a few tiles).  There each tile comes twice, and the second
  // time the sums take what the rounding of P and dS left (2^-17 remains).  The rule asks
  // for the shape of one sequence, not for how many of them, or of groups, a call has: the
  // same sequence's gradients are as exact in a batch as alone.  A training step of 3 x 97
  // tokens, 8 / 1 heads, L2 cold: 48 us, once 44; 64 x 97: 95 and 76; 32 x 256, 32 / 4 heads:
  // 337 and 243, 8192 tokens, 32 / 4 heads, window 8: 286 and 220, so not there.
  int64_t keys = a.q_pos0 + a.n_q;
  if (a.window > 0) keys = min64(keys, min64(a.window, keys) + a.sink);
  p.twice = total * keys <= kWbTwiceTerms || keys <= kWbTwiceKeys;
  total *= a.batch * a.G;
  // Tiles of a chunk: at least 4 (where they come twice, 2), few while SMs stand idle (512
  // tokens, 8 / 1 heads, no window: 4 tiles 46 us, 8: 52, 32: 83); then a 90th of all tiles,
  // 0.6 chunks an SM, up to 32.  More and shorter chunks fill the SMs, and leave more fp32
  // sums to be added: with a 74th, 90th, 120th, 148th (one an SM), 3 ragged x 1111 tokens
  // take 115, 109, 105, 105 us, 1024 tokens of 16 / 2 heads 62, 62, 66, 69 (with 32 tiles 97).
  // Past 32 * 296 tiles a chunk is a 296th: two an SM at most, which bounds the workspace.
  p.chunk = (int32_t)max64(max64(p.twice ? 2 : 4, min64(32, (total + 89) / 90)),
                           (total + 295) / 296);
  p.c_lo = p.nblk;
  for (int64_t c = 0; c < p.nblk; ++c) {
    int32_t f, n;
    wb_query_tiles(a, c, f, n);
    const int32_t k = wb_chunks(n, p.chunk);
    p.n_cut += k;
    if (k > 1) {
      p.n_part += k;
      p.c_lo = min64(p.c_lo, c);
      p.c_hi = c + 1;
    }
  }
  p.n_dkv = p.n_cut * a.batch * a.G;
  p.n_dq = a.batch * a.G * ((a.n_q * a.R + 127) / 128);
  // few row tiles of many keys: up to eight items a tile, four key tiles each at least (a
  // training step of one query over 4096 keys, 8 / 1 heads, L2 cold: 49 us, 78 in one; 16 over
  // 32768, 16 / 2 heads: 125 and 385; 16 over 1024: 59 and 65)
  p.kq = 1;
  while (p.kq < 8 && p.n_dq * p.kq * 2 <= 148 && keys >= 1024 * p.kq) p.kq *= 2;
  return p;
}
size_t pad32(size_t n) { return (n + 31) / 32 * 32; }

// one work item, as every role sees it: decoded once by the scheduler and kept in
// shared memory, so that the softmax warps need not hold it in registers
struct WbItem {
  bool dkv, end;             // end: there are no more
  int32_t b, g, nt;          // nt: steps, a streamed tile each
  int32_t half;              // 1: tiles come twice, in adjacent steps; else 0
  int32_t k0, q_tile, part;  // dkv: first key, first query tile, partial (-1: final)
  int32_t len;
  WinItem w;                 // dq
};
static_assert(sizeof(WbItem) <= kWbItemBytes, "an item's slot");
template <bool kTwice>
__device__ __forceinline__ void wb_item(WbItem& it, const WindowBwdArgs& p, int32_t idx) {
  const WindowArgs& a = p.w;
  const int32_t bg_all = (int32_t)a.batch * a.G;
  it.dkv = idx < p.n_dkv;
  if (it.dkv) {
    const int32_t e = idx / bg_all, bg = idx - e * bg_all;
    it.b = bg / a.G;
    it.g = bg - it.b * a.G;
    const int2 t = p.table[e];
    int32_t first, count;
    wb_query_tiles(a, t.x, first, count);
    const int32_t k = wb_chunks(count, p.chunk);
    const int32_t q0 = (int32_t)((int64_t)count * t.y / k);
    int32_t q1 = (int32_t)((int64_t)count * (t.y + 1) / k);
    it.k0 = t.x * 128;
    it.q_tile = first + q0;
    it.part = k > 1 ? bg * p.n_part + p.pbase[t.x] + t.y : -1;
    it.len = win_len(a, it.b);
    const int64_t live = (int64_t)it.len - a.q_pos0;         // queries before the padding
    const int32_t tpt = 128 / a.R;
    const int32_t end = live <= 0 || it.k0 >= it.len ? 0 : (int32_t)((live + tpt - 1) / tpt);
    it.nt = max(0, min(q1 - q0, end - it.q_tile));
  } else {
    const int32_t e = idx - p.n_dkv, tile = e / p.kq, c = e - tile * p.kq;
    win_item(it.w, a, tile, 1);
    it.part = p.kq > 1 ? e : -1;
    it.w.j0 = it.w.nt * c / p.kq;
    it.w.nt = it.w.nt * (c + 1) / p.kq - it.w.j0;
    it.b = it.w.b;
    it.g = it.w.g;
    it.nt = it.w.nt;
    it.len = it.w.len;
  }
  // else it is the row tile whose first rows see at most kWbTwiceKeys keys (dq: one item of
  // a sequence and group; one sequence of 8192 tokens, 64 / 8 heads, no window: 1505 us, without
  // 1493)
  it.half = kTwice || (!it.dkv && it.w.i0 == 0 && a.q_pos0 < kWbTwiceKeys) ? 1 : 0;
  it.nt <<= it.half;
}

}  // namespace

// D = dO.o of every row: 16 lanes of 8 features a row, 4 rows in flight a lane; the
// last block lays out the cut key blocks and sets the item counter back
constexpr int kWbPrepRows = 64;        // rows of a 256-thread block
__global__ void __launch_bounds__(256)
    window_bwd_prep_kernel(const __grid_constant__ WindowArgs a, float* __restrict__ delta,
                           int2* __restrict__ table, int32_t* __restrict__ pbase,
                           int32_t* __restrict__ counter, int32_t chunk, int32_t nblk) {
  const int lane = threadIdx.x & 31;
  grid_launch_dependents();
  if (blockIdx.x + 1 < gridDim.x) {
    const uint32_t H = (uint32_t)(a.G * a.R), n = (uint32_t)a.n_q;
    const uint32_t rows = (uint32_t)a.batch * n * H;
    const uint32_t r0 = blockIdx.x * kWbPrepRows + (threadIdx.x >> 4);
    const int c = 8 * (threadIdx.x & 15);
    uint4 ov[4], dv[4];
    uint2 rv[4];                       // the 8 bits behind each o, when kept
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t r = min(r0 + 16 * u, rows - 1);
      const uint32_t bt = r / H, h = r - bt * H, b = bt / n, t = bt - b * n;
      ov[u] = *reinterpret_cast<const uint4*>(a.o + b * a.os_b + t * a.os_t + h * a.os_h + c);
      dv[u] = *reinterpret_cast<const uint4*>(a.d_o + b * a.ds_b + t * a.ds_t + h * a.ds_h + c);
      rv[u] = make_uint2(0u, 0u);
      if (a.rest != nullptr)
        rv[u] = *reinterpret_cast<const uint2*>(a.rest + (int64_t)r * kHeadDim + c);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t x[4] = {ov[u].x, ov[u].y, ov[u].z, ov[u].w};
      const uint32_t y[4] = {dv[u].x, dv[u].y, dv[u].z, dv[u].w};
      const uint32_t z[2] = {rv[u].x, rv[u].y};
      // o as fp32 bits: (bf16 << 16) + (signed rest << 8)
      auto rest = [&](int i) {
        return (uint32_t)((int32_t)(z[i >> 2] << (24 - 8 * (i & 3))) >> 16) & 0xFFFFFF00u;
      };
      float s = 0.f;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        s += u2f((x[q] << 16) + rest(2 * q)) * u2f(y[q] << 16) +
             u2f((x[q] & 0xFFFF0000u) + rest(2 * q + 1)) * u2f(y[q] & 0xFFFF0000u);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if ((lane & 15) == 0 && r0 + 16 * u < rows) delta[r0 + 16 * u] = s;
    }
    return;
  }
  __shared__ int2 wsum[8], carry;
  const int tid = threadIdx.x, warp = tid >> 5;
  if (tid == 0) {
    *counter = 0;
    carry = make_int2(0, 0);
  }
  for (int32_t c0 = 0; c0 < nblk; c0 += 256) {
    const int32_t c = c0 + tid;
    int32_t first, count = 0, k = 0;
    if (c < nblk) {
      wb_query_tiles(a, c, first, count);
      k = wb_chunks(count, chunk);
    }
    int2 inc = make_int2(k, k > 1 ? k : 0);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, inc.x, o);
      const int y = __shfl_up_sync(0xffffffffu, inc.y, o);
      if (lane >= o) {
        inc.x += x;
        inc.y += y;
      }
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int2 off = carry;
    for (int w = 0; w < warp; ++w) {
      off.x += wsum[w].x;
      off.y += wsum[w].y;
    }
    if (c < nblk) {
      const int32_t e = off.x + inc.x - k;
      for (int32_t j = 0; j < k; ++j) table[e + j] = make_int2(c, j);
      pbase[c] = k > 1 ? off.y + inc.y - k : -1;
    }
    __syncthreads();
    if (tid == 255) carry = make_int2(off.x + inc.x, off.y + inc.y);
    __syncthreads();
  }
}

// two bf16, or (low) what their rounding leaves, rounded
__device__ __forceinline__ uint32_t pack_part(float u, float v, bool low) {
  const uint32_t h = pack_bf16x2(u, v);
  return low ? pack_bf16x2(u - u2f(h << 16), v - u2f(h & 0xFFFF0000u)) : h;
}

// kTwice: every streamed tile comes twice, for the high and the low parts of P and dS
template <bool kTwice>
__global__ void __launch_bounds__(kWbThreads, 1)
    window_attn_bwd_kernel(const __grid_constant__ CUtensorMap tm_q,
                           const __grid_constant__ CUtensorMap tm_do,
                           const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v,
                           const __grid_constant__ CUtensorMap tm_k32,
                           const __grid_constant__ CUtensorMap tm_v32,
                           const __grid_constant__ WindowBwdArgs p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = smem_raw;
  uint64_t* bar = reinterpret_cast<uint64_t*>(base + kWbOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + kWbOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base + kWbOffMisc + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const WindowArgs& a = p.w;
  int32_t* err = a.err;
  grid_launch_dependents();

  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar + XB_ITEM_FULL + s, 1);
      mbar_init(bar + XB_ITEM_EMPTY + s, kWbItemReaders);
      mbar_init(bar + XB_DS_FULL + s, 16);          // a lane of each warp
      mbar_init(bar + XB_DONE + s, 1);
    }
    for (int s = 0; s < kWbSlots; ++s) {
      mbar_init(bar + XB_STR_FULL + s, 1);
      mbar_init(bar + XB_STR_EMPTY + s, 1);
    }
    for (int s = 0; s < kWbMeta; ++s) {
      mbar_init(bar + XB_META_FULL + s, 1);
      mbar_init(bar + XB_META_EMPTY + s, 16);
    }
    mbar_init(bar + XB_STAY_FULL, 1);
    mbar_init(bar + XB_STAY_EMPTY, 1);
    mbar_init(bar + XB_S_FULL, 1);
    mbar_init(bar + XB_S_READ, 16);
    mbar_init(bar + XB_DP_FULL, 1);
    mbar_init(bar + XB_ACC_FULL, 1);
    mbar_init(bar + XB_ACC_EMPTY, 16);
    mbar_init(bar + XB_DRAIN, 1);
    mbar_init(bar + XB_DRAIN + 1, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == kWbCtl + 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;          // tile buffers 0, 1, dV, dK or dQ: 128 columns each
  // k-th completion of a barrier has parity k & 1; the whole warp decides together
  auto W = [&](int id, uint32_t k) {
    return __all_sync(0xffffffffu, mbar_wait(bar + id, k & 1u, abort_flag, err));
  };
  auto arrive = [&](int id) {                // for the whole warp
    __syncwarp();
    if (lane == 0) mbar_arrive(bar + id);
  };
  // slot and use of streamed tile m: half 0 (Q or K) goes round three, half 1 two
  auto slot_of = [](int h, uint32_t m) { return h ? 3 + (int)(m & 1) : (int)(m % 3); };
  auto use_of = [](int h, uint32_t m) { return h ? m >> 1 : m / 3; };
  auto item_slot = [&](uint32_t k) -> WbItem& {
    return *reinterpret_cast<WbItem*>(base + kWbOffItem + (int)(k & 1) * kWbItemBytes);
  };
  // the k-th item has been decoded (false: no more); a reading warp gives it back when done
  auto next_item = [&](uint32_t k) {
    return W(XB_ITEM_FULL + (int)(k & 1), k >> 1) && !item_slot(k).end;
  };
  auto done_item = [&](uint32_t k) { arrive(XB_ITEM_EMPTY + (int)(k & 1)); };
  const int32_t tpt = 128 / a.R;             // tokens per query tile
  // streamed tile of step t
  auto tile_of = [](const WbItem& it, int32_t t) { return t >> (kTwice ? 1 : it.half); };
  const float log2e = 1.4426950408889634f;

  if (warp >= kWbCtl) {
    setmaxnreg_dec<kWbRegsControl>();
    if (warp == kWbCtl) {
      // ---------------- scheduler, TMA ----------------
      if (lane == 0) {
        prefetch_tensormap(&tm_q);
        prefetch_tensormap(&tm_do);
        prefetch_tensormap(&tm_k);
        prefetch_tensormap(&tm_v);
      }
      grid_wait();                           // the work list and its counter are written
      uint32_t n = 0, ni = 0, issued[2] = {0, 0};   // streamed tiles, items with tiles
      bool ok = true;
      WbItem it{};
      auto load = [&](uint8_t* dst, const CUtensorMap* tm, uint64_t* b, int32_t y, int32_t z) {
        tma_load_4d(dst, tm, b, 0, y, z, it.b);
        tma_load_4d(dst + 16384, tm, b, 64, y, z, it.b);
      };
      for (uint32_t k = 0; ok; ++k) {
        if (k >= 2 && !W(XB_ITEM_EMPTY + (int)(k & 1), (k >> 1) - 1)) break;
        int32_t idx = 0;
        if (lane == 0) idx = atomicAdd(p.counter, 1);
        idx = __shfl_sync(0xffffffffu, idx, 0);
        it.end = idx >= p.n_all;
        if (!it.end) wb_item<kTwice>(it, p, idx);
        if (lane == 0) {
          item_slot(k) = it;
          mbar_arrive(bar + XB_ITEM_FULL + (int)(k & 1));
        }
        __syncwarp();
        if (it.end) break;
        if (it.nt == 0) continue;
        if (ni > 0 && !W(XB_STAY_EMPTY, ni - 1)) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar + XB_STAY_FULL, 65536u);
          const int32_t y = it.dkv ? it.k0 : it.g * a.R, z = it.dkv ? it.g : it.w.i0;
          load(base + kWbOffStay, it.dkv ? &tm_k : &tm_q, bar + XB_STAY_FULL, y, z);
          load(base + kWbOffStay + 32768, it.dkv ? &tm_v : &tm_do, bar + XB_STAY_FULL, y, z);
        }
        ++ni;
        for (int32_t t = 0; t < it.nt; ++t, ++n) {
          for (int h = 0; ok && h < 2; ++h) {
            const int s = slot_of(h, n);
            const uint32_t use = use_of(h, n);
            ok = use == 0 || W(XB_STR_EMPTY + s, use - 1);
            if (ok && lane == 0) {
              mbar_arrive_expect_tx(bar + XB_STR_FULL + s, 32768u);
              uint8_t* dst = base + kWbOffStream + s * 32768;
              if (it.dkv)
                load(dst, h ? &tm_do : &tm_q, bar + XB_STR_FULL + s, it.g * a.R,
                     (it.q_tile + tile_of(it, t)) * tpt);
              else
                win_load_keys(dst, h ? &tm_v : &tm_k, h ? &tm_v32 : &tm_k32,
                              bar + XB_STR_FULL + s, it.w, it.w.j0 + tile_of(it, t));
            }
            if (ok) issued[h] = n + 1;
          }
          if (!ok) break;
        }
      }
      // no copy may still be writing shared memory when the block exits
      if (lane == 0) {
        for (int h = 0; h < 2; ++h)
          for (uint32_t k = issued[h] > 3 ? issued[h] - 3 : 0; k < issued[h]; ++k)
            if (k + (h ? 2 : 3) >= issued[h])
              mbar_drain(bar + XB_STR_FULL + slot_of(h, k), use_of(h, k) & 1u, err);
        if (ni > 0) mbar_drain(bar + XB_STAY_FULL, (uint32_t)((ni - 1) & 1), err);
      }
    } else if (warp == kWbCtl + 1) {
      // ---------------- S, dP ----------------
      constexpr uint32_t kIdT = idesc_bf16_f32(128, 128, 0);
      const uint32_t sa = smem_u32(base + kWbOffStay), str = smem_u32(base + kWbOffStream);
      uint32_t n = 0, ni = 0;                // tiles, items with tiles
      bool ok = true;
      // D = X Y^T of two 128 x 128 tiles in shared memory
      auto product = [&](uint32_t d, uint32_t xa, uint32_t ya) {
        const uint64_t xd = smem_desc_sw128(xa, 16, 1024), yd = smem_desc_sw128(ya, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {     // the start address counts 16-byte units
          const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) / 16;
          umma_bf16(d, xd + off, yd + off, kIdT, kk > 0 ? 1u : 0u);
        }
      };
      // half h (Q or K; dO or V) of tile t (number m) has landed; its rows past the
      // sequence are cleared: they may hold anything, and their P and dS are 0, but
      // 0 * NaN is not.  (V needs none: a column of dP that nobody sees is dropped.)
      auto landed = [&](const WbItem& it, int h, int32_t t, uint32_t m) {
        const int s = slot_of(h, m);
        if (!W(XB_STR_FULL + s, use_of(h, m))) return false;
        if (it.len < a.n_kv && (a.kv_len != nullptr || !it.dkv) && (it.dkv || h == 0)) {
          uint8_t* rows = base + kWbOffStream + s * 32768;
          if (it.dkv)
            win_clear_rows(rows,
                           (it.len - (int32_t)a.q_pos0 - (it.q_tile + tile_of(it, t)) * tpt) * a.R,
                           128, lane);
          else
            win_clear_keys(rows, it.w, it.w.j0 + tile_of(it, t), lane);
        }
        return true;
      };
      // S of tile t, into the buffer that tile m - 2 has left
      auto issue_s = [&](const WbItem& it, int32_t t, uint32_t m) {
        if (!landed(it, 0, t, m)) return false;
        if (m >= 2 && !W(XB_DONE + (int)(m & 1), (m >> 1) - 1)) return false;
        tc_fence_after();
        if (elect_one()) {
          product(tmem + 128 * (m & 1), sa, str + slot_of(0, m) * 32768);
          umma_commit(bar + XB_S_FULL);
        }
        __syncwarp();
        return true;
      };
      for (uint32_t k = 0; ok && next_item(k); ++k) {
        const WbItem& it = item_slot(k);
        const bool dkv = it.dkv;
        const int32_t nt = it.nt;
        if (nt > 0) ok = W(XB_STAY_FULL, ni) && issue_s(it, 0, n);
        if (!ok) break;
        for (int32_t t = 0; t < nt; ++t, ++n) {
          // dP over S, once that is in registers
          if (!landed(it, 1, t, n) || !W(XB_S_READ, n)) { ok = false; break; }
          tc_fence_after();
          if (elect_one()) {
            const uint32_t b = n & 1;
            product(tmem + 128 * b, sa + 32768, str + slot_of(1, n) * 32768);
            umma_commit(bar + XB_DP_FULL);
            if (!dkv) umma_commit(bar + XB_STR_EMPTY + slot_of(1, n));  // V's last use
            if (t + 1 == nt) umma_commit(bar + XB_STAY_EMPTY);
          }
          __syncwarp();
          if (t + 1 < nt && !issue_s(it, t + 1, n + 1)) { ok = false; break; }
        }
        if (nt > 0) ++ni;
        if (ok) done_item(k);
      }
      // every MMA issued has finished before the tensor memory is freed
      if (elect_one()) {
        umma_commit(bar + XB_DRAIN);
        mbar_drain(bar + XB_DRAIN, 0, err);
      }
      __syncwarp();
    } else if (warp == kWbCtl + 2) {
      // ---------------- dV, dK or dQ ----------------
      constexpr uint32_t kIdA = idesc_bf16_f32(128, 128, 1);
      const uint32_t str0 = smem_u32(base + kWbOffStream);
      uint32_t n = 0, ni = 0;
      bool ok = true;
      // D (+)= X Y, X (bf16, runs of 32 elements, 32 columns apart) in TMEM, Y in shared memory
      auto product = [&](uint32_t d, uint32_t x, uint32_t ya, bool add) {
        const uint64_t yd = smem_desc_sw128(ya, 16384, 1024);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          umma_bf16_ts(d, x + (kk >> 1) * 32 + (kk & 1) * 8, yd + kk * (2048 / 16), kIdA,
                       add || kk > 0 ? 1u : 0u);
      };
      for (uint32_t k = 0; ok && next_item(k); ++k) {
        const bool dkv = item_slot(k).dkv;
        const int32_t nt = item_slot(k).nt;
        done_item(k);
        if (nt == 0) continue;
        if (ni > 0 && !W(XB_ACC_EMPTY, ni - 1)) { ok = false; break; }
        for (int32_t t = 0; t < nt; ++t, ++n) {
          const uint32_t b = n & 1, x = tmem + 128 * b;
          const int s0 = slot_of(0, n), s1 = slot_of(1, n);
          // the tiles it reads (landed long ago; V's slot may have been refilled)
          if (!W(XB_STR_FULL + s0, use_of(0, n))) { ok = false; break; }
          if (dkv && !W(XB_STR_FULL + s1, use_of(1, n))) { ok = false; break; }
          if (!W(XB_DS_FULL + (int)b, n >> 1)) { ok = false; break; }
          tc_fence_after();
          if (elect_one()) {
            product(tmem + 384, x + 16, str0 + s0 * 32768, t > 0);
            umma_commit(bar + XB_STR_EMPTY + s0);
            if (dkv) {
              product(tmem + 256, x, str0 + s1 * 32768, t > 0);
              umma_commit(bar + XB_STR_EMPTY + s1);
            }
            umma_commit(bar + XB_DONE + b);
            if (t + 1 == nt) umma_commit(bar + XB_ACC_FULL);
          }
          __syncwarp();
        }
        ++ni;
      }
      if (elect_one()) {
        umma_commit(bar + XB_DRAIN + 1);
        mbar_drain(bar + XB_DRAIN + 1, 0, err);
      }
      __syncwarp();
    } else {
      // ------------ -lse log2 e, -D of the streamed rows (dk, dv) or the item's (dq) ------------
      grid_wait();                           // and so is D
      uint32_t n = 0;                        // slots filled: one per tile, or per dq item
      bool ok = true;
      for (uint32_t k = 0; ok && next_item(k); ++k) {
        const WbItem& it = item_slot(k);
        const int32_t nt = it.dkv ? it.nt : min(it.nt, 1);
        const int32_t q_tile = it.dkv ? it.q_tile : it.w.i0 / tpt;
        for (int32_t t = 0; t < nt; ++t, ++n) {
          const int s = (int)(n % kWbMeta);
          float v[4][2];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int r = 32 * u + lane;
            const int64_t i = (int64_t)(q_tile + (kTwice ? t >> 1 : t)) * tpt + r / a.R;
            const bool live = i < a.n_q && a.q_pos0 + i < it.len;
            const int64_t row =
                ((int64_t)it.b * a.n_q + i) * ((int64_t)a.G * a.R) + it.g * a.R + r % a.R;
            // padding: p = 2^{0 - inf} = 0
            v[u][0] = live ? -log2e * __ldg(a.lse + row) : -INFINITY;
            v[u][1] = live ? -p.delta[row] : 0.f;
          }
          if (n >= kWbMeta && !W(XB_META_EMPTY + s, n / kWbMeta - 1)) { ok = false; break; }
          float* m = reinterpret_cast<float*>(base + kWbOffMeta + s * 1024);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            m[32 * u + lane] = v[u][0];
            m[128 + 32 * u + lane] = v[u][1];
          }
          arrive(XB_META_FULL + s);
        }
        if (ok) done_item(k);
      }
    }
  } else {
    setmaxnreg_inc<kWbRegsMath>();
    // ---------------- P, dS; outputs ----------------
    const int wg = warp >> 2, row = (warp & 3) * 32 + lane, c0 = 32 * wg;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const float scale_log2 = a.scale * log2e;
    const uint64_t scale2 = pack_f32x2(__float_as_uint(scale_log2), __float_as_uint(scale_log2));
    const int64_t H = (int64_t)a.G * a.R;
    uint32_t n = 0, nm = 0, ni = 0;          // tiles, slots of lse and D, items with tiles
    bool ok = true;
    for (uint32_t k = 0; ok && next_item(k); ++k) {
      const WbItem& it = item_slot(k);
      // dq: this thread's query row
      auto query = [&]() { return it.w.i0 + row / a.R; };
      auto qrow = [&]() {
        return ((int64_t)it.b * a.n_q + query()) * H + (int64_t)it.g * a.R + row % a.R;
      };
      // key (dk, dv) or query position
      auto position = [&]() { return it.dkv ? it.k0 + row : it.w.q_pos0 + query(); };
      float nl = 0.f, nd = 0.f;
      const int32_t nt = it.nt;
      if (!it.dkv && nt > 0) {                // (padding rows: -inf, 0)
        ok = W(XB_META_FULL + (int)(nm % kWbMeta), nm / kWbMeta);
        const float* m =
            reinterpret_cast<const float*>(base + kWbOffMeta + (int)(nm % kWbMeta) * 1024);
        nl = m[row];
        nd = m[128 + row];
        arrive(XB_META_EMPTY + (int)(nm % kWbMeta));
        ++nm;
      }
      const int32_t win = a.window > 0 ? (int32_t)min64(a.window, int64_t(1) << 30) : 1 << 30;
      const int32_t sink = (int32_t)a.sink;
      // one step; kDkv: lse and D come with the columns, P goes to the tensor core too; kHalf:
      // the tile may come twice (low: this is the second time); alone: columns or row of a
      // query that sees one key, dS = 0.  Of its 32 columns of the buffer, P takes the first
      // 16, dS the others
      auto tile = [&](auto kind, uint32_t vis, bool low, uint32_t alone) {
        constexpr bool kDkv = decltype(kind)::value, kHalf = kTwice || !kDkv;
        const bool full = __all_sync(0xffffffffu, vis == ~0u);
        const ulonglong2* m = reinterpret_cast<const ulonglong2*>(
            base + kWbOffMeta + (int)(nm % kWbMeta) * 1024 + 4 * c0);
        const uint32_t ts = tmem + lane_base + 128 * (n & 1) + c0;
        if (kDkv && !W(XB_META_FULL + (int)(nm % kWbMeta), nm / kWbMeta)) return false;
        if (!W(XB_S_FULL, n)) return false;
        tc_fence_after();
        uint32_t s[32];
        tmem_ld_32x32b_x32(ts, s);
        tmem_ld_wait();
        tc_fence_before();
        arrive(XB_S_READ);
        const uint64_t nl2 = pack_f32x2(__float_as_uint(nl), __float_as_uint(nl));
#pragma unroll
        for (int q = 0; q < 8; ++q) {         // columns c0 + 4 q .. + 3
          uint64_t l0 = nl2, l1 = nl2;
          if (kDkv) {
            const ulonglong2 v = m[q];
            l0 = v.x;
            l1 = v.y;
          }
          const int c = 4 * q;
          float e[4];
          unpack_f32x2(fma_f32x2(pack_f32x2(s[c], s[c + 1]), scale2, l0), e[0], e[1]);
          unpack_f32x2(fma_f32x2(pack_f32x2(s[c + 2], s[c + 3]), scale2, l1), e[2], e[3]);
#pragma unroll
          for (int i = 0; i < 4; ++i) s[c + i] = __float_as_uint(ex2_approx(e[i]));
        }
        if (!full) {
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (!((vis >> c) & 1)) s[c] = 0u;
        }
        if (!W(XB_DP_FULL, n)) return false;
        tc_fence_after();
        // 16 columns of dP at a time: P takes the place of the first, dS of the second
        uint32_t d[16], pk[16];
        tmem_ld_32x32b_x16(ts, d);
        const uint64_t nd2 = pack_f32x2(__float_as_uint(nd), __float_as_uint(nd));
        tmem_ld_wait();
        if (kHalf) vis &= ~alone;
        if (kDkv) {
#pragma unroll
          for (int q = 0; q < 16; ++q)
            pk[q] = pack_part(u2f(s[2 * q]), u2f(s[2 * q + 1]), kHalf && low);
          tmem_st_32x32b_x16(ts, pk);
        }
        auto make_ds = [&](auto part) {
          constexpr bool kPart = kHalf && decltype(part)::value;
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            if (cc == 1) {
              tmem_ld_32x32b_x16(ts + 16, d);
              tmem_ld_wait();
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint64_t d0 = nd2, d1 = nd2;
              if (kDkv) {
                const ulonglong2 v = m[32 + 4 * cc + q];
                d0 = v.x;
                d1 = v.y;
              }
              const int c = 16 * cc + 4 * q;
              float e[4];
              unpack_f32x2(mul_f32x2(pack_f32x2(s[c], s[c + 1]),
                                     add_f32x2(pack_f32x2(d[4 * q], d[4 * q + 1]), d0)),
                           e[0], e[1]);
              unpack_f32x2(mul_f32x2(pack_f32x2(s[c + 2], s[c + 3]),
                                     add_f32x2(pack_f32x2(d[4 * q + 2], d[4 * q + 3]), d1)),
                           e[2], e[3]);
              if (!full) {                      // dO.v may be anything where nothing is seen
#pragma unroll
                for (int i = 0; i < 4; ++i) e[i] = (vis >> (c + i)) & 1 ? e[i] : 0.f;
              }
              pk[8 * cc + 2 * q] = pack_part(e[0], e[1], kPart && low);
              pk[8 * cc + 2 * q + 1] = pack_part(e[2], e[3], kPart && low);
            }
          }
        };
        // apart: most steps are not second ones and need no choice between the parts (8192
        // tokens, 64 / 8 heads, W = 1024: 957 us, with the choice 970)
        if (kHalf && !low) make_ds(std::false_type{});
        else make_ds(std::true_type{});
        tmem_st_32x32b_x16(ts + 16, pk);
        tmem_st_wait();
        tc_fence_before();
        arrive(XB_DS_FULL + (int)(n & 1));
        if (kDkv) {
          arrive(XB_META_EMPTY + (int)(nm % kWbMeta));
          ++nm;
        }
        ++n;
        return true;
      };
      // visible columns of this thread's 32, as bits.  A query that sees one key -- position 0's,
      // or all -- has dS = 0 exactly (its tile is never full).  In dk, where a sum over many rows
      // takes one such row in, what it leaves, 2^-17 of a term, is masked only where tiles come
      // twice, or below, where nothing else is in the sum
      const bool lone = kTwice && win == 1 && sink == 0;       // all of them
      if (it.dkv) {                           // columns: rows of query tile q_tile + t
        const int32_t pos = position();
        int32_t d = pos - (int32_t)a.q_pos0 - it.q_tile * tpt;   // first query that sees the key
        for (int32_t t = 0; ok && t < nt; ++t) {
          const int32_t e = d + win;                             // first one past the window
          const bool at0 = kTwice && c0 == 0 && a.q_pos0 == 0 && it.q_tile + (t >> 1) == 0;
          const uint32_t alone = lone ? ~0u : at0 ? (1u << a.R) - 1u : 0u;
          ok = tile(std::true_type{},
                    range_bits(d > tpt ? 128 : d * a.R, pos < sink || e > tpt ? 128 : e * a.R, c0),
                    kTwice && (t & 1), alone);
          if (!kTwice || (t & 1)) d -= tpt;
        }
      } else {                                // columns: keys
        const int32_t pos = position();
        for (int32_t t = 0; ok && t < nt; ++t) {
          ok = tile(std::false_type{},
                    win_visible(it.w, 4 * (it.w.j0 + tile_of(it, t)) + wg, pos, sink),
                    t & it.half, it.half && (lone || pos == 0) ? ~0u : 0u);
        }
      }
      if (!ok) break;
      // outputs: dk, dv items: warps 0-7 dV, 8-15 dK, 64 columns each; dq: 32 columns each
      const bool any = nt > 0;
      if (any) {
        if (!W(XB_ACC_FULL, ni)) { ok = false; break; }
        tc_fence_after();
      }
      const int ncol = it.dkv ? 4 : 2;        // groups of 16 columns
      const int which = wg >> 1, oc = it.dkv ? 64 * (wg & 1) : c0;
      const uint32_t src = tmem + lane_base + (it.dkv ? 256 + 128 * which : 384) + oc;
      const float f = it.dkv && which == 0 ? 1.f : a.scale;
      const int32_t pos = position();
      const bool store = it.dkv ? pos < a.n_kv : query() < a.n_q;
      const bool live = any && store && pos < it.len &&
                        !(it.dkv && which == 1 && it.len == 1 && a.q_pos0 == 0);
      const bool part = it.part >= 0;
      uint8_t* dst;
      if (part)
        dst = reinterpret_cast<uint8_t*>(
            it.dkv ? p.part + (((int64_t)it.part * 2 + which) * 128 + row) * kHeadDim + oc
                   : p.part_q + ((int64_t)it.part * 128 + row) * kHeadDim + oc);
      else if (it.dkv)
        dst = reinterpret_cast<uint8_t*>(
            (which == 0 ? a.dv : a.dk) +
            (((int64_t)it.b * a.G + it.g) * a.n_kv + pos) * kHeadDim + oc);
      else
        dst = reinterpret_cast<uint8_t*>(a.dq + qrow() * kHeadDim + oc);
#pragma unroll 1
      for (int cc = 0; cc < ncol; ++cc) {
        uint32_t r[16];
        if (any) {
          tmem_ld_32x32b_x16(src + 16 * cc, r);
          tmem_ld_wait();
        }
#pragma unroll
        for (int q = 0; q < 16; ++q) r[q] = live ? __float_as_uint(f * u2f(r[q])) : 0u;
        float* o = reinterpret_cast<float*>(dst + cc * (part ? 64 : 32));
        if (part) {
#pragma unroll
          for (int q = 0; q < 2; ++q)
            st_global_v8(o + 8 * q, u2f(r[8 * q]), u2f(r[8 * q + 1]), u2f(r[8 * q + 2]),
                         u2f(r[8 * q + 3]), u2f(r[8 * q + 4]), u2f(r[8 * q + 5]),
                         u2f(r[8 * q + 6]), u2f(r[8 * q + 7]));
        } else if (store) {
#pragma unroll
          for (int q = 0; q < 8; ++q) r[q] = pack_bf16x2(u2f(r[2 * q]), u2f(r[2 * q + 1]));
          st_global_v8(o, u2f(r[0]), u2f(r[1]), u2f(r[2]), u2f(r[3]), u2f(r[4]), u2f(r[5]),
                       u2f(r[6]), u2f(r[7]));
        }
      }
      if (any) {
        tc_fence_before();
        arrive(XB_ACC_EMPTY);
        ++ni;
      }
      done_item(k);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kWbCtl + 1) tmem_dealloc(tmem, 512);
}

// dv, dk of the cut blocks: their chunks' sums added in chunk order, 4 values a
// thread.  blockIdx.x: (batch, group, key block of the cut ones' range).
__global__ void __launch_bounds__(256)
    window_bwd_join_kernel(const __grid_constant__ WindowBwdArgs p, int32_t c_lo, int32_t n_c) {
  grid_wait();
  const WindowArgs& a = p.w;
  const int32_t bg = blockIdx.x / n_c, c = c_lo + blockIdx.x - bg * n_c;
  int32_t first, count;
  wb_query_tiles(a, c, first, count);
  const int32_t k = wb_chunks(count, p.chunk);
  if (k == 1) return;
  const int i = blockIdx.y * 256 + threadIdx.x;             // of 2 x 128 x 32 float4
  const float4* src = reinterpret_cast<const float4*>(p.part) +
                      ((int64_t)bg * p.n_part + p.pbase[c]) * 8192 + i;
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int32_t j = 0; j < k; ++j) {
    const float4 u = src[(int64_t)j * 8192];
    t.x += u.x;
    t.y += u.y;
    t.z += u.z;
    t.w += u.w;
  }
  const int64_t key = (int64_t)c * 128 + ((i >> 5) & 127);
  if (key >= a.n_kv) return;
  __nv_bfloat16* dst =
      (i >= 4096 ? a.dk : a.dv) + ((int64_t)bg * a.n_kv + key) * kHeadDim + 4 * (i & 31);
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(t.x, t.y), pack_bf16x2(t.z, t.w));
}

// dq of row tiles whose keys were shared: the shares' sums in their order, 4 values a thread.
// Row tiles count down from the last queries, as items do.
__global__ void __launch_bounds__(256)
    window_bwd_join_dq_kernel(const __grid_constant__ WindowBwdArgs p) {
  grid_wait();
  const WindowArgs& a = p.w;
  const int32_t tile = blockIdx.x, i = blockIdx.y * 256 + threadIdx.x;   // of 128 x 32 float4
  const int32_t n_bg = (int32_t)a.batch * a.G, tpt = 128 / a.R;
  const int32_t n_it = ((int32_t)a.n_q + tpt - 1) / tpt, r = tile / n_bg, bg = tile - r * n_bg;
  const float4* src = reinterpret_cast<const float4*>(p.part_q) + (int64_t)tile * p.kq * 4096 + i;
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int32_t j = 0; j < p.kq; ++j) {
    const float4 u = src[(int64_t)j * 4096];
    t.x += u.x;
    t.y += u.y;
    t.z += u.z;
    t.w += u.w;
  }
  const int32_t row = i >> 5, b = bg / a.G, g = bg - b * a.G;
  const int64_t q = (int64_t)(n_it - 1 - r) * tpt + row / a.R;
  if (q >= a.n_q) return;
  __nv_bfloat16* dst = a.dq + (((int64_t)b * a.n_q + q) * a.G * a.R + (int64_t)g * a.R + row % a.R) *
                                  kHeadDim + 4 * (i & 31);
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(t.x, t.y), pack_bf16x2(t.z, t.w));
}

size_t window_attn_bwd_workspace(const WindowArgs& a) {
  const WbPlan p = wb_plan(a);
  if (p.n_dkv + p.n_dq * p.kq > 0x7FFFFF00 || a.batch * a.n_q * a.G * a.R > 0x7FFFFF00) return 0;
  return pad32((size_t)a.batch * a.n_q * a.G * a.R * 4) + pad32((size_t)p.n_cut * 8) +
         pad32((size_t)p.nblk * 4) + 32 +
         ((size_t)a.batch * a.G * p.n_part * 2 + (p.kq > 1 ? p.n_dq * p.kq : 0)) * 128 * 128 *
             sizeof(float);
}

cudaError_t launch_window_attn_bwd(const CUtensorMap& tm_q, const CUtensorMap& tm_do,
                                   const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                                   const CUtensorMap& tm_k32, const CUtensorMap& tm_v32,
                                   WindowArgs a, void* ws, cudaStream_t st) {
  const WbPlan pl = wb_plan(a);
  auto kernel = pl.twice ? window_attn_bwd_kernel<true> : window_attn_bwd_kernel<false>;
  static KernelSetup setup[2];
  int sms = 0;
  cudaError_t e = kernel_setup(setup[pl.twice], reinterpret_cast<const void*>(kernel), kWbSmemBytes,
                               kWbRegsAtLaunch, &sms);
  if (e != cudaSuccess) return e;
  WindowBwdArgs p;
  p.w = a;
  uint8_t* w = static_cast<uint8_t*>(ws);
  float* delta = reinterpret_cast<float*>(w);
  w += pad32((size_t)a.batch * a.n_q * a.G * a.R * 4);
  int2* table = reinterpret_cast<int2*>(w);
  w += pad32((size_t)pl.n_cut * 8);
  int32_t* pbase = reinterpret_cast<int32_t*>(w);
  w += pad32((size_t)pl.nblk * 4);
  p.counter = reinterpret_cast<int32_t*>(w);
  p.part = reinterpret_cast<float*>(w + 32);
  p.delta = delta;
  p.table = table;
  p.pbase = pbase;
  p.chunk = pl.chunk;
  p.nblk = (int32_t)pl.nblk;
  p.n_cut = (int32_t)pl.n_cut;
  p.n_part = (int32_t)pl.n_part;
  p.n_dkv = (int32_t)pl.n_dkv;
  p.n_all = (int32_t)(pl.n_dkv + pl.n_dq * pl.kq);
  p.part_q = p.part + (size_t)a.batch * a.G * pl.n_part * 2 * 128 * 128;
  p.kq = pl.kq;
  const int64_t rows = a.batch * a.n_q * a.G * a.R;
  window_bwd_prep_kernel<<<(unsigned)((rows + kWbPrepRows - 1) / kWbPrepRows + 1), 256, 0, st>>>(
      a, delta, table, pbase, p.counter, pl.chunk, p.nblk);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  e = launch_dependent(kernel, (unsigned)min64(p.n_all, sms), kWbThreads,
                       kWbSmemBytes, st, tm_q, tm_do, tm_k, tm_v, tm_k32, tm_v32, p);
  if (e == cudaSuccess && pl.n_part > 0) {
    const int32_t n_c = (int32_t)(pl.c_hi - pl.c_lo);
    e = launch_dependent(window_bwd_join_kernel, dim3((unsigned)(a.batch * a.G * n_c), 32), 256, 0,
                         st, p, (int32_t)pl.c_lo, n_c);
  }
  if (e == cudaSuccess && pl.kq > 1)
    e = launch_dependent(window_bwd_join_dq_kernel, dim3((unsigned)pl.n_dq, 16), 256, 0, st, p);
  return e;
}

}  // namespace msa
