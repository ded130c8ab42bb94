// Attention with a sliding window and sink tokens (forward).  Query i of batch
// b sits at position t = q_pos0 + i and sees the keys
//   J(t) = {j <= t : t - j < W or j < S}   (W = window, S = sinks; no window: all),
//   o = sum_{j in J} softmax_{j in J}(scale q.k_j) v_j,  lse = ln sum e^{scale q.k_j}.
// Rows at t >= kv_len[b] are padding: o = 0, lse = -inf.
//
// Bound: the tensor cores (4 * 128 flops per visible pair and head; K and V are
// shared by the R heads of a group and come from L2) together with the
// exponentials: a 128 x 128 tile costs 1024 clocks of MMA and 1024 of ex2.
// Design: persistent, one CTA per SM, warp-specialised:
//   warps 0-3, 4-7  softmax halves A and B: thread = row; S from TMEM into
//                   registers, one running (m, l) per row, P = bf16(2^{s - m}) into
//                   TMEM, the A operand of O += P V
//   warp 8          TMA: the item's Q tiles, then K and V tiles through a ring
//   warp 9          issues S = Q K^T;  warp 10  issues O += P V
//   warp 11         idle (it fills the control warpgroup)
// A row tile is 128 / R tokens x the R heads of a group, so that a short window
// is covered by few key tiles (W + 128 / R keys instead of W + 128) and the
// heads share K and V.  An item is two adjacent row tiles, one per half -- or,
// when that would leave SMs without work, one row tile whose key tiles the halves
// take in turn, each with its own (m, l, O), joined at the end.  Key tiles start
// at the first key the item's window reaches (TMA rows need no alignment).
// Few row tiles of many keys: a cluster of up to 8 CTAs takes one row tile, each a run of
// its key tiles; their (m, l, O) meet through distributed shared memory, every CTA joining
// and storing a slice of the rows (16 queries over 32768 keys, 16 / 2 heads: 45 us, one CTA
// a tile 227).
// TMEM: one S buffer (128 columns) that the halves use in turn, P_A, P_B (64 each),
// O_A, O_B (128 each).  S is free again as soon as it is in registers, so neither
// half waits for a product of its own: the next S is made while a half is at its
// exponentials.  (With P in S's columns, S(j + 1) had to wait for P V(j): 2800
// clocks a tile; with one warp issuing both products, 2300: the issue of eight MMAs
// takes as long as they do, and the waits between came on top.)
// The running maximum is kept until a row exceeds it by 2^8: then O is
// rescaled by the softmax warps themselves, after P V of the tile before.
// Exact: P and l use the same maximum.
// P is rounded to bf16 (at most 2^-8 of a weight) for the product; l sums fp32.
// Rows leave 32 columns at a time straight from TMEM: the lanes' rows are whole
// 64-byte runs.
// Measured: 32768 tokens, 32 / 8 heads, W = 4096, S = 64 (2.09 TFLOP): 1600 us, 1.31
// PFLOP/s (0.80 of the burst rate; long runs meet the power cap: 1900 us).  8192
// tokens, 64 / 8 heads, W = 1024: 310 us.  4096 tokens, 4 / 1 heads, W = 512: 16 us,
// 12 of them on the SM: 3 until the first tile is there, 2 x 3 tiles a half.
#include <type_traits>

#include "common.cuh"
#include "layer_args.cuh"
#include "window_tiles.cuh"

namespace msa {

namespace {
constexpr int kWaThreads = 384;
// registers per thread: 168 at launch (65536 / 384 rounded down to the allocation
// unit; the launcher checks the compiled count); the control warpgroup gives
// some to the two softmax warpgroups, whose S row alone takes 128
constexpr int kWaRegsAtLaunch = 168, kWaRegsControl = 72, kWaRegsSoftmax = 216;
static_assert(kWaRegsControl + 2 * kWaRegsSoftmax == 3 * kWaRegsAtLaunch,
              "warpgroup register shares must add up to the launch allocation");
constexpr int kWaRing = 5;                              // 32 KB K or V tiles in flight
constexpr int kWaOffQ = 0;                              // Q_A, Q_B
constexpr int kWaOffRing = 65536;
constexpr int kWaOffML = 32768;      // m, l of both halves' rows when they share a tile (no Q_B then)
constexpr int kWaOffBar = kWaOffRing + kWaRing * 32768;
enum {
  WB_Q_FULL = 0, WB_Q_EMPTY = 2, WB_S_FULL = 4, WB_P_FULL = 6, WB_PV_DONE = 8, WB_O_EMPTY = 10,
  WB_S_READ = 12, WB_JOIN, WB_KV_FULL = WB_JOIN + 2, WB_KV_EMPTY = WB_KV_FULL + kWaRing,
  WB_DRAIN = WB_KV_EMPTY + kWaRing, WB_ITEM_FULL = WB_DRAIN + 2, WB_ITEM_EMPTY = WB_ITEM_FULL + 2,
  WB_COUNT = WB_ITEM_EMPTY + 2
};
constexpr int kWaOffMisc = kWaOffBar + WB_COUNT * 8;
constexpr int kWaOffItem = kWaOffMisc + 16;              // two slots
constexpr int kWaSmemBytes = 1024 + kWaOffItem + 2 * (int)sizeof(WinItem);
constexpr int kWaMaxCluster = 8;                        // the portable limit
constexpr int kWaItemReaders = 10;                      // warps 0-7, 9, 10
static_assert(kWaSmemBytes <= 232448, "shared memory per block");
// the 8 bits of x behind its bf16 rounding b (as fp32 bits): a signed count of 2^8
// fp32 units from b; of two values, above the low half of c
__device__ __forceinline__ uint32_t rest_pair(float x0, float x1, uint32_t pk, uint32_t c) {
  const int32_t d0 = (int32_t)(__float_as_uint(x0) - (pk << 16) + 128u) >> 8;
  const int32_t d1 = (int32_t)(__float_as_uint(x1) - (pk & 0xFFFF0000u) + 128u) >> 8;
  uint32_t r;
  asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(d1), "r"(d0), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t f2u(float x) { return __float_as_uint(x); }
__device__ __forceinline__ void st_words_v8(void* p, const uint32_t* w) {
  st_global_v8(static_cast<float*>(p), u2f(w[0]), u2f(w[1]), u2f(w[2]), u2f(w[3]), u2f(w[4]),
               u2f(w[5]), u2f(w[6]), u2f(w[7]));
}
// O of a CTA's share for the join: rows of 132 floats, so that the 16-byte stores of 8
// lanes meet no bank twice
constexpr int kWaJoinRow = 132;
static_assert(128 * kWaJoinRow * 4 <= kWaRing * 32768, "the join's rows lie in the ring");
__device__ __forceinline__ uint32_t peer_smem(const void* p, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_peer_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_peer_f2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
               : "=f"(v.x), "=f"(v.y)
               : "r"(a)
               : "memory");
  return v;
}
// all threads of all CTAs of the cluster; every path of the kernel comes here
__device__ __forceinline__ void cluster_sync() {
  asm volatile(
      "barrier.cluster.arrive.release;\n\t"
      "barrier.cluster.wait.acquire;" ::: "memory");
}
constexpr float kLazyLog2 = 8.f;     // rescale O when a row's maximum grows by more than 2^8
}  // namespace

// kCluster: launched in clusters of n_share CTAs (else n_share is 1)
template <bool kCluster>
__global__ void __launch_bounds__(kWaThreads, 1)
    window_attn_fwd_kernel(const __grid_constant__ CUtensorMap tm_q,
                           const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v,
                           const __grid_constant__ CUtensorMap tm_k32,
                           const __grid_constant__ CUtensorMap tm_v32,
                           const __grid_constant__ WindowArgs a, int32_t tiles_per_item,
                           int32_t n_items, int32_t n_share) {
  const int32_t cluster = kCluster ? n_share : 1;
  extern __shared__ uint8_t smem_raw[];
  // (an offset, so that the compiler still knows the address space)
  uint8_t* base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bar = reinterpret_cast<uint64_t*>(base + kWaOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + kWaOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base + kWaOffMisc + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int32_t* err = a.err;
  const bool split = tiles_per_item == 1;              // the halves share one row tile

  WinItem it0{};                             // the first item, decoded while the barriers are made
  if (warp == 8) {
    if (lane == 0) {
      prefetch_tensormap(&tm_q);
      prefetch_tensormap(&tm_k);
      prefetch_tensormap(&tm_v);
    }
    win_item(it0, a, (int32_t)(blockIdx.x / (uint32_t)cluster), tiles_per_item);
    if (kCluster) {                       // this CTA's run of the key tiles
      const int32_t r = (int32_t)(blockIdx.x % (uint32_t)cluster), nt = it0.nt;
      it0.j0 = nt * r / cluster;
      it0.nt = nt * (r + 1) / cluster - it0.j0;
    }
  }
  if (tid == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar + WB_Q_FULL + x, 1);
      mbar_init(bar + WB_Q_EMPTY + x, 1);
      mbar_init(bar + WB_S_FULL + x, 1);
      mbar_init(bar + WB_P_FULL + x, 4);           // a lane of each warp
      mbar_init(bar + WB_PV_DONE + x, 1);
      mbar_init(bar + WB_O_EMPTY + x, split ? 8 : 4);
      mbar_init(bar + WB_JOIN + x, 4);
    }
    for (int s = 0; s < kWaRing; ++s) {
      mbar_init(bar + WB_KV_FULL + s, 1);
      mbar_init(bar + WB_KV_EMPTY + s, 1);
    }
    mbar_init(bar + WB_S_READ, 4);
    mbar_init(bar + WB_DRAIN, 1);
    mbar_init(bar + WB_DRAIN + 1, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar + WB_ITEM_FULL + s, 1);
      mbar_init(bar + WB_ITEM_EMPTY + s, kWaItemReaders);
    }
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  constexpr uint32_t kColP = 128, kColO = 256;         // S at 0; P_A, P_B; O_A, O_B
  // k-th completion of a barrier has parity k & 1; the whole warp decides together
  auto W = [&](int id, uint32_t k) {
    return __all_sync(0xffffffffu, mbar_wait(bar + id, k & 1u, abort_flag, err));
  };
  auto arrive = [&](int id) {                          // for the whole warp
    __syncwarp();
    if (lane == 0) mbar_arrive(bar + id);
  };
  // Items are decoded once, by the TMA warp, and kept in shared memory: the softmax
  // warps need their registers.  `cur`: the role's item
  auto item_slot = [&](uint32_t k) {
    return reinterpret_cast<WinItem*>(base + kWaOffItem) + (k & 1);
  };
  const WinItem* cur = item_slot(0);
  auto next_item = [&](uint32_t k) {
    if (!W(WB_ITEM_FULL + (int)(k & 1), k >> 1)) return false;
    cur = item_slot(k);
    return cur->nt >= 0;                               // -1: there are no more
  };
  auto done_item = [&](uint32_t k) { arrive(WB_ITEM_EMPTY + (int)(k & 1)); };
  // step i of an item is key tile tile_of(i) of half i & 1; does the half need it?
  auto n_steps = [&]() { return split ? cur->nt : 2 * cur->nt; };
  auto tile_of = [&](int i) { return split ? i : i >> 1; };
  auto takes = [&](int i) {
    if (split) return i < cur->nt;
    const int j = i >> 1;
    return (i & 1) ? cur->rows[1] && j < cur->nt && (4 * j < cur->nc || j >= cur->beg_b)
                   : j <= cur->end_a;
  };
  // ring slots of an item's tiles, in the order K0 K1 V0 K2 V1 ... (counted from its first)
  auto slot_k = [&](int j) { return (uint32_t)(j == 0 ? 0 : 2 * j - 1); };
  auto slot_v = [&](int j) { return (uint32_t)(j == cur->nt - 1 ? 2 * j + 1 : 2 * j + 2); };

  if (warp >= 8) {
    setmaxnreg_dec<kWaRegsControl>();
  if (warp == 8) {
    // ---------------- TMA ----------------
    uint32_t nq[2] = {0, 0}, n = 0;          // Q loads per tile, ring slots
    WinItem it = it0;
    bool ok = true;
    auto push = [&](const CUtensorMap* tm, const CUtensorMap* tm32, int j) {
      const uint32_t s = n % kWaRing;
      if (n >= kWaRing && !W(WB_KV_EMPTY + s, n / kWaRing - 1)) return false;
      if (lane == 0) {
        uint8_t* dst = base + kWaOffRing + s * 32768;
        mbar_arrive_expect_tx(bar + WB_KV_FULL + s, 32768u);
        win_load_keys(dst, tm, tm32, bar + WB_KV_FULL + s, it, it.j0 + j);
      }
      ++n;
      return true;
    };
    for (uint32_t k = 0; ok; ++k) {
      // largest first, the rounds in alternating directions: evens out the CTAs' sums
      const uint32_t at = (k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x;
      const int64_t i = (int64_t)k * gridDim.x + at;
      if (k >= 2 && !W(WB_ITEM_EMPTY + (int)(k & 1), (k >> 1) - 1)) break;
      const bool end = kCluster ? k > 0 : i >= n_items;
      if (k > 0 && !end) win_item(it, a, (int32_t)i, tiles_per_item);
      if (lane == 0) {
        *item_slot(k) = it;
        if (end) item_slot(k)->nt = -1;
        mbar_arrive(bar + WB_ITEM_FULL + (int)(k & 1));
      }
      __syncwarp();
      if (end) break;
      for (int x = 0; ok && x < 2; ++x) {
        if (!it.rows[x]) continue;
        ok = nq[x] == 0 || W(WB_Q_EMPTY + x, nq[x] - 1);
        if (ok && lane == 0) {
          uint8_t* dst = base + kWaOffQ + x * 32768;
          const int32_t tok = it.i0 + x * (128 / a.R);
          mbar_arrive_expect_tx(bar + WB_Q_FULL + x, 32768u);
          tma_load_4d(dst, &tm_q, bar + WB_Q_FULL + x, 0, it.g * a.R, tok, it.b);
          tma_load_4d(dst + 16384, &tm_q, bar + WB_Q_FULL + x, 64, it.g * a.R, tok, it.b);
        }
        if (ok) ++nq[x];
      }
      if (ok && it.nt > 0) ok = push(&tm_k, &tm_k32, 0);
      for (int j = 0; ok && j < it.nt; ++j)
        ok = (j + 1 == it.nt || push(&tm_k, &tm_k32, j + 1)) && push(&tm_v, &tm_v32, j);
    }
    // no copy may still be writing shared memory when the block exits
    if (lane == 0) {
      for (uint32_t k = n > kWaRing ? n - kWaRing : 0; k < n; ++k)
        mbar_drain(bar + WB_KV_FULL + k % kWaRing, (k / kWaRing) & 1u, err);
      for (int x = 0; x < 2; ++x)
        if (nq[x] > 0) mbar_drain(bar + WB_Q_FULL + x, (nq[x] - 1) & 1u, err);
    }
  } else if (warp == 9) {
    // ---------------- S = Q K^T ----------------
    constexpr uint32_t kIdS = idesc_bf16_f32(128, 128, 0);
    const uint32_t ring = smem_u32(base + kWaOffRing), qs = smem_u32(base + kWaOffQ);
    uint32_t nq[2] = {0, 0}, ns = 0, n0 = 0;     // Q tiles used, S products, ring slots
    bool ok = true;
    for (uint32_t ki = 0; ok && next_item(ki); ++ki) {
      bool seen_q[2] = {false, false};
      const int n_st = n_steps();
      int left = 0;                          // products still to come
      for (int k = 0; k < n_st; ++k) left += takes(k) ? 1 : 0;
      // step k (of half x), once the buffer's last S is in registers
      auto issue = [&](auto half, int k) {
        constexpr int x = decltype(half)::value;
        if (!ok || k >= n_st || !takes(k)) return;
        const uint32_t sk = n0 + slot_k(tile_of(k)), slot = sk % kWaRing;
        if (split || x == 0 || !takes(k - 1))
          if (!W(WB_KV_FULL + slot, sk / kWaRing)) { ok = false; return; }
        if (!seen_q[x] && (!split || x == 0) && !W(WB_Q_FULL + x, nq[x])) { ok = false; return; }
        seen_q[x] = true;
        if (ns > 0 && !W(WB_S_READ, ns - 1)) { ok = false; return; }
        ++ns;
        --left;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t qd = smem_desc_sw128(qs + (split ? 0 : x) * 32768, 16, 1024);
          const uint64_t kd = smem_desc_sw128(ring + slot * 32768, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {      // the start address counts 16-byte units
            const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) / 16;
            umma_bf16(tmem, qd + off, kd + off, kIdS, kk > 0 ? 1u : 0u);
          }
          umma_commit(bar + WB_S_FULL + x);
          if (split || x == 1 || !takes(k + 1)) umma_commit(bar + WB_KV_EMPTY + slot);
          if (left == 0) {
            umma_commit(bar + WB_Q_EMPTY);
            if (cur->rows[1]) umma_commit(bar + WB_Q_EMPTY + 1);
          }
        }
        __syncwarp();
      };
      for (int k = 0; ok && k < n_st; k += 2) {
        issue(std::integral_constant<int, 0>{}, k);
        issue(std::integral_constant<int, 1>{}, k + 1);
      }
      n0 += 2 * (uint32_t)cur->nt;
      for (int x = 0; x < 2; ++x)
        if (cur->rows[x]) ++nq[x];
      if (ok) done_item(ki);
    }
    // every MMA issued has finished before the tensor memory is freed
    if (elect_one()) {
      umma_commit(bar + WB_DRAIN);
      mbar_drain(bar + WB_DRAIN, 0, err);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ---------------- O += P V ----------------
    constexpr uint32_t kIdO = idesc_bf16_f32(128, 128, 1);
    uint32_t np[2] = {0, 0}, no[2] = {0, 0}, n0 = 0;     // products, items with an O, ring slots
    bool ok = true;
    for (uint32_t ki = 0; ok && next_item(ki); ++ki) {
      bool begun[2] = {false, false};
      const int n_st = n_steps();
      auto issue = [&](auto half, int k) {
        constexpr int x = decltype(half)::value;
        if (!ok || k >= n_st || !takes(k)) return;
        const int j = tile_of(k);
        const uint32_t sv = n0 + slot_v(j), slot = sv % kWaRing;
        uint8_t* tile = base + kWaOffRing + slot * 32768;
        if (split || x == 0 || !takes(k - 1)) {          // the tile's first use
          if (!W(WB_KV_FULL + slot, sv / kWaRing)) { ok = false; return; }
          // keys past the sequence's end, or behind the last query, may hold anything: their V
          // rows are cleared (P is 0 there, and 0 * NaN would not be)
          if (cur->len < a.n_kv)
            win_clear_keys(tile, *cur, cur->j0 + j, lane);
        }
        if (!begun[x] && no[x] > 0 && !W(WB_O_EMPTY + x, no[x] - 1)) { ok = false; return; }
        if (!W(WB_P_FULL + x, np[x])) { ok = false; return; }
        ++np[x];
        tc_fence_after();
        if (elect_one()) {
          const uint64_t vd = smem_desc_sw128(smem_u32(tile), 16384, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_bf16_ts(tmem + kColO + 128 * x, tmem + kColP + 64 * x + kk * 8,
                         vd + kk * (2048 / 16), kIdO, begun[x] || kk > 0 ? 1u : 0u);
          umma_commit(bar + WB_PV_DONE + x);
          if (split || x == 1 || !takes(k + 1)) umma_commit(bar + WB_KV_EMPTY + slot);
        }
        __syncwarp();
        begun[x] = true;
      };
      for (int k = 0; ok && k < n_st; k += 2) {
        issue(std::integral_constant<int, 0>{}, k);
        issue(std::integral_constant<int, 1>{}, k + 1);
      }
      n0 += 2 * (uint32_t)cur->nt;
      for (int x = 0; x < 2; ++x)
        if (begun[x]) ++no[x];
      if (ok) done_item(ki);
    }
    if (elect_one()) {
      umma_commit(bar + WB_DRAIN + 1);
      mbar_drain(bar + WB_DRAIN + 1, 0, err);
    }
    __syncwarp();
  }
  } else {
    setmaxnreg_inc<kWaRegsSoftmax>();
    // ---------------- softmax of half x; thread = row ----------------
    const int x = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t tp = lanes + kColP + 64 * x, to = lanes + kColO + 128 * x;
    const float scale_log2 = a.scale * 1.4426950408889634f;
    const uint64_t scale2 = pack_f32x2(__float_as_uint(scale_log2), __float_as_uint(scale_log2));
    const int32_t tpt = 128 / a.R;            // tokens per row tile
    const int32_t sink = (int32_t)a.sink;
    float2* ml = reinterpret_cast<float2*>(base + kWaOffML);   // [half][row]
    uint32_t ns = 0, np = 0, np_other = 0, nj = 0;
    bool ok = true;
    for (uint32_t ki = 0; ok && next_item(ki); ++ki) {
      const WinItem& it = *cur;
      const int32_t first = it.i0 + (split ? 0 : x * tpt);       // the row tile's first query
      const int32_t i_row = first + row / a.R;
      const int32_t t = it.q_pos0 + i_row;
      const int32_t t_min = it.q_pos0 + first + (quarter * 32) / a.R, t_max = t_min + (31 / a.R);
      float m = -INFINITY, l = 0.f;
      bool begun = false;
      const int n_st = n_steps();
      for (int k = x; k < n_st; k += 2) {
        if (!takes(k)) continue;
        const int j = it.j0 + tile_of(k);
        if (!W(WB_S_FULL + x, ns)) { ok = false; break; }
        ++ns;
        tc_fence_after();
        uint32_t s[128];
#pragma unroll
        for (int cc = 0; cc < 4; ++cc)
          tmem_ld_32x32b_x32(lanes + 32 * cc, *reinterpret_cast<uint32_t(*)[32]>(s + 32 * cc));
        tmem_ld_wait();
        tc_fence_before();
        arrive(WB_S_READ);
        // is every column visible to every row of the warp?
        const int32_t k0 = win_chunk(it, 4 * j);
        const bool full = !win_mixed(it, j) &&
                          (4 * j < it.nc ? k0 + 128 <= it.s_end
                                         : k0 + 127 <= t_min && (t_max - it.W + 1 <= k0 ||
                                                                 sink - k0 >= 128));
        if (!full) {
#pragma unroll
          for (int cc = 0; cc < 4; ++cc) {
            const uint32_t vis = win_visible(it, 4 * j + cc, t, sink);
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!((vis >> c) & 1)) s[32 * cc + c] = 0xFF800000u;   // -inf
          }
        }
        float mq[4];                          // four chains: the latency of one is 64 steps
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          mq[q] = fmaxf(u2f(s[32 * q]), u2f(s[32 * q + 1]));
#pragma unroll
          for (int c = 2; c < 32; c += 2)
            mq[q] = fmax3f(mq[q], u2f(s[32 * q + c]), u2f(s[32 * q + c + 1]));
        }
        const float mx = fmaxf(fmax3f(mq[0], mq[1], mq[2]), mq[3]) * scale_log2;
        const bool grow = mx > m + kLazyLog2 || (m == -INFINITY && mx > -INFINITY);
        // P V of this half's tile before: P and O are free
        if (begun && !W(WB_PV_DONE + x, np - 1)) { ok = false; break; }
        if (__any_sync(0xffffffffu, grow)) {
          const float mn = grow ? mx : m;
          const float f = m == -INFINITY ? 0.f : ex2_approx(m - mn);
          l *= f;
          m = mn;
          if (begun) {
            tc_fence_after();
            const uint64_t f2 = pack_f32x2(__float_as_uint(f), __float_as_uint(f));
#pragma unroll 1
            for (int cc = 0; cc < 8; ++cc) {
              uint32_t r[16];
              tmem_ld_32x32b_x16(to + 16 * cc, r);
              tmem_ld_wait();
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                float u, v;
                unpack_f32x2(mul_f32x2(pack_f32x2(r[2 * q], r[2 * q + 1]), f2), u, v);
                r[2 * q] = __float_as_uint(u);
                r[2 * q + 1] = __float_as_uint(v);
              }
              tmem_st_32x32b_x16(to + 16 * cc, r);
            }
          }
        }
        const float nm = m == -INFINITY ? 0.f : -m;
        const uint64_t nm2 = pack_f32x2(__float_as_uint(nm), __float_as_uint(nm));
        uint64_t l2[2] = {0ull, 0ull};
#pragma unroll
        for (int cc = 0; cc < 4; ++cc) {
          uint32_t pk[16];
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            const int c = 32 * cc + 2 * q;
            float u, v;
            unpack_f32x2(fma_f32x2(pack_f32x2(s[c], s[c + 1]), scale2, nm2), u, v);
            u = ex2_approx(u);
            v = ex2_approx(v);
            l2[q & 1] = add_f32x2(l2[q & 1], pack_f32x2(__float_as_uint(u), __float_as_uint(v)));
            pk[q] = pack_bf16x2(u, v);
          }
          tmem_st_32x32b_x16(tp + 16 * cc, pk);
        }
        float u, v;
        unpack_f32x2(add_f32x2(l2[0], l2[1]), u, v);
        l += u + v;
        tmem_st_wait();
        tc_fence_before();
        arrive(WB_P_FULL + x);
        begun = true;
        ++np;
      }
      if (!ok) break;
      if (begun) {
        if (!W(WB_PV_DONE + x, np - 1)) { ok = false; break; }
        tc_fence_after();
      }
      // shared row tile: the halves exchange (m, l); each stores half of the columns
      float fa = 1.f, fb = 0.f;
      if (split) {
        ml[128 * x + row] = make_float2(m, l);
        arrive(WB_JOIN + x);
        if (!W(WB_JOIN + (x ^ 1), nj)) { ok = false; break; }
        ++nj;
        const int n_other = (it.nt + x) >> 1;              // its products: every second tile
        np_other += n_other;
        if (n_other > 0 && !W(WB_PV_DONE + (x ^ 1), np_other - 1)) { ok = false; break; }
        tc_fence_after();
        const float2 ma = ml[row], mb = ml[128 + row];
        m = fmaxf(ma.x, mb.x);
        const float z = m == -INFINITY ? 0.f : m;
        fa = ex2_approx(ma.x - z);
        fb = ex2_approx(mb.x - z);
        l = ma.y * fa + mb.y * fb;
      }
      const bool has = split ? it.nt > 0 : begun, both = split && it.nt > 1;
      if (kCluster) {                     // to shared memory, for the join below
        float* orow = reinterpret_cast<float*>(base + kWaOffRing) + row * kWaJoinRow;
        if (x == 0) ml[256 + row] = make_float2(m, l);
#pragma unroll 1
        for (int cc = 4 * x; cc < 4 * x + 4; ++cc) {
          uint32_t r[16], rb[16];
          if (has) tmem_ld_32x32b_x16(lanes + kColO + 16 * cc, r);
          if (both) tmem_ld_32x32b_x16(lanes + kColO + 128 + 16 * cc, rb);
          tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            float u = has ? u2f(r[q]) * fa : 0.f;
            if (both) u += u2f(rb[q]) * fb;
            r[q] = f2u(u);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4*>(orow + 16 * cc + 4 * q) =
                make_uint4(r[4 * q], r[4 * q + 1], r[4 * q + 2], r[4 * q + 3]);
        }
        tc_fence_before();
        done_item(ki);
        continue;
      }
      // the item's rows leave: o = O / l
      const bool store = i_row < a.n_q;
      const bool live = store && t < it.len && has;
      const int64_t orow =
          ((int64_t)it.b * a.n_q + i_row) * ((int64_t)a.G * a.R) + (int64_t)it.g * a.R + row % a.R;
      const float inv = live && l != 0.f ? 1.f / l : 0.f;
      const float f = both ? 1.f : fa * inv;
      fa *= inv;
      fb *= inv;
      if (store && !(split && x == 1))
        a.lse[orow] = live ? m * 0.6931471805599453f + logf(l) : -INFINITY;
      const uint32_t ta = split ? lanes + kColO : to;
      const int c0 = split ? 2 * x : 0, c1 = split ? c0 + 2 : 4;
#pragma unroll 1
      for (int cc = c0; cc < c1; ++cc) {
        uint32_t r[32];
        if (has) tmem_ld_32x32b_x32(ta + 32 * cc, r);
        tmem_ld_wait();
        if (both) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t rb[16];
            tmem_ld_32x32b_x16(ta + 128 + 32 * cc + 16 * h, rb);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 16; ++q)
              r[16 * h + q] = f2u(u2f(r[16 * h + q]) * fa + u2f(rb[q]) * fb);
          }
        }
        if (store) {
          uint32_t pk[16], rest[8];
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            const float u = live ? u2f(r[2 * q]) * f : 0.f, v = live ? u2f(r[2 * q + 1]) * f : 0.f;
            pk[q] = pack_bf16x2(u, v);
            r[2 * q] = f2u(u);
            r[2 * q + 1] = f2u(v);
          }
          st_words_v8(a.out + orow * kHeadDim + 32 * cc, pk);
          st_words_v8(a.out + orow * kHeadDim + 32 * cc + 16, pk + 8);
          if (a.rest != nullptr) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              rest[q] = rest_pair(
                  u2f(r[4 * q]), u2f(r[4 * q + 1]), pk[2 * q],
                  rest_pair(u2f(r[4 * q + 2]), u2f(r[4 * q + 3]), pk[2 * q + 1], 0u));
            uint4* ro = reinterpret_cast<uint4*>(a.rest + orow * kHeadDim + 32 * cc);
            ro[0] = make_uint4(rest[0], rest[1], rest[2], rest[3]);
            ro[1] = make_uint4(rest[4], rest[5], rest[6], rest[7]);
          }
        }
      }
      tc_fence_before();
      if (split) {
        if (has) arrive(WB_O_EMPTY);
        if (both) arrive(WB_O_EMPTY + 1);
      } else if (begun) {
        arrive(WB_O_EMPTY + x);
      }
      done_item(ki);
    }
  }
  if (kCluster) {
    // the shares' (m, l, O) of each row, in the CTAs' order: a slice of the rows per CTA
    cluster_sync();
    if (warp < 8) {
      const WinItem& it = *item_slot(0);
      const uint32_t rank = blockIdx.x % (uint32_t)cluster;
      const int rows = 128 / cluster;
      for (int u = tid; u < rows * 16; u += 256) {
        const int row = (int)rank * rows + (u >> 4), col = 8 * (u & 15);
        const int32_t i_row = it.i0 + row / a.R;
        const float2* mlc = reinterpret_cast<const float2*>(base + kWaOffML) + 256 + row;
        const float* oc =
            reinterpret_cast<const float*>(base + kWaOffRing) + row * kWaJoinRow + col;
        float mx = -INFINITY;
        for (int c = 0; c < cluster; ++c) mx = fmaxf(mx, ld_peer_f2(peer_smem(mlc, c)).x);
        const float z = mx == -INFINITY ? 0.f : mx;
        float l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        for (int c = 0; c < cluster; ++c) {
          const float2 v = ld_peer_f2(peer_smem(mlc, c));
          const uint32_t src = peer_smem(oc, c);
          const float4 p = ld_peer_f4(src), q = ld_peer_f4(src + 16);
          const float f = ex2_approx(v.x - z);
          l += f * v.y;
          o[0] += f * p.x; o[1] += f * p.y; o[2] += f * p.z; o[3] += f * p.w;
          o[4] += f * q.x; o[5] += f * q.y; o[6] += f * q.z; o[7] += f * q.w;
        }
        if (i_row >= a.n_q) continue;
        const bool live = it.q_pos0 + i_row < it.len && l != 0.f;
        const float inv = live ? 1.f / l : 0.f;
        const int64_t orow = ((int64_t)it.b * a.n_q + i_row) * ((int64_t)a.G * a.R) +
                             (int64_t)it.g * a.R + row % a.R;
        uint32_t pk[4];
#pragma unroll
        for (int q = 0; q < 8; ++q) o[q] = live ? o[q] * inv : 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) pk[q] = pack_bf16x2(o[2 * q], o[2 * q + 1]);
        *reinterpret_cast<uint4*>(a.out + orow * kHeadDim + col) =
            make_uint4(pk[0], pk[1], pk[2], pk[3]);
        if (a.rest != nullptr)
          *reinterpret_cast<uint2*>(a.rest + orow * kHeadDim + col) =
              make_uint2(rest_pair(o[0], o[1], pk[0], rest_pair(o[2], o[3], pk[1], 0u)),
                         rest_pair(o[4], o[5], pk[2], rest_pair(o[6], o[7], pk[3], 0u)));
        if (col == 0) a.lse[orow] = live ? mx * 0.6931471805599453f + logf(l) : -INFINITY;
      }
    }
    cluster_sync();                          // nobody's shared memory goes before it was read
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

cudaError_t launch_window_attn_fwd(const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                                   const CUtensorMap& tm_v, const CUtensorMap& tm_k32,
                                   const CUtensorMap& tm_v32, const WindowArgs& a,
                                   cudaStream_t st) {
  static KernelSetup setup[2];
  int sms = 0;
  cudaError_t e =
      kernel_setup(setup[0], reinterpret_cast<const void*>(window_attn_fwd_kernel<false>),
                   kWaSmemBytes, kWaRegsAtLaunch, &sms);
  if (e != cudaSuccess) return e;
  // two row tiles per item share the key tiles' loads (8192 tokens, 64 heads: 274 us, one
  // per item 373); one per item when all of them run at once (1024 tokens, 16 heads: 16.4
  // us, two per item 18.5; twice the tokens: 26.6 and 20.5)
  const int64_t tiles = (a.n_q * a.R + 127) / 128;
  const int32_t per = a.batch * a.G * tiles <= sms ? 1 : 2;
  const int64_t items = a.batch * a.G * ((tiles + per - 1) / per);
  if (items > 0x7FFFFFFF) return cudaErrorInvalidValue;
  // keys of the longest row tile.  The join costs 2 us: two CTAs a tile from 2048 keys on
  // (there 24.6 us either way; 1024 keys: 18.4, alone 16.4), four from 4096 (512 queries, 8 / 1
  // heads: 24.6, alone 36.9), eight from 8192 and only while all clusters run at once:
  // sixteen of eight did not (36.9 us, in fours 22.6)
  int64_t keys = a.q_pos0 + a.n_q;
  if (a.window > 0) keys = min64(keys, min64(a.window, keys) + 128 / a.R + a.sink);
  int cluster = 1;
  while (per == 1 && cluster < kWaMaxCluster && keys >= 2048 * cluster &&
         items * 2 * cluster <= (cluster < 4 ? sms * 7 / 8 : sms / 2))
    cluster *= 2;
  if (cluster == 1) {
    window_attn_fwd_kernel<false><<<(unsigned)min64(items, sms), kWaThreads, kWaSmemBytes, st>>>(
        tm_q, tm_k, tm_v, tm_k32, tm_v32, a, per, (int32_t)items, 1);
    return cudaGetLastError();
  }
  e = kernel_setup(setup[1], reinterpret_cast<const void*>(window_attn_fwd_kernel<true>),
                   kWaSmemBytes, kWaRegsAtLaunch, &sms);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(items * cluster));
  cfg.blockDim = dim3(kWaThreads);
  cfg.dynamicSmemBytes = kWaSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)cluster;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, window_attn_fwd_kernel<true>, tm_q, tm_k, tm_v, tm_k32, tm_v32, a,
                         per, (int32_t)items, (int32_t)cluster);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace msa
