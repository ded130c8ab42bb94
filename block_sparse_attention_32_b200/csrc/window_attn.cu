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
//   warps 0-3, 4-7  softmax of row tile A / B: thread = row; S from TMEM, one
//                   running (m, l) per row, P = bf16(2^{s - m}) back into the
//                   first 64 columns of S, the A operand of O += P V
//   warp 8          TMA: the item's Q tiles, then K and V tiles through a ring
//   warps 10, 11    idle (they fill the control warpgroup)
//   warp 9          MMA: S_X = Q_X K^T, O_X += P_X V for X = A, B in turn, so that
//                   one tile's softmax runs under the other's products
// A row tile is 128 / R tokens x the R heads of a group, so that a short window
// is covered by few key tiles (W + 128 / R keys instead of W + 128) and the
// heads share K and V; an item is two adjacent row tiles.  Key tiles start at
// the first key the item's window reaches (TMA rows need no alignment).
// The running maximum is kept until a row exceeds it by 2^8: then O is
// rescaled by the softmax warps themselves, between S(j) and P(j), while no
// product of that tile is in flight.  Exact: P and l use the same maximum.
// P is rounded to bf16 (2^-9 relative a weight) for the product; l sums fp32.
#include "common.cuh"
#include "layer_args.cuh"
#include "window_tiles.cuh"

namespace msa {

namespace {
constexpr int kWaThreads = 384;
// registers per thread: 168 at launch (65536 / 384 rounded down to the allocation
// unit; the launcher checks the compiled count); the control warpgroup gives
// some to the two softmax warpgroups, whose S row alone takes 128
constexpr int kWaRegsAtLaunch = 168, kWaRegsControl = 104, kWaRegsSoftmax = 200;
static_assert(kWaRegsControl + 2 * kWaRegsSoftmax == 3 * kWaRegsAtLaunch,
              "warpgroup register shares must add up to the launch allocation");
constexpr int kWaRing = 5;                              // 32 KB K or V tiles in flight
constexpr int kWaOffQ = 0;                              // Q_A, Q_B
constexpr int kWaOffRing = 65536;
constexpr int kWaOffBar = kWaOffRing + kWaRing * 32768;
enum {
  WB_Q_FULL = 0, WB_Q_EMPTY = 2, WB_S_FULL = 4, WB_P_FULL = 6, WB_PV_DONE = 8, WB_O_EMPTY = 10,
  WB_KV_FULL = 12, WB_KV_EMPTY = 12 + kWaRing, WB_DRAIN = 12 + 2 * kWaRing, WB_COUNT
};
constexpr int kWaOffMisc = kWaOffBar + WB_COUNT * 8;
constexpr int kWaSmemBytes = 1024 + kWaOffMisc + 16;
static_assert(kWaSmemBytes <= 232448, "shared memory per block");
constexpr float kLazyLog2 = 8.f;     // rescale O when a row's maximum grows by more than 2^8
}  // namespace

__global__ void __launch_bounds__(kWaThreads, 1)
    window_attn_fwd_kernel(const __grid_constant__ CUtensorMap tm_q,
                           const __grid_constant__ CUtensorMap tm_k,
                           const __grid_constant__ CUtensorMap tm_v,
                           const __grid_constant__ WindowArgs a, int32_t tiles_per_item,
                           int64_t n_items) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* bar = reinterpret_cast<uint64_t*>(base + kWaOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(base + kWaOffMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base + kWaOffMisc + 4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int32_t* err = a.err;

  if (tid == 0) {
    for (int x = 0; x < 2; ++x) {
      mbar_init(bar + WB_Q_FULL + x, 1);
      mbar_init(bar + WB_Q_EMPTY + x, 1);
      mbar_init(bar + WB_S_FULL + x, 1);
      mbar_init(bar + WB_P_FULL + x, 128);
      mbar_init(bar + WB_PV_DONE + x, 1);
      mbar_init(bar + WB_O_EMPTY + x, 128);
    }
    for (int s = 0; s < kWaRing; ++s) {
      mbar_init(bar + WB_KV_FULL + s, 1);
      mbar_init(bar + WB_KV_EMPTY + s, 1);
    }
    mbar_init(bar + WB_DRAIN, 1);
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
  const uint32_t tmem = *tmem_slot;          // S_A, S_B, O_A, O_B: 128 columns each
  // k-th completion of a barrier has parity k & 1; the whole warp decides together
  auto W = [&](int id, int64_t k) {
    return __all_sync(0xffffffffu,
                      mbar_wait(bar + id, (uint32_t)(k & 1), abort_flag, err));
  };
  WinItem it{};

  if (warp >= 8) {
    setmaxnreg_dec<kWaRegsControl>();
  if (warp == 8) {
    // ---------------- TMA ----------------
    if (lane == 0) {
      prefetch_tensormap(&tm_q);
      prefetch_tensormap(&tm_k);
      prefetch_tensormap(&tm_v);
    }
    int64_t nq[2] = {0, 0}, n = 0;           // Q loads per tile, ring slots
    bool ok = true;
    auto push = [&](const CUtensorMap* tm, int32_t key0) {
      const int s = (int)(n % kWaRing);
      if (n >= kWaRing && !W(WB_KV_EMPTY + s, n / kWaRing - 1)) return false;
      if (lane == 0) {
        uint8_t* dst = base + kWaOffRing + s * 32768;
        mbar_arrive_expect_tx(bar + WB_KV_FULL + s, 32768u);
        tma_load_4d(dst, tm, bar + WB_KV_FULL + s, 0, key0, it.g, it.b);
        tma_load_4d(dst + 16384, tm, bar + WB_KV_FULL + s, 64, key0, it.g, it.b);
      }
      ++n;
      return true;
    };
    for (int64_t i = blockIdx.x; ok && i < n_items; i += gridDim.x) {
      win_item(it, a, i, tiles_per_item);
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
      for (int j = 0; ok && j < it.nt; ++j)
        ok = push(&tm_k, win_key0(it, j)) && push(&tm_v, win_key0(it, j));
    }
    // no copy may still be writing shared memory when the block exits
    if (lane == 0) {
      for (int64_t k = n > kWaRing ? n - kWaRing : 0; k < n; ++k)
        mbar_drain(bar + WB_KV_FULL + k % kWaRing, (uint32_t)((k / kWaRing) & 1), err);
      for (int x = 0; x < 2; ++x)
        if (nq[x] > 0) mbar_drain(bar + WB_Q_FULL + x, (uint32_t)((nq[x] - 1) & 1), err);
    }
  } else if (warp == 9) {
    // ---------------- MMA ----------------
    constexpr uint32_t kIdS = idesc_bf16_f32(128, 128, 0), kIdO = idesc_bf16_f32(128, 128, 1);
    int64_t nq[2] = {0, 0}, np[2] = {0, 0}, no[2] = {0, 0}, n = 0;
    bool ok = true;
    for (int64_t i = blockIdx.x; ok && i < n_items; i += gridDim.x) {
      win_item(it, a, i, tiles_per_item);
      int last[2], pend[2] = {-1, -1};       // last key tile of X; tile whose P V is due
      bool begun[2] = {false, false};
      for (int x = 0; x < 2; ++x) {
        last[x] = -1;
        for (int j = it.nt - 1; j >= 0 && last[x] < 0; --j)
          if (win_need(it, a, x, j)) last[x] = j;
      }
      const int64_t n0 = n;
      auto slot_k = [&](int j) { return n0 + 2 * j; };
      auto slot_v = [&](int j) { return n0 + 2 * j + 1; };
      // O_X (+)= P_X V(j)
      auto pv = [&](int x, int j) {
        if (!W(WB_P_FULL + x, np[x])) return false;
        if (!begun[x] && no[x] > 0 && !W(WB_O_EMPTY + x, no[x] - 1)) return false;
        const int64_t sv = slot_v(j);
        if (!W(WB_KV_FULL + (int)(sv % kWaRing), sv / kWaRing)) return false;
        const uint32_t va = smem_u32(base + kWaOffRing + (int)(sv % kWaRing) * 32768);
        tc_fence_after();
        if (lane == 0) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_bf16_ts(tmem + 256 + 128 * x, tmem + 128 * x + kk * 8,
                         smem_desc_sw128(va + kk * 2048, 16384, 1024), kIdO,
                         begun[x] || kk > 0 ? 1u : 0u);
          umma_commit(bar + WB_PV_DONE + x);
        }
        __syncwarp();
        begun[x] = true;
        ++np[x];
        return true;
      };
      for (int j = 0; ok && j <= it.nt; ++j) {
        if (j < it.nt) {
          const int64_t sk = slot_k(j);
          ok = W(WB_KV_FULL + (int)(sk % kWaRing), sk / kWaRing);
          if (!ok) break;
          // keys past the sequence's end may hold anything: their V rows are
          // cleared (P is 0 there, and 0 * NaN would not be)
          const int32_t k0 = win_key0(it, j);
          if (it.len < a.n_kv && k0 + 128 > it.len) {
            const int64_t sv = slot_v(j);
            ok = W(WB_KV_FULL + (int)(sv % kWaRing), sv / kWaRing);
            if (!ok) break;
            win_clear_rows(base + kWaOffRing + (int)(sv % kWaRing) * 32768, it.len - k0, lane);
          }
        }
        for (int x = 0; ok && x < 2; ++x) {
          if (pend[x] >= 0) {
            ok = pv(x, pend[x]);
            pend[x] = -1;
          }
          if (!ok || j >= it.nt || !win_need(it, a, x, j)) continue;
          // S_X overwrites the columns P_X was read from
          if (np[x] > 0 && !W(WB_PV_DONE + x, np[x] - 1)) { ok = false; break; }
          if (!begun[x] && !W(WB_Q_FULL + x, nq[x])) { ok = false; break; }
          tc_fence_after();
          if (lane == 0) {
            const int64_t sk = slot_k(j);
            const uint32_t ka = smem_u32(base + kWaOffRing + (int)(sk % kWaRing) * 32768);
            const uint32_t qa = smem_u32(base + kWaOffQ + x * 32768);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
              umma_bf16(tmem + 128 * x, smem_desc_sw128(qa + off, 16, 1024),
                        smem_desc_sw128(ka + off, 16, 1024), kIdS, kk > 0 ? 1u : 0u);
            }
            umma_commit(bar + WB_S_FULL + x);
            if (j == last[x]) umma_commit(bar + WB_Q_EMPTY + x);
          }
          __syncwarp();
          pend[x] = j;
        }
        // K(j) is free after this step's S, V(j - 1) after its P V
        if (ok && lane == 0) {
          if (j < it.nt) umma_commit(bar + WB_KV_EMPTY + (int)(slot_k(j) % kWaRing));
          if (j > 0) umma_commit(bar + WB_KV_EMPTY + (int)(slot_v(j - 1) % kWaRing));
        }
        __syncwarp();
      }
      n = n0 + 2 * (int64_t)it.nt;
      for (int x = 0; x < 2; ++x) {
        if (it.rows[x]) ++nq[x];
        if (last[x] >= 0) ++no[x];
      }
    }
    // every MMA issued has finished before the tensor memory is freed
    if (lane == 0) {
      umma_commit(bar + WB_DRAIN);
      mbar_drain(bar + WB_DRAIN, 0, err);
    }
    __syncwarp();
  }
  } else {
    setmaxnreg_inc<kWaRegsSoftmax>();
    // ---------------- softmax of row tile x; thread = row ----------------
    const int x = warp >> 2, quarter = warp & 3;
    const int row = quarter * 32 + lane;
    const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
    const uint32_t ts = tmem + lane_base + 128 * x, to = ts + 256;
    const float scale_log2 = a.scale * 1.4426950408889634f;
    const uint64_t scale2 = pack_f32x2(__float_as_uint(scale_log2), __float_as_uint(scale_log2));
    const int32_t tpt = 128 / a.R;            // tokens per row tile
    int64_t ns = 0, np = 0;
    bool ok = true;
    for (int64_t i = blockIdx.x; ok && i < n_items; i += gridDim.x) {
      win_item(it, a, i, tiles_per_item);
      const int32_t i_row = it.i0 + x * tpt + row / a.R;         // query index
      const int32_t t = it.q_pos0 + i_row;
      const int32_t i_w0 = it.i0 + x * tpt + (quarter * 32) / a.R;
      const int32_t t_min = it.q_pos0 + i_w0, t_max = t_min + (31 / a.R);
      float m = -INFINITY, l = 0.f;
      bool begun = false;
      for (int j = 0; j < it.nt; ++j) {
        if (!win_need(it, a, x, j)) continue;
        if (!W(WB_S_FULL + x, ns)) { ok = false; break; }
        ++ns;
        tc_fence_after();
        const int32_t k0 = win_key0(it, j);
        uint32_t s[128];
#pragma unroll
        for (int cc = 0; cc < 4; ++cc)
          tmem_ld_32x32b_x32(ts + 32 * cc, *reinterpret_cast<uint32_t(*)[32]>(s + 32 * cc));
        tmem_ld_wait();
        // visible columns c: c <= hi and (c >= lo or c < sk)
        int32_t hi, lo, sk;
        bool full;
        if (j < it.ns) {                      // a tile of sinks before the window
          hi = it.s_end - 1 - k0;
          lo = 0;
          sk = 0;
          full = hi >= 127;
        } else {
          hi = t - k0;
          lo = t - it.W + 1 - k0;
          sk = (int32_t)min64(max64(a.sink - k0, 0), 128);
          full = k0 + 127 <= t_min && (t_max - it.W + 1 <= k0 || sk >= 128);
        }
        if (!full) {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (!(c <= hi && (c >= lo || c < sk))) s[c] = 0xFF800000u;   // -inf
        }
        float mx = u2f(s[0]);
#pragma unroll
        for (int c = 1; c < 127; c += 2) mx = fmax3f(mx, u2f(s[c]), u2f(s[c + 1]));
        mx = fmaxf(mx, u2f(s[127])) * scale_log2;
        const bool grow = mx > m + kLazyLog2 || (m == -INFINITY && mx > -INFINITY);
        if (__any_sync(0xffffffffu, grow)) {
          const float mn = grow ? mx : m;
          const float f = m == -INFINITY ? 0.f : ex2_approx(m - mn);
          l *= f;
          m = mn;
          if (begun) {
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
          tmem_st_32x32b_x16(ts + 16 * cc, pk);
        }
        float u, v;
        unpack_f32x2(add_f32x2(l2[0], l2[1]), u, v);
        l += u + v;
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar + WB_P_FULL + x);
        begun = true;
        ++np;
      }
      if (!ok) break;
      // the item's rows leave: o = O / l
      const bool store = i_row < a.n_q && x < tiles_per_item;
      const bool live = store && t < it.len && begun;
      const int64_t orow =
          ((int64_t)it.b * a.n_q + i_row) * ((int64_t)a.G * a.R) + (int64_t)it.g * a.R + row % a.R;
      if (begun) {
        if (!W(WB_PV_DONE + x, np - 1)) { ok = false; break; }
        tc_fence_after();
      }
      const float inv = live && l != 0.f ? 1.f / l : 0.f;
      if (store) a.lse[orow] = live ? m * 0.6931471805599453f + logf(l) : -INFINITY;
#pragma unroll 1
      for (int cc = 0; cc < 4; ++cc) {
        uint32_t r[32];
        if (begun) {
          tmem_ld_32x32b_x32(to + 32 * cc, r);
          tmem_ld_wait();
        }
        if (store) {
          __nv_bfloat16* dst = a.out + orow * kHeadDim + 32 * cc;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
              pk[q] = live ? pack_bf16x2(u2f(r[16 * h + 2 * q]) * inv,
                                         u2f(r[16 * h + 2 * q + 1]) * inv)
                           : 0u;
            st_global_v8(reinterpret_cast<float*>(dst + 16 * h), u2f(pk[0]), u2f(pk[1]),
                         u2f(pk[2]), u2f(pk[3]), u2f(pk[4]), u2f(pk[5]), u2f(pk[6]), u2f(pk[7]));
          }
        }
      }
      if (begun) {
        tc_fence_before();
        mbar_arrive(bar + WB_O_EMPTY + x);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 512);
}

cudaError_t launch_window_attn_fwd(const CUtensorMap& tm_q, const CUtensorMap& tm_k,
                                   const CUtensorMap& tm_v, const WindowArgs& a,
                                   cudaStream_t st) {
  static KernelSetup setup;
  int sms = 0;
  cudaError_t e = kernel_setup(setup, reinterpret_cast<const void*>(window_attn_fwd_kernel), kWaSmemBytes, kWaRegsAtLaunch, &sms);
  if (e != cudaSuccess) return e;
  // two row tiles per item overlap their products and softmax; one per item
  // when that would leave SMs without work
  const int64_t tiles = (a.n_q * a.R + 127) / 128;
  int32_t per = 2;
  if (a.batch * a.G * ((tiles + 1) / 2) < sms) per = 1;
  const int64_t items = a.batch * a.G * ((tiles + per - 1) / per);
  window_attn_fwd_kernel<<<(unsigned)min64(items, sms), kWaThreads, kWaSmemBytes, st>>>(
      tm_q, tm_k, tm_v, a, per, items);
  return cudaGetLastError();
}

}  // namespace msa
