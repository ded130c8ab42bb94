// Which key tiles a window-attention item walks: shared by every warp role of
// the forward and the dq kernel, so that all see the same sequence.
#pragma once

#include "common.cuh"
#include "layer_args.cuh"

namespace msa {

// one thread of the warp, always the same, in a form that lets the compiler keep
// what the branch computes in uniform registers (tcgen05.mma takes its operands
// from there)
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(e));
  return e != 0;
}

// An item: one or two adjacent row tiles (128 / R queries x R heads each) of
// one (batch, group), and its key tiles: the `nc` chunks of 32 keys that hold the
// sinks [0, s_end) before the window, then the window's from wlo on, four chunks a
// tile.  (A tile of its own for a few sinks is a tenth of the work of a
// 1024-key window.)  Sinks that reach the window make one run from key 0.
struct WinItem {
  int32_t b, g, i0;          // first query of row tile A
  int32_t q_pos0, W, len;    // len: min(kv_len[b], q_pos0 + n_q)
  int32_t wlo, s_end, nc, nt;
  int32_t j0;                // first tile of this CTA's share (cluster), its nt tiles follow
  int32_t end_a, beg_b;      // last key tile that A sees; first behind the sinks that B sees
  bool rows[2];              // row tile X has a query below n_q and len
  int32_t x0[2], x1[2];      // positions of its first and last such query
};

// the keys that a query of sequence b can see end here: behind its last token, and behind
// the last query of the call (a cache may be longer than what has been written)
__device__ __forceinline__ int32_t win_len(const WindowArgs& a, int32_t b) {
  const int32_t n = (int32_t)(a.q_pos0 + a.n_q);         // <= n_kv
  if (a.kv_len == nullptr) return n;
  const int32_t v = __ldg(a.kv_len + b);
  if (v < 0 || v > a.n_kv) report(a.err, MSA_DEVERR_BAD_LENGTH);
  return max(0, min(v, n));
}

// items in descending query order over all (batch, group): with no window the
// longest rows go first
__device__ __forceinline__ void win_item(WinItem& it, const WindowArgs& a, int32_t i,
                                         int32_t per) {
  const int32_t step = 128 / a.R * per, n_it = ((int32_t)a.n_q + step - 1) / step;
  const int32_t tpt = 128 / a.R, n_bg = (int32_t)a.batch * a.G, r = i / n_bg, bg = i - r * n_bg;
  it.b = bg / a.G;
  it.g = bg - it.b * a.G;
  it.i0 = (n_it - 1 - r) * step;
  it.q_pos0 = (int32_t)a.q_pos0;
  it.W = a.window > 0 ? (int32_t)min64(a.window, int64_t(1) << 30) : 1 << 30;
  it.len = win_len(a, it.b);
  int32_t tlo = 0, thi = -1;
  for (int x = 0; x < 2; ++x) {
    const int32_t f = it.i0 + x * tpt;
    const int32_t e = (int32_t)min64(min64(f + tpt, a.n_q) - 1, (int64_t)it.len - 1 - it.q_pos0);
    it.rows[x] = x < per && e >= f;
    it.x0[x] = it.q_pos0 + f;
    it.x1[x] = it.q_pos0 + e;
    if (it.rows[x]) {
      if (thi < 0) tlo = it.x0[x];
      thi = it.x1[x];
    }
  }
  it.wlo = max(0, tlo - it.W + 1);
  if (a.sink >= it.wlo) it.wlo = 0;
  it.s_end = (int32_t)min64(a.sink, it.wlo);
  it.j0 = 0;
  it.nc = thi < 0 ? 0 : (it.s_end + 31) / 32;
  it.nt = thi < 0 ? 0 : (it.nc + (thi + 1 - it.wlo + 31) / 32 + 3) / 4;
  it.end_a = it.rows[0] ? (it.nc + (it.x1[0] - it.wlo) / 32) / 4 : -1;
  it.beg_b = it.rows[1] && a.sink <= it.wlo && it.wlo > 0
                 ? (it.nc + max(0, it.x0[1] - it.W + 1 - it.wlo) / 32) / 4
                 : 0;
}
// first key of chunk q; the tile of chunks 4 j .. 4 j + 3 is one run of keys unless mixed
__device__ __forceinline__ int32_t win_chunk(const WinItem& it, int q) {
  return q < it.nc ? 32 * q : it.wlo + 32 * (q - it.nc);
}
__device__ __forceinline__ bool win_mixed(const WinItem& it, int j) {
  return 4 * j < it.nc && 4 * j + 4 > it.nc;
}
// columns lo .. hi - 1 of the 32 from c0 on, as bits
__device__ __forceinline__ uint32_t range_bits(int32_t lo, int32_t hi, int32_t c0) {
  lo = max(lo - c0, 0);
  hi = min(hi - c0, 32);
  if (lo >= hi) return 0u;
  return (0xffffffffu >> (32 - hi)) & (0xffffffffu << lo);
}
// of chunk q's 32 keys, those that the query at position t sees, as bits
__device__ __forceinline__ uint32_t win_visible(const WinItem& it, int q, int32_t t,
                                                int32_t sink) {
  const int32_t kc = win_chunk(it, q), hi = t + 1 - kc;
  return q < it.nc ? range_bits(0, it.s_end - kc, 0)
                   : range_bits(hi - it.W, hi, 0) | range_bits(0, min(sink - kc, hi), 0);
}
// brings key tile j by TMA: two 128 x 64 boxes, or 32 x 64 ones for a mixed tile
__device__ __forceinline__ void win_load_keys(uint8_t* dst, const CUtensorMap* tm,
                                              const CUtensorMap* tm32, uint64_t* bar,
                                              const WinItem& it, int j) {
  if (!win_mixed(it, j)) {
    const int32_t k0 = win_chunk(it, 4 * j);
    tma_load_4d(dst, tm, bar, 0, k0, it.g, it.b);
    tma_load_4d(dst + 16384, tm, bar, 64, k0, it.g, it.b);
  } else {
    for (int i = 0; i < 8; ++i)
      tma_load_4d(dst + (i >> 2) * 16384 + (i & 3) * 4096, tm32, bar, 64 * (i >> 2),
                  win_chunk(it, 4 * j + (i & 3)), it.g, it.b);
  }
}

// zeroes rows r0 .. r1 - 1 of a 128 x 128 bf16 tile (two 64-column panels), by a warp
__device__ __forceinline__ void win_clear_rows(uint8_t* tile, int32_t r0, int32_t r1, int lane) {
  r0 = max(r0, 0);
  for (int r = r0; r < r1; ++r)
    *reinterpret_cast<uint2*>(tile + (lane >> 4) * 16384 + r * 128 + (lane & 15) * 8) =
        make_uint2(0, 0);
  fence_proxy_async_smem();
  __syncwarp();
}
// the rows of key tile j at or behind the end of what queries see
__device__ __forceinline__ void win_clear_keys(uint8_t* tile, const WinItem& it, int j,
                                               int lane) {
  for (int i = 0; i < 4; ++i) {
    const int32_t k0 = win_chunk(it, 4 * j + i);
    if (k0 + 32 > it.len)
      win_clear_rows(tile, 32 * i + max(it.len - k0, 0), 32 * i + 32, lane);
  }
}

}  // namespace msa
