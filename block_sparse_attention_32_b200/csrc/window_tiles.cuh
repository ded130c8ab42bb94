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
// one (batch, group), and its key tiles: `ns` tiles of sinks [0, s_end) that lie
// before the window, then tiles of 128 keys from `wlo` on.
struct WinItem {
  int32_t b, g, i0;          // first query of row tile A
  int32_t q_pos0, W, len;    // len: min(kv_len[b], n_kv)
  int32_t wlo, s_end, ns, nt;
  int32_t end_a, beg_b;      // last key tile that A sees; first behind the sinks that B sees
  bool rows[2];              // row tile X has a query below n_q and len
  int32_t x0[2], x1[2];      // positions of its first and last such query
};

__device__ __forceinline__ int32_t win_len(const WindowArgs& a, int32_t b) {
  const int32_t n = (int32_t)a.n_kv;
  if (a.kv_len == nullptr) return n;
  const int32_t v = __ldg(a.kv_len + b);
  if (v < 0 || v > n) report(a.err, MSA_DEVERR_BAD_LENGTH);
  return max(0, min(v, n));
}

// items in descending query order: with no window the longest rows go first
__device__ __forceinline__ void win_item(WinItem& it, const WindowArgs& a, int64_t i,
                                         int32_t per) {
  const int32_t tpt = 128 / a.R;
  const int64_t n_it = (a.n_q + (int64_t)tpt * per - 1) / ((int64_t)tpt * per);
  const int64_t bg = i / n_it;
  it.b = (int32_t)(bg / a.G);
  it.g = (int32_t)(bg - (int64_t)it.b * a.G);
  it.i0 = (int32_t)(n_it - 1 - (i - bg * n_it)) * tpt * per;
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
  it.s_end = (int32_t)min64(a.sink, it.wlo);
  it.ns = thi < 0 ? 0 : (it.s_end + 127) / 128;
  it.nt = thi < 0 ? 0 : it.ns + (thi + 1 - it.wlo + 127) / 128;
  it.end_a = it.rows[0] ? it.ns + (it.x1[0] - it.wlo) / 128 : -1;
  // (sinks that reach past wlo are visible to B from the first tile on)
  it.beg_b = it.rows[1] && a.sink <= it.wlo ? it.ns + max(0, it.x0[1] - it.W + 1 - it.wlo) / 128
                                            : it.ns;
}
__device__ __forceinline__ int32_t win_key0(const WinItem& it, int j) {
  return j < it.ns ? 128 * j : it.wlo + 128 * (j - it.ns);
}

// zeroes rows r0 .. 127 of a 128 x 128 bf16 tile (two 64-column panels), by a warp
__device__ __forceinline__ void win_clear_rows(uint8_t* tile, int32_t r0, int lane) {
  r0 = max(r0, 0);
  for (int r = r0; r < 128; ++r)
    *reinterpret_cast<uint2*>(tile + (lane >> 4) * 16384 + r * 128 + (lane & 15) * 8) =
        make_uint2(0, 0);
  fence_proxy_async_smem();
  __syncwarp();
}

}  // namespace msa
