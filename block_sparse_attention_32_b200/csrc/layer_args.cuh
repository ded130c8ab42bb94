// Launch arguments shared by the C ABI and the kernels of the operators around
// the sparse path (norm + rotation, paged decode, window attention).
#pragma once

#include <atomic>

#include "common.cuh"

namespace msa {

// Host: the current device's SM count, after setting the kernel's shared-memory
// limit (and, with regs > 0, checking its compiled register count, which a kernel
// that shares registers out among its warpgroups relies on).  Done once per
// device; `done` is the kernel's own table.
struct KernelSetup {
  std::atomic<int> sms[64];
};
inline cudaError_t kernel_setup(KernelSetup& done, const void* kernel, int smem, int regs,
                                int* sms) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool kept = dev >= 0 && dev < 64;
  if (kept && (*sms = done.sms[dev].load(std::memory_order_acquire)) > 0) return cudaSuccess;
  if ((e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
    return e;
  if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) !=
      cudaSuccess)
    return e;
  if (regs > 0) {
    cudaFuncAttributes attr;
    if ((e = cudaFuncGetAttributes(&attr, kernel)) != cudaSuccess) return e;
    if (attr.numRegs != regs) return cudaErrorInvalidConfiguration;
  }
  if (kept) done.sms[dev].store(*sms, std::memory_order_release);
  return cudaSuccess;
}

// Dependent launches: the kernel's blocks may take their places while the one
// before it on the stream still runs (after its grid_launch_dependents), and
// wait there, in grid_wait, until it is complete and its writes are visible -- to plain
// loads: what that kernel wrote is not read by __ldg or through const __restrict__, which
// promise data that stays as it is while the kernel runs.
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem,
                             cudaStream_t st, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// 32 lanes x 16 consecutive 32-bit TMEM columns
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

struct NormRopeArgs {
  const __nv_bfloat16* src[3];   // q, k, v (v: paged form only, copied)
  int64_t ss_b[3], ss_t[3], ss_h[3];
  __nv_bfloat16* dst[3];         // q_out, k_out (dense) or the K / V pages
  int64_t ds_b[3], ds_t[3], ds_h[3];   // paged k, v: ds_b is the page stride
  const float* w[2];             // may be null: ones
  const float* table;            // [n_pos, rot]: rot / 2 cosines, rot / 2 sines
  const int64_t* positions;      // [B, T], null: pos0 + i
  int64_t n_pos, pos0, batch, n_tok, n_items;
  const int32_t* block_table;    // paged form: [B, table_stride]
  int64_t table_stride, n_pages;
  int32_t page_size;
  int32_t heads[3];              // h_q, h_k, h_k (0 without v)
  int32_t chunks[3];             // ceil(heads / hc)
  int32_t hc, rot;
  float eps;
  int32_t* err;
};

struct NormRopeBwdArgs {
  NormRopeArgs f;                 // src: q, k; dst: dx of q, k; w, table, positions, sizes
  const void* dy[2];              // bf16 or fp32
  int64_t ys_b[2], ys_t[2], ys_h[2];
  float* part;                    // [grid, 2, D] weight-gradient sums of each block
};

struct PagedDecodeArgs {
  const __nv_bfloat16* q;         // [B, 1, H, 128]
  int64_t qs_b, qs_h;
  const int32_t* block_table;     // [B, table_stride]
  const int32_t* seq_lens;        // [B]
  int64_t table_stride, n_pages;
  int32_t cap;                    // tokens a sequence may have (< 2^30)
  int32_t page_size, page_shift, batch, G, R;   // page_size = 1 << page_shift
  int32_t window, sink;           // in [1, cap], [0, cap]
  float scale;
  __nv_bfloat16* out;             // [B, 1, H, 128]
  float* lse;                     // [B, 1, H]
  int32_t* prefix;                // workspace: [B + 1] tiles before each sequence (per group)
  float* part_ml;                 // workspace: [workers, 2, R, 2]
  float* part_acc;                // workspace: [workers, 2, R, 128]
  int32_t* err;
};

struct WindowArgs {
  const __nv_bfloat16 *o, *d_o;   // [B, n_q, H, 128], strided (backward)
  int64_t os_b, os_t, os_h, ds_b, ds_t, ds_h;
  int64_t batch, n_q, n_kv, q_pos0;
  int64_t window, sink;           // visible: j <= t and (t - j < window or j < sink)
  int32_t G, R;
  float scale;
  const int32_t* kv_len;          // [B] or null: queries at positions >= kv_len are padding
  __nv_bfloat16* out;             // [B, n_q, H, 128]
  int8_t* rest;                   // [B, n_q, H, 128] or null: the 8 bits behind out
  float* lse;                     // [B, n_q, H]
  __nv_bfloat16 *dq, *dk, *dv;    // backward
  int32_t* err;
};

}  // namespace msa
