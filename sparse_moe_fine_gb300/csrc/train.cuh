// Internal launch interfaces of the calls declared in usaf_train.h.
#pragma once

#include <atomic>

#include "common.cuh"
#include "usaf_train.h"

namespace usaf {

// A kernel that may be set up while the one before it in the stream still runs: it must pass
// dep_wait(), in every thread, before it touches memory that other kernels write or read, whichever
// of the kernels before it that was: a kernel that has let the next one in orders nothing for it before
// it ends. A kernel lets the next one in by dep_launch(); one that never does lets it in when it ends.
__device__ __forceinline__ void dep_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void dep_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <class... P, class... A>
usaf_status launch_dep(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem,
                       cudaStream_t st, const A&... args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...) != cudaSuccess) {
    cudaGetLastError();  // reported here, not again by the next launch's check
    return USAF_ERR_CUDA;
  }
  count_launch();
  return USAF_OK;
}

// Runs set() once for each device that is current when it is called (a kernel's attributes belong to
// a device; setting them again costs a small call about a microsecond). set() returns success; one
// that failed is tried again by the next call. One variable of this type per kernel.
struct OncePerDevice {
  std::atomic<uint64_t> done{0};
  template <class F>
  bool operator()(F set) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return true;
    if (!set()) return false;
    done.fetch_or(bit, std::memory_order_release);
    return true;
  }
};

// ---------------------------------------------------------------- router auxiliary losses
struct AuxArgs {
  int64_t T, G, ld;
  int E, k;
  const float* logits;
  const int32_t* topk_idx;
  const uint8_t* mask;    // [T] or null
  const int32_t* offset;  // [G+1] or null (one group)
  double coef_balance, coef_z;
  uint32_t* status;
};
// Partial sums of the forward: a chunk of tokens and a group that meet own slot chunk + group
// (each step along the tokens moves to the next chunk, the next group or both, so no two share one).
struct AuxWs {
  float* prob;  // [slots][E]
  int32_t* count;
  int32_t* n;  // [slots]
  float* z;
  float* bal;         // [G][ceil(E / 32)] shares of the balance sum
  float* group_z;     // [G]
  uint32_t* arrived;  // blocks of the final kernel that are done
};
int64_t aux_chunk_tokens(int64_t T, int64_t E);  // tokens of a chunk
void aux_ws_layout(int64_t T, int64_t E, int64_t G, Carver& c, AuxWs& w);
usaf_status aux_fwd_launch(const AuxArgs& a, int32_t* count, float* prob_sum, int32_t* n_tok,
                           float* loss, const AuxWs& w, cudaStream_t st);
usaf_status aux_bwd_launch(const AuxArgs& a, const int32_t* count, const int32_t* n_tok,
                           const float* d_loss, float* dlogit, int64_t ld_out, int accumulate,
                           cudaStream_t st);

// ---------------------------------------------------------------- router gradient products
struct RouterGradArgs {
  int64_t T, E, H, ld;
  usaf_dtype dt;
  const float* dlogit;
  const void* x;
  const float* w_router;
  const float* g_in;
  float* g_router;
  const void* dx_in;
  void* dx;
  uint32_t* status;
};
struct RouterGradWs {
  float* g_part;  // [splits][E][H] sums of g_router over stretches of the tokens
  void* parts;    // bf16 layers: [T][3][experts in eights] dlogit in three bf16 parts
  void* w_parts;  // [2][experts in sixteens][H] w_router in two bf16 parts
};
void router_grad_ws_layout(int64_t T, int64_t E, int64_t H, usaf_dtype dt, Carver& c,
                           RouterGradWs& w);
usaf_status router_grad_launch(const RouterGradArgs& a, const RouterGradWs& w, cudaStream_t st);
// the same on tensor cores (bf16 x, dx)
void router_grad_tc_layout(int64_t T, int64_t E, int64_t H, Carver& c, RouterGradWs& w);
usaf_status router_grad_tc(const RouterGradArgs& a, const RouterGradWs& w, cudaStream_t st);

// ---------------------------------------------------------------- 8-bit activation store
struct Act8Args {
  usaf_moe_shape s;
  usaf_dtype dt;
  int64_t R_cap;
  usaf_routing rt;
  int8_t* x_code;
  uint8_t* x_exp;
  int8_t* h_code;
  uint8_t* h_exp;
};
usaf_status act8_save_launch(const Act8Args& a, const void* x, const void* h, uint32_t* status,
                             cudaStream_t st);
usaf_status act8_restore_launch(const Act8Args& a, void* x_out, void* x_perm, void* h, void* wa,
                                cudaStream_t st);

}  // namespace usaf
