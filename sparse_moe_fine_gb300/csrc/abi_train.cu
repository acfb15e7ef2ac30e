// The extern "C" entry points declared in include/usaf_train.h: argument checks, workspace carving
// and the launch of each call. The arithmetic is in router_aux.cu, router_grad.cu and act8.cu.
#include "train.cuh"

using namespace usaf;

namespace {

bool aux_shape_ok(int64_t T, int64_t E, int64_t k, int64_t G) {
  return T >= 1 && E >= 1 && E <= 1024 && k >= 1 && k <= E && k <= 32 && G >= 1 &&
         G <= (int64_t(1) << 20) && T < (int64_t(1) << 31) - 65536 &&
         T * k < (int64_t(1) << 31) - 65536;
}

bool grad_shape_ok(int64_t T, int64_t E, int64_t H, usaf_dtype dt) {
  return T >= 1 && T < (int64_t(1) << 31) - 65536 && E >= 1 && E <= 1024 && H >= 1 &&
         H < (int64_t(1) << 31) && E * H < (int64_t(1) << 31) &&
         (dt == USAF_F32 || dt == USAF_BF16);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// the coefficients are host scalars: a NaN or infinity is an argument error
bool coef_ok(double c) { return std::isfinite(c) && std::isfinite((float)c); }

usaf_status fill_aux(AuxArgs& a, int64_t T, int64_t E, int64_t k, const float* logits, int64_t ld,
                     const uint8_t* mask, const int32_t* offset, int64_t G, double cb, double cz,
                     uint32_t* status) {
  if (!aux_shape_ok(T, E, k, G) || !logits || ld < E) return USAF_ERR_INVALID_ARG;
  if (!offset && G != 1) return USAF_ERR_INVALID_ARG;
  if (!coef_ok(cb) || !coef_ok(cz)) return USAF_ERR_INVALID_ARG;
  a.T = T;
  a.G = G;
  a.ld = ld;
  a.E = (int)E;
  a.k = (int)k;
  a.logits = logits;
  a.mask = mask;
  a.offset = offset;
  a.coef_balance = cb;
  a.coef_z = cz;
  a.status = status;
  return USAF_OK;
}

usaf_status fill_act8(Act8Args& a, const usaf_moe_shape* s, usaf_dtype dt, const void* x_code,
                      const void* x_exp, const void* h_code, const void* h_exp,
                      const usaf_routing* rt) {
  const int64_t cap = s ? usaf_routed_rows_capacity(s) : -1;
  if (cap < 0 || (dt != USAF_F32 && dt != USAF_BF16)) return USAF_ERR_INVALID_ARG;
  if (!x_code || !x_exp || !h_code || !h_exp || !rt || !rt->expert_offset)
    return USAF_ERR_INVALID_ARG;
  if (!aligned16(x_code) || !aligned16(x_exp) || !aligned16(h_code) || !aligned16(h_exp))
    return USAF_ERR_INVALID_ARG;
  a.s = *s;
  a.dt = dt;
  a.R_cap = cap;
  a.rt = *rt;
  a.x_code = static_cast<int8_t*>(const_cast<void*>(x_code));
  a.x_exp = static_cast<uint8_t*>(const_cast<void*>(x_exp));
  a.h_code = static_cast<int8_t*>(const_cast<void*>(h_code));
  a.h_exp = static_cast<uint8_t*>(const_cast<void*>(h_exp));
  return USAF_OK;
}

}  // namespace

extern "C" {

size_t usaf_router_aux_workspace_size(int64_t T, int64_t E, int64_t k, int64_t G) {
  if (!aux_shape_ok(T, E, k, G)) return 0;
  Carver c(nullptr);
  AuxWs w;
  aux_ws_layout(T, E, G, c, w);
  return c.size();
}

usaf_status usaf_router_aux_fwd(int64_t T, int64_t E, int64_t k, const float* logits,
                                int64_t ld_logits, const int32_t* topk_idx,
                                const uint8_t* token_mask, const int32_t* group_offset, int64_t G,
                                double coef_balance, double coef_z, int32_t* count,
                                float* prob_sum, int32_t* n_tok, float* loss,
                                uint32_t* dev_status, void* ws, size_t ws_bytes, void* stream) {
  AuxArgs a{};
  USAF_TRY(fill_aux(a, T, E, k, logits, ld_logits, token_mask, group_offset, G, coef_balance,
                    coef_z, dev_status));
  if (!topk_idx || !count || !prob_sum || !n_tok || !loss) return USAF_ERR_INVALID_ARG;
  if (!ws || ws_bytes < usaf_router_aux_workspace_size(T, E, k, G)) return USAF_ERR_WORKSPACE;
  if (!aligned16(ws)) return USAF_ERR_INVALID_ARG;
  a.topk_idx = topk_idx;
  Carver c(ws);
  AuxWs w;
  aux_ws_layout(T, E, G, c, w);
  return aux_fwd_launch(a, count, prob_sum, n_tok, loss, w, static_cast<cudaStream_t>(stream));
}

usaf_status usaf_router_aux_bwd(int64_t T, int64_t E, int64_t k, const float* logits,
                                int64_t ld_logits, const uint8_t* token_mask,
                                const int32_t* group_offset, int64_t G, double coef_balance,
                                double coef_z, const int32_t* count, const int32_t* n_tok,
                                const float* d_loss, float* dlogit, int64_t ld_dlogit,
                                int accumulate, uint32_t* dev_status, void* stream) {
  AuxArgs a{};
  USAF_TRY(fill_aux(a, T, E, k, logits, ld_logits, token_mask, group_offset, G, coef_balance,
                    coef_z, dev_status));
  if (!count || !n_tok || !dlogit || ld_dlogit < E) return USAF_ERR_INVALID_ARG;
  if (accumulate != 0 && accumulate != 1) return USAF_ERR_INVALID_ARG;
  if (dlogit == logits && (accumulate || ld_dlogit != ld_logits)) return USAF_ERR_INVALID_ARG;
  return aux_bwd_launch(a, count, n_tok, d_loss, dlogit, ld_dlogit, accumulate,
                        static_cast<cudaStream_t>(stream));
}

size_t usaf_router_grad_workspace_size(int64_t T, int64_t E, int64_t H, usaf_dtype dtype) {
  if (!grad_shape_ok(T, E, H, dtype) || (dtype == USAF_BF16 && H % 64 != 0)) return 0;
  Carver c(nullptr);
  RouterGradWs w;
  router_grad_ws_layout(T, E, H, dtype, c, w);
  return c.size();
}

usaf_status usaf_router_grad(int64_t T, int64_t E, int64_t H, usaf_dtype dtype,
                             const float* dlogit, int64_t ld_dlogit, const void* x,
                             const float* w_router, const float* g_in, float* g_router,
                             const void* dx_in, void* dx, uint32_t* dev_status, void* ws,
                             size_t ws_bytes, void* stream) {
  if (!grad_shape_ok(T, E, H, dtype) || !dlogit || ld_dlogit < E) return USAF_ERR_INVALID_ARG;
  if ((!g_router && !dx) || (g_router && !x) || (dx && !w_router)) return USAF_ERR_INVALID_ARG;
  // dx is written while g_router's product may still read x
  if (g_router && dx && dx == x) return USAF_ERR_INVALID_ARG;
  if (dtype == USAF_BF16) {
    if (H % 64 != 0) return USAF_ERR_UNSUPPORTED;
    if (!aligned16(x) || !aligned16(dx_in) || !aligned16(dx) || !aligned16(w_router))
      return USAF_ERR_INVALID_ARG;
  }
  if (!ws || ws_bytes < usaf_router_grad_workspace_size(T, E, H, dtype)) return USAF_ERR_WORKSPACE;
  if (!aligned16(ws)) return USAF_ERR_INVALID_ARG;
  RouterGradArgs a{T, E, H, ld_dlogit, dtype, dlogit, x, w_router, g_in, g_router, dx_in, dx,
                   dev_status};
  Carver c(ws);
  RouterGradWs w;
  router_grad_ws_layout(T, E, H, dtype, c, w);
  return router_grad_launch(a, w, static_cast<cudaStream_t>(stream));
}

usaf_status usaf_act8_save(const usaf_moe_shape* shape, usaf_dtype dtype, const void* x,
                           const void* h, const usaf_routing* rt, int8_t* x_code, uint8_t* x_exp,
                           int8_t* h_code, uint8_t* h_exp, uint32_t* dev_status, void* stream) {
  Act8Args a{};
  USAF_TRY(fill_act8(a, shape, dtype, x_code, x_exp, h_code, h_exp, rt));
  if (!x || !h || !aligned16(x) || !aligned16(h)) return USAF_ERR_INVALID_ARG;
  return act8_save_launch(a, x, h, dev_status, static_cast<cudaStream_t>(stream));
}

usaf_status usaf_act8_restore(const usaf_moe_shape* shape, usaf_dtype dtype, const int8_t* x_code,
                              const uint8_t* x_exp, const int8_t* h_code, const uint8_t* h_exp,
                              const usaf_routing* rt, void* x_out, void* x_perm, void* h,
                              void* wa, void* stream) {
  Act8Args a{};
  USAF_TRY(fill_act8(a, shape, dtype, x_code, x_exp, h_code, h_exp, rt));
  if (!x_perm || !h || !wa || !rt->topk_w || !rt->perm_tok || !rt->perm_slot)
    return USAF_ERR_INVALID_ARG;
  if (!aligned16(x_out) || !aligned16(x_perm) || !aligned16(h) || !aligned16(wa) ||
      !aligned16(rt->perm_tok) || !aligned16(rt->perm_slot))
    return USAF_ERR_INVALID_ARG;
  return act8_restore_launch(a, x_out, x_perm, h, wa, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
