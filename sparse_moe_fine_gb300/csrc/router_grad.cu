// The two products of a dense router gradient (usaf_router_grad): g_router = g_in + dlogit^T x and
// dx = dx_in + dlogit w_router. Here for fp32 tokens, on CUDA cores in fp32; bf16 tokens are in
// router_grad_tc.cu.
#include "train.cuh"

namespace usaf {

namespace {

constexpr int RG_E = 32, RG_H = 64, RG_T = 32;  // tile of g_router, tokens per step
constexpr int DX_T = 64, DX_H = 64, DX_E = 32;  // tile of dx, experts per step

// part[s][e][h] = sum over the tokens of split s of dlogit[t,e] x[t,h]; with one split the result
// goes to g_router (+ g_in).
__global__ void __launch_bounds__(256)
    router_grad_w_kernel(const RouterGradArgs a, int64_t per_split, float* __restrict__ part) {
  __shared__ float s_d[RG_T][RG_E];
  __shared__ float s_x[RG_T][RG_H];
  const float* x = static_cast<const float*>(a.x);
  const int h0 = blockIdx.x * RG_H, e0 = blockIdx.y * RG_E;
  const int64_t t0 = blockIdx.z * per_split, t1 = min(a.T, t0 + per_split);
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;  // 4 h, 2 e
  float acc[2][4] = {};
  for (int64_t t = t0; t < t1; t += RG_T) {
    for (int i = threadIdx.x; i < RG_T * RG_E; i += 256) {
      const int r = i / RG_E, c = i % RG_E;
      s_d[r][c] = t + r < t1 && e0 + c < a.E ? a.dlogit[(t + r) * a.ld + e0 + c] : 0.f;
    }
    for (int i = threadIdx.x; i < RG_T * RG_H; i += 256) {
      const int r = i / RG_H, c = i % RG_H;
      s_x[r][c] = t + r < t1 && h0 + c < a.H ? x[(t + r) * a.H + h0 + c] : 0.f;
    }
    __syncthreads();
#pragma unroll 8
    for (int r = 0; r < RG_T; ++r) {
      const float4 xv = *reinterpret_cast<const float4*>(&s_x[r][tx * 4]);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float d = s_d[r][ty * 2 + u];
        acc[u][0] = fmaf(d, xv.x, acc[u][0]);
        acc[u][1] = fmaf(d, xv.y, acc[u][1]);
        acc[u][2] = fmaf(d, xv.z, acc[u][2]);
        acc[u][3] = fmaf(d, xv.w, acc[u][3]);
      }
    }
    __syncthreads();
  }
  const bool last = gridDim.z == 1;
  bool bad = false;
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int e = e0 + ty * 2 + u, h = h0 + tx * 4 + q;
      if (e >= a.E || h >= a.H) continue;
      const int64_t i = (int64_t)e * a.H + h;
      if (last) {
        const float v = (a.g_in ? a.g_in[i] : 0.f) + acc[u][q];
        a.g_router[i] = v;
        bad |= !finite_f(v);
      } else {
        part[blockIdx.z * a.E * a.H + i] = acc[u][q];
      }
    }
  flag_status_warp(a.status, bad, USAF_DEV_NONFINITE);
}

// g_router = g_in + the splits' sums in split order
__global__ void __launch_bounds__(256)
    router_grad_reduce_kernel(const RouterGradArgs a, const float* __restrict__ part, int splits) {
  const int64_t n = a.E * a.H;
  bool bad = false;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    float v = a.g_in ? a.g_in[i] : 0.f;
    for (int s = 0; s < splits; ++s) v += part[s * n + i];
    a.g_router[i] = v;
    bad |= !finite_f(v);
  }
  flag_status_warp(a.status, bad, USAF_DEV_NONFINITE);
}

__global__ void __launch_bounds__(256) router_grad_x_kernel(const RouterGradArgs a) {
  __shared__ float s_d[DX_T][DX_E + 1];
  __shared__ float s_w[DX_E][DX_H];
  const float* dx_in = static_cast<const float*>(a.dx_in);
  float* dx = static_cast<float*>(a.dx);
  const int h0 = blockIdx.x * DX_H;
  const int64_t t0 = (int64_t)blockIdx.y * DX_T;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  for (int e0 = 0; e0 < a.E; e0 += DX_E) {
    for (int i = threadIdx.x; i < DX_T * DX_E; i += 256) {
      const int r = i / DX_E, c = i % DX_E;
      s_d[r][c] = t0 + r < a.T && e0 + c < a.E ? a.dlogit[(t0 + r) * a.ld + e0 + c] : 0.f;
    }
    for (int i = threadIdx.x; i < DX_E * DX_H; i += 256) {
      const int r = i / DX_H, c = i % DX_H;
      s_w[r][c] = e0 + r < a.E && h0 + c < a.H ? a.w_router[(e0 + r) * a.H + h0 + c] : 0.f;
    }
    __syncthreads();
#pragma unroll 8
    for (int r = 0; r < DX_E; ++r) {
      const float4 wv = *reinterpret_cast<const float4*>(&s_w[r][tx * 4]);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float d = s_d[ty * 4 + u][r];
        acc[u][0] = fmaf(d, wv.x, acc[u][0]);
        acc[u][1] = fmaf(d, wv.y, acc[u][1]);
        acc[u][2] = fmaf(d, wv.z, acc[u][2]);
        acc[u][3] = fmaf(d, wv.w, acc[u][3]);
      }
    }
    __syncthreads();
  }
  bool bad = false;
#pragma unroll
  for (int u = 0; u < 4; ++u)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t t = t0 + ty * 4 + u;
      const int h = h0 + tx * 4 + q;
      if (t >= a.T || h >= a.H) continue;
      const float v = (dx_in ? dx_in[t * a.H + h] : 0.f) + acc[u][q];
      dx[t * a.H + h] = v;
      bad |= !finite_f(v);
    }
  flag_status_warp(a.status, bad, USAF_DEV_NONFINITE);
}

// Parts of the token axis that g_router's sum is split into: about two blocks per SM, at least
// 64 tokens each.
int64_t splits_for(int64_t T, int64_t E, int64_t H) {
  const int64_t tiles = ceil_div(E, RG_E) * ceil_div(H, RG_H);
  int64_t s = ceil_div(2 * 152, tiles);
  const int64_t most = ceil_div(T, 64);
  if (s > most) s = most;
  return s < 1 ? 1 : s;
}

usaf_status launch_reduce(const RouterGradArgs& a, const float* part, int64_t splits,
                          cudaStream_t st) {
  USAF_TRACE("router_grad_reduce", st);
  router_grad_reduce_kernel<<<grid_dim_for(a.E * a.H), 256, 0, st>>>(a, part, (int)splits);
  USAF_CHECK_LAUNCH();
  return USAF_OK;
}

usaf_status launch_w(const RouterGradArgs& a, float* part, cudaStream_t st) {
  const int64_t s = splits_for(a.T, a.E, a.H);
  const int64_t per = round_up(ceil_div(a.T, s), RG_T);
  const dim3 grid((unsigned)ceil_div(a.H, RG_H), (unsigned)ceil_div(a.E, RG_E),
                  (unsigned)ceil_div(a.T, per));
  {
    USAF_TRACE("router_grad_w", st);
    router_grad_w_kernel<<<grid, 256, 0, st>>>(a, per, part);
    USAF_CHECK_LAUNCH();
  }
  return grid.z > 1 ? launch_reduce(a, part, grid.z, st) : USAF_OK;
}

usaf_status launch_x(const RouterGradArgs& a, cudaStream_t st) {
  USAF_TRACE("router_grad_x", st);
  const int64_t rows = ceil_div(a.T, DX_T);
  // the grid's y axis holds 65,535 blocks: longer token axes go in several launches
  for (int64_t r0 = 0; r0 < rows; r0 += 65535) {
    RouterGradArgs b = a;
    const int64_t skip = r0 * DX_T;
    b.T = a.T - skip;
    b.dlogit = a.dlogit + skip * a.ld;
    b.dx_in = a.dx_in ? static_cast<const float*>(a.dx_in) + skip * a.H : nullptr;
    b.dx = static_cast<float*>(a.dx) + skip * a.H;
    const int64_t n = rows - r0 < 65535 ? rows - r0 : 65535;
    if (b.T > n * DX_T) b.T = n * DX_T;
    router_grad_x_kernel<<<dim3((unsigned)ceil_div(a.H, DX_H), (unsigned)n), 256, 0, st>>>(b);
    USAF_CHECK_LAUNCH();
  }
  return USAF_OK;
}

}  // namespace

void router_grad_ws_layout(int64_t T, int64_t E, int64_t H, usaf_dtype dt, Carver& c,
                           RouterGradWs& w) {
  if (dt == USAF_BF16) {
    router_grad_tc_layout(T, E, H, c, w);
    return;
  }
  const int64_t s = splits_for(T, E, H);
  w.g_part = c.take<float>(s > 1 ? s * E * H : 1);
}

usaf_status router_grad_launch(const RouterGradArgs& a, const RouterGradWs& w, cudaStream_t st) {
  if (a.dt == USAF_BF16) return router_grad_tc(a, w, st);
  if (a.g_router) USAF_TRY(launch_w(a, w.g_part, st));
  return a.dx ? launch_x(a, st) : USAF_OK;
}

}  // namespace usaf
