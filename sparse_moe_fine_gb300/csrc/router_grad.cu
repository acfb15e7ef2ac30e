// The two products of a dense router gradient (usaf_router_grad): g_router = g_in + dlogit^T x and
// dx = dx_in + dlogit w_router. Here for fp32 tokens, on CUDA cores in fp32; bf16 tokens are in
// router_grad_tc.cu.
//
// Both are C[m, n] += sum_k A[k or m, ...] B[k, n] over 64 x 64 tiles of C, 16 values a thread, in
// steps of 32 along the contraction: each step's products are summed on their own before they join
// the total, which keeps the chains of dependent roundings short. The products do not depend on one
// another, so one launch holds the tiles of both; small layers are bound by launches. Where
// g_router's tiles are too few for the SMs, the tokens are split into stretches whose sums a second
// launch adds in their order.
#include "train.cuh"

namespace usaf {

namespace {

constexpr int TILE = 64;
constexpr int STEP = 32;
constexpr int THREADS = 256;

struct Shared {
  float a[STEP][TILE + 4];  // [k][m]
  float b[STEP][TILE];      // [k][n]
};

// acc[u][v] += sum over k0 <= k < k1 of A(k, m0 + 4 ty + u) B(k, n0 + 4 tx + v). a_at(k, j) is A's j-th
// value of the step that starts at k, as the thread that stores it at a_slot(j) reads it; b_row(k) is
// B's row. The next step's values are on their way in registers while one is multiplied.
template <class AAt, class ASlot, class BRow>
__device__ __forceinline__ void tile_product(Shared& s, int64_t k0, int64_t k1, int64_t n0,
                                             int64_t N, AAt a_at, ASlot a_slot, BRow b_row,
                                             float (&acc)[4][4]) {
  constexpr int PER = STEP * TILE / THREADS;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int bc = threadIdx.x % TILE, br = threadIdx.x / TILE;  // B: rows br, br + 4, ...
  float ra[PER], rb[PER];
  auto load = [&](int64_t k) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      ra[i] = a_at(k, threadIdx.x + i * THREADS);
      const int64_t r = k + br + i * (THREADS / TILE);
      rb[i] = r < k1 && n0 + bc < N ? __ldg(b_row(r) + n0 + bc) : 0.f;
    }
  };
  load(k0);
  for (int64_t k = k0; k < k1; k += STEP) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      *a_slot(threadIdx.x + i * THREADS) = ra[i];
      s.b[br + i * (THREADS / TILE)][bc] = rb[i];
    }
    __syncthreads();
    if (k + STEP < k1) load(k + STEP);
    float part[4][4] = {};
#pragma unroll 8
    for (int r = 0; r < STEP; ++r) {
      const float4 av = *reinterpret_cast<const float4*>(&s.a[r][ty * 4]);
      const float4 bv = *reinterpret_cast<const float4*>(&s.b[r][tx * 4]);
      const float a4[4] = {av.x, av.y, av.z, av.w}, b4[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int v = 0; v < 4; ++v) part[u][v] = fmaf(a4[u], b4[v], part[u][v]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[u][v] += part[u][v];
    __syncthreads();
  }
}

// Blocks [0, w_blocks): tiles of g_router by stretches of `per` tokens; the rest: tiles of dx.
__global__ void __launch_bounds__(THREADS)
    router_grad_f32_kernel(const RouterGradArgs a, int64_t w_blocks, int64_t splits, int64_t per,
                           float* __restrict__ part) {
  __shared__ __align__(16) Shared s;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int64_t htiles = (a.H + TILE - 1) / TILE, etiles = (a.E + TILE - 1) / TILE;
  float acc[4][4] = {};
  bool bad = false;
  dep_launch();
  if (blockIdx.x < w_blocks) {
    const int64_t sp = blockIdx.x / (htiles * etiles), i = blockIdx.x - sp * htiles * etiles;
    const int64_t e0 = i / htiles * TILE, h0 = i % htiles * TILE;
    const int64_t t0 = sp * per, t1 = min(a.T, t0 + per);
    const float* x = static_cast<const float*>(a.x);
    tile_product(
        s, t0, t1, h0, a.H,
        // dlogit's rows are the contraction's: experts next to one another
        [&](int64_t k, int j) {
          const int64_t t = k + j / TILE, e = e0 + j % TILE;
          return t < t1 && e < a.E ? __ldg(a.dlogit + t * a.ld + e) : 0.f;
        },
        [&](int j) { return &s.a[j / TILE][j % TILE]; },
        [&](int64_t k) { return x + k * a.H; }, acc);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t e = e0 + ty * 4 + u, h = h0 + tx * 4 + v;
        if (e >= a.E || h >= a.H) continue;
        const int64_t o = e * a.H + h;
        if (splits > 1) {
          part[sp * a.E * a.H + o] = acc[u][v];
        } else {
          const float r = (a.g_in ? a.g_in[o] : 0.f) + acc[u][v];
          a.g_router[o] = r;
          bad |= !finite_f(r);
        }
      }
  } else {
    const int64_t i = blockIdx.x - w_blocks;
    const int64_t t0 = i / htiles * TILE, h0 = i % htiles * TILE;
    tile_product(
        s, 0, a.E, h0, a.H,
        // dlogit's columns are the contraction's: turned on the way in
        [&](int64_t k, int j) {
          const int64_t t = t0 + j / STEP, e = k + j % STEP;
          return t < a.T && e < a.E ? __ldg(a.dlogit + t * a.ld + e) : 0.f;
        },
        [&](int j) { return &s.a[j % STEP][j / STEP]; },
        [&](int64_t k) { return a.w_router + k * a.H; }, acc);
    const float* dx_in = static_cast<const float*>(a.dx_in);
    float* dx = static_cast<float*>(a.dx);
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int64_t t = t0 + ty * 4 + u, h = h0 + tx * 4 + v;
        if (t >= a.T || h >= a.H) continue;
        const int64_t o = t * a.H + h;
        const float r = (dx_in ? dx_in[o] : 0.f) + acc[u][v];
        dx[o] = r;
        bad |= !finite_f(r);
      }
  }
  flag_status_warp(a.status, bad, USAF_DEV_NONFINITE);
}

// g_router = g_in + the stretches' sums in their order
__global__ void __launch_bounds__(THREADS)
    router_grad_reduce_kernel(const RouterGradArgs a, const float* __restrict__ part, int splits) {
  dep_wait();
  const int64_t n = a.E * a.H;
  bool bad = false;
  for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < n;
       i += (int64_t)gridDim.x * THREADS) {
    float v = 0.f;
#pragma unroll 8
    for (int s = 0; s < splits; ++s) v += __ldcg(part + s * n + i);
    if (a.g_in) v += a.g_in[i];
    a.g_router[i] = v;
    bad |= !finite_f(v);
  }
  flag_status_warp(a.status, bad, USAF_DEV_NONFINITE);
}

// Stretches of the token axis: about two blocks per SM, at least 128 tokens each (a shorter one
// costs less than the launch that would add it).
int64_t stretch_f32(int64_t T, int64_t E, int64_t H) {
  const int64_t tiles = ceil_div(E, TILE) * ceil_div(H, TILE);
  int64_t s = ceil_div(2 * 152, tiles);
  const int64_t most = ceil_div(T, 128);
  if (s > most) s = most;
  return round_up(ceil_div(T, s), STEP);
}

}  // namespace

void router_grad_ws_layout(int64_t T, int64_t E, int64_t H, usaf_dtype dt, Carver& c,
                           RouterGradWs& w) {
  if (dt == USAF_BF16) {
    router_grad_tc_layout(T, E, H, c, w);
    return;
  }
  const int64_t s = ceil_div(T, stretch_f32(T, E, H));
  w.g_part = c.take<float>(s > 1 ? s * E * H : 1);
}

usaf_status router_grad_launch(const RouterGradArgs& a, const RouterGradWs& w, cudaStream_t st) {
  if (a.dt == USAF_BF16) return router_grad_tc(a, w, st);
  const int64_t per = stretch_f32(a.T, a.E, a.H), splits = ceil_div(a.T, per);
  const int64_t htiles = ceil_div(a.H, TILE);
  const int64_t wb = a.g_router ? htiles * ceil_div(a.E, TILE) * splits : 0;
  const int64_t xb = a.dx ? htiles * ceil_div(a.T, TILE) : 0;
  if (wb + xb >= (int64_t(1) << 31)) return USAF_ERR_UNSUPPORTED;
  {
    USAF_TRACE("router_grad_f32", st);
    router_grad_f32_kernel<<<(unsigned)(wb + xb), THREADS, 0, st>>>(a, wb, splits, per, w.g_part);
    USAF_CHECK_LAUNCH();
  }
  if (!a.g_router || splits == 1) return USAF_OK;
  USAF_TRACE("router_grad_reduce", st);
  return launch_dep(router_grad_reduce_kernel, dim3(grid_dim_for(a.E * a.H)), THREADS, 0, st, a,
                    (const float*)w.g_part, (int)splits);
}

}  // namespace usaf
