// Load-balance loss, z-loss and per-expert counts of a router's logits, and their gradient
// (usaf_router_aux_fwd / _bwd). Softmax statistics and sums are fp32, counts integers.
//
// A row of E logits is held by LPR neighbouring lanes, NV values each (expert sub + LPR i), so a
// softmax is one read of the row, two butterflies and no shared memory; routers of at most 16
// experts put several rows into a warp.
#include <cooperative_groups.h>

#include <type_traits>

#include "train.cuh"

namespace usaf {

namespace {

constexpr int AUX_WARPS = 8;
constexpr int AUX_THREADS = 32 * AUX_WARPS;
constexpr int FIN_CTAS = 8;
constexpr int FIN_THREADS = 512;

struct AuxParams {
  int64_t T, ld;
  int E, k, G;
  int chunk, nchunks;
  const float* logits;
  const int32_t* topk;
  const uint8_t* mask;
  const int32_t* off;
  float share;          // E / k
  float coef_b, coef_z;
  uint32_t* status;
};

__device__ __forceinline__ int64_t clamp_off(const AuxParams& p, int g) {
  if (!p.off) return g == 0 ? 0 : p.T;
  const int64_t o = p.off[g];
  return o < 0 ? 0 : (o > p.T ? p.T : o);
}

// The group of token t (off[g] <= t < off[g + 1]), or -1.
__device__ __forceinline__ int group_of(const AuxParams& p, int64_t t) {
  if (!p.off) return 0;
  int lo = 0, hi = p.G + 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (clamp_off(p, mid) <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo - 1 < p.G ? lo - 1 : -1;
}

__device__ __forceinline__ void check_offsets(const AuxParams& p, int64_t i0, int64_t stride) {
  if (!p.off) return;
  bool bad = false;
  for (int64_t i = i0; i <= p.G; i += stride) {
    const int o = p.off[i];
    bad |= o < 0 || o > p.T || (i < p.G && p.off[i + 1] < o);
  }
  if (bad) flag_status(p.status, USAF_DEV_BAD_INDEX);
}

template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int LPR>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = LPR / 2; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// Softmax of one row from its logits v (-inf where there is no expert): v becomes the
// probabilities, lse the log of the sum. False (all probabilities 0) where every logit is -inf;
// a NaN or +inf makes every probability NaN. All lanes of the warp call it.
template <int LPR, int NV>
__device__ __forceinline__ bool row_softmax(float (&v)[NV], float& lse) {
  float mx = -INFINITY;
  bool some = false;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    mx = fmaxf(mx, v[i]);
    some |= !(v[i] == -INFINITY);
  }
  mx = row_max<LPR>(mx);
  const unsigned b = __ballot_sync(0xffffffffu, some);
  const int lane = threadIdx.x & 31;
  const unsigned rowbits = LPR == 32 ? 0xffffffffu : (((1u << (LPR & 31)) - 1u) << (lane & ~(LPR - 1)));
  const bool alive = (b & rowbits) != 0;
  const float m = alive ? mx : 0.f;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    v[i] = expf(v[i] - m);
    s += v[i];
  }
  s = row_sum<LPR>(s);
  const float inv = alive ? 1.f / s : 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] *= inv;
  lse = alive ? m + logf(s) : 0.f;
  return alive;
}

template <int LPR, int NV>
__device__ __forceinline__ void load_row(const AuxParams& p, int64_t t, bool in, int sub,
                                         float (&v)[NV]) {
  const float* row = p.logits + t * p.ld;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = sub + LPR * i;
    v[i] = in && e < p.E ? row[e] : -INFINITY;
  }
}

__device__ __forceinline__ void write_loss(const AuxParams& p, double bal, double z, int64_t n,
                                           float* loss) {
  const double inv = n > 0 ? 1.0 / (double)n : 0.0;
  const float b = n > 0 ? (float)((double)p.share * inv * bal) : 0.f;
  const float zz = n > 0 ? (float)(inv * z) : 0.f;
  const float tot = (p.coef_b != 0.f ? p.coef_b * b : 0.f) + (p.coef_z != 0.f ? p.coef_z * zz : 0.f);
  loss[0] = tot;
  loss[1] = b;
  loss[2] = zz;
  if (!finite_f(b) || !finite_f(zz)) flag_status(p.status, USAF_DEV_NONFINITE);
}

// One block per chunk of tokens. Per (chunk, group) that meet: the warps' rows are summed in
// registers, then over rows of a warp and over the warps in a fixed order.
// ONE: the only chunk; the block also forms the outputs and the loss (one launch).
template <int LPR, int NV, bool ONE>
__global__ void __launch_bounds__(AUX_THREADS)
    aux_part_kernel(const AuxParams p, AuxWs w, int32_t* __restrict__ count_out,
                    float* __restrict__ prob_out, int32_t* __restrict__ n_out,
                    float* __restrict__ loss) {
  extern __shared__ float sm[];
  float* s_prob = sm;                                                   // [AUX_WARPS][E]
  int32_t* s_cnt = reinterpret_cast<int32_t*>(sm + AUX_WARPS * p.E);    // [E]
  uint8_t* s_live = reinterpret_cast<uint8_t*>(s_cnt + p.E);            // [chunk]
  __shared__ float s_z[AUX_WARPS];
  __shared__ int s_n[AUX_WARPS];
  __shared__ double s_red[AUX_THREADS];
  constexpr int RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int sub = lane % LPR, rw = lane / LPR;
  const int64_t t0 = (int64_t)blockIdx.x * p.chunk, t1 = min(p.T, t0 + p.chunk);
  check_offsets(p, (int64_t)blockIdx.x * blockDim.x + threadIdx.x,
                (int64_t)gridDim.x * blockDim.x);
  for (int e = threadIdx.x; e < p.E; e += AUX_THREADS) s_cnt[e] = 0;
  if constexpr (ONE) {
    for (int64_t i = threadIdx.x; i < (int64_t)p.G * p.E; i += AUX_THREADS) {
      count_out[i] = 0;
      prob_out[i] = 0.f;
    }
    for (int i = threadIdx.x; i < p.G; i += AUX_THREADS) n_out[i] = 0;
  }
  double bal_all = 0.0, z_all = 0.0;  // ONE: of this thread's experts / of thread 0
  int64_t n_all = 0;
  bool badidx = false;
  int64_t t = t0;
  while (t < t1) {
    const int g = group_of(p, t);
    if (g < 0) {  // before the first group or behind the last
      const int64_t f = clamp_off(p, 0);
      t = f > t ? f : t1;
      continue;
    }
    int64_t te = min(t1, clamp_off(p, g + 1));
    if (te <= t) te = t + 1;  // only where the offsets decrease
    __syncthreads();  // the last segment's counts are out; ONE: the zeroed outputs too
    float acc[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) acc[i] = 0.f;
    float z = 0.f;
    int n = 0;
    for (int64_t base = t + wid * RPW; base < te; base += AUX_WARPS * RPW) {
      const int64_t tok = base + rw;
      const bool in = tok < te && (!p.mask || p.mask[tok] != 0);
      float v[NV], lse;
      load_row<LPR, NV>(p, tok, in, sub, v);
      const bool alive = row_softmax<LPR, NV>(v, lse);
#pragma unroll
      for (int i = 0; i < NV; ++i) acc[i] += v[i];
      if (sub == 0) {
        z += lse * lse;
        n += alive ? 1 : 0;
        if (tok < te) s_live[tok - t0] = alive ? 1 : 0;
      }
    }
#pragma unroll
    for (int o = 16; o >= LPR; o >>= 1)
#pragma unroll
      for (int i = 0; i < NV; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    z = row_sum<32>(z);
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    if (rw == 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = sub + LPR * i;
        if (e < p.E) s_prob[wid * p.E + e] = acc[i];
      }
    }
    if (lane == 0) {
      s_z[wid] = z;
      s_n[wid] = n;
    }
    __syncthreads();
    // the experts that the segment's live tokens went to
    const int64_t q1 = te * p.k;
    for (int64_t q = t * p.k + threadIdx.x; q < q1; q += AUX_THREADS) {
      if (!s_live[q / p.k - t0]) continue;
      const int e = p.topk[q];
      if (e >= 0 && e < p.E) atomicAdd(&s_cnt[e], 1);
      else badidx = true;
    }
    __syncthreads();
    const int64_t slot = ONE ? g : (int64_t)blockIdx.x + g;
    float* po = ONE ? prob_out : w.prob;
    int32_t* co = ONE ? count_out : w.count;
    int ng = 0;
#pragma unroll
    for (int u = 0; u < AUX_WARPS; ++u) ng += s_n[u];
    for (int e = threadIdx.x; e < p.E; e += AUX_THREADS) {
      float s = 0.f;
#pragma unroll
      for (int u = 0; u < AUX_WARPS; ++u) s += s_prob[u * p.E + e];
      const int c = s_cnt[e];
      s_cnt[e] = 0;
      po[slot * p.E + e] = s;
      co[slot * p.E + e] = c;
      if (ONE && ng > 0) bal_all += (double)((float)c * s) / ng;
    }
    if (threadIdx.x == 0) {
      float s = 0.f;
#pragma unroll
      for (int u = 0; u < AUX_WARPS; ++u) s += s_z[u];
      if constexpr (ONE) {
        n_out[g] = ng;
        n_all += ng;
        z_all += s;
      } else {
        w.n[slot] = ng;
        w.z[slot] = s;
      }
    }
    t = te;
  }
  if (badidx) flag_status(p.status, USAF_DEV_BAD_INDEX);
  if constexpr (ONE) {
    s_red[threadIdx.x] = bal_all;
    __syncthreads();
    for (int h = AUX_THREADS / 2; h; h >>= 1) {
      if (threadIdx.x < h) s_red[threadIdx.x] += s_red[threadIdx.x + h];
      __syncthreads();
    }
    if (threadIdx.x == 0) write_loss(p, s_red[0], z_all, n_all, loss);
  }
}

// Sums the chunks' partials into the groups' outputs and forms the loss: one cluster, CTA r the
// experts [r w, (r + 1) w), w = ceil(E / FIN_CTAS). A CTA's threads are (group lane, slot lane, expert): `sl`
// slot lanes share a group's chunks and are added by a tree.
__global__ void __cluster_dims__(FIN_CTAS, 1, 1) __launch_bounds__(FIN_THREADS)
    aux_final_kernel(const AuxParams p, AuxWs w, int el, int sl, int32_t* __restrict__ count,
                     float* __restrict__ prob, int32_t* __restrict__ n_tok,
                     float* __restrict__ loss) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  __shared__ float s_p[FIN_THREADS], s_z[FIN_THREADS];
  __shared__ int32_t s_c[FIN_THREADS], s_n[FIN_THREADS];
  __shared__ double s_bal;
  const int rank = (int)cluster.block_rank();
  const int tx = threadIdx.x % el, ty = threadIdx.x / el;
  const int ls = ty % sl, lg = ty / sl, gl = FIN_THREADS / el / sl;
  const int wd = (p.E + FIN_CTAS - 1) / FIN_CTAS;
  const int e = rank * wd + tx;
  const bool ev = tx < wd && e < p.E;
  double bal = 0.0;
  float z = 0.f;
  int64_t n_all = 0;
  for (int g0 = 0; g0 < p.G; g0 += gl) {
    const int g = g0 + lg;
    float a = 0.f, zz = 0.f;
    int32_t c = 0, n = 0;
    if (g < p.G) {
      const int64_t o0 = clamp_off(p, g), o1 = clamp_off(p, g + 1);
      if (o1 > o0) {
        const int64_t c1 = (o1 - 1) / p.chunk;
        for (int64_t ch = o0 / p.chunk + ls; ch <= c1; ch += sl) {
          const int64_t slot = ch + g;
          if (ev) {
            a += w.prob[slot * p.E + e];
            c += w.count[slot * p.E + e];
          }
          if (tx == 0) {
            n += w.n[slot];
            zz += w.z[slot];
          }
        }
      }
    }
    s_p[threadIdx.x] = a;
    s_c[threadIdx.x] = c;
    s_n[threadIdx.x] = n;
    s_z[threadIdx.x] = zz;
    __syncthreads();
    for (int h = sl / 2; h; h >>= 1) {
      if (ls < h) {
        s_p[threadIdx.x] += s_p[threadIdx.x + h * el];
        s_c[threadIdx.x] += s_c[threadIdx.x + h * el];
        s_n[threadIdx.x] += s_n[threadIdx.x + h * el];
        s_z[threadIdx.x] += s_z[threadIdx.x + h * el];
      }
      __syncthreads();
    }
    if (ls == 0 && g < p.G) {
      const int ng = s_n[threadIdx.x - tx];
      if (ev) {
        const float P = s_p[threadIdx.x];
        const int32_t cc = s_c[threadIdx.x];
        prob[(int64_t)g * p.E + e] = P;
        count[(int64_t)g * p.E + e] = cc;
        if (ng > 0) bal += (double)((float)cc * P) / ng;
      }
      if (tx == 0) {
        z += s_z[threadIdx.x];
        n_all += ng;
        if (rank == 0) n_tok[g] = ng;
      }
    }
    __syncthreads();
  }
  // the block's sums in a fixed order: warps by butterfly, then the warps in turn
  for (int o = 16; o; o >>= 1) {
    bal += __shfl_xor_sync(0xffffffffu, bal, o);
    z += __shfl_xor_sync(0xffffffffu, z, o);
    n_all += __shfl_xor_sync(0xffffffffu, n_all, o);
  }
  __shared__ double r_bal[FIN_THREADS / 32];
  __shared__ float r_z[FIN_THREADS / 32];
  __shared__ int64_t r_n[FIN_THREADS / 32];
  if ((threadIdx.x & 31) == 0) {
    r_bal[threadIdx.x >> 5] = bal;
    r_z[threadIdx.x >> 5] = z;
    r_n[threadIdx.x >> 5] = n_all;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double b = 0.0;
    for (int i = 0; i < FIN_THREADS / 32; ++i) b += r_bal[i];
    s_bal = b;
  }
  cluster.sync();
  if (rank == 0 && threadIdx.x == 0) {
    double b = 0.0, zs = 0.0;
    int64_t n = 0;
    for (int r = 0; r < FIN_CTAS; ++r) b += *cluster.map_shared_rank(&s_bal, r);
    for (int i = 0; i < FIN_THREADS / 32; ++i) {
      zs += r_z[i];
      n += r_n[i];
    }
    write_loss(p, b, zs, n, loss);
  }
  cluster.sync();  // no CTA leaves while its shared memory may be read
}

// The gradient: each row is read once, its group's counts stay in registers while the group lasts.
template <int LPR, int NV>
__global__ void __launch_bounds__(AUX_THREADS)
    aux_bwd_kernel(const AuxParams p, const int32_t* __restrict__ count,
                   const int32_t* __restrict__ n_tok, const float* __restrict__ d_loss, float* out,
                   int64_t ld_out, int accumulate, int rows_per_lane) {
  __shared__ int64_t s_n[AUX_WARPS];
  constexpr int RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int sub = lane % LPR, rw = lane / LPR;
  check_offsets(p, (int64_t)blockIdx.x * blockDim.x + threadIdx.x,
                (int64_t)gridDim.x * blockDim.x);
  int64_t n = 0;
  for (int i = threadIdx.x; i < p.G; i += AUX_THREADS) n += n_tok[i];
  for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  if (lane == 0) s_n[wid] = n;
  __syncthreads();
  n = 0;
#pragma unroll
  for (int u = 0; u < AUX_WARPS; ++u) n += s_n[u];
  const float up = d_loss ? *d_loss : 1.f;
  const float inv_n = n > 0 ? 1.f / (float)n : 0.f;
  const float zc = p.coef_z != 0.f ? up * 2.f * p.coef_z * inv_n : 0.f;
  const int64_t first = ((int64_t)blockIdx.x * AUX_WARPS + wid) * RPW * rows_per_lane;
  int cur = -2;       // group whose counts are in c
  int64_t cur_end = 0;
  float c[NV], cg = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) c[i] = 0.f;
  bool bad = false;
  for (int r = 0; r < rows_per_lane; ++r) {
    if (first + r * RPW >= p.T) break;
    const int64_t tok = first + r * RPW + rw;
    bool in = tok < p.T;
    if (in && (cur == -2 || tok >= cur_end)) {
      cur = group_of(p, tok);
      cur_end = cur >= 0 ? clamp_off(p, cur + 1) : (tok < clamp_off(p, 0) ? clamp_off(p, 0) : p.T);
      const int ng = cur >= 0 ? n_tok[cur] : 0;
      cg = p.coef_b != 0.f && ng > 0 ? up * p.coef_b * p.share * inv_n / (float)ng : 0.f;
      if (cur >= 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int e = sub + LPR * i;
          c[i] = e < p.E ? (float)count[(int64_t)cur * p.E + e] : 0.f;
        }
      }
    }
    const bool row_in = in && cur >= 0 && (!p.mask || p.mask[tok] != 0);
    float v[NV], lse;
    load_row<LPR, NV>(p, tok, row_in, sub, v);
    row_softmax<LPR, NV>(v, lse);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) s = fmaf(v[i], c[i], s);
    s = row_sum<LPR>(s);
    const float zt = zc * lse;
    if (in) {
      float* o = out + tok * ld_out;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = sub + LPR * i;
        if (e < p.E) {
          float d = v[i] * fmaf(cg, c[i] - s, zt);
          if (accumulate) d += o[e];
          o[e] = d;
          bad |= !finite_f(d);
        }
      }
    }
  }
  flag_status_warp(p.status, bad, USAF_DEV_NONFINITE);
}

AuxParams make_params(const AuxArgs& a) {
  AuxParams p{};
  p.T = a.T;
  p.ld = a.ld;
  p.E = a.E;
  p.k = a.k;
  p.G = (int)a.G;
  p.chunk = (int)aux_chunk_tokens(a.T);
  p.nchunks = (int)ceil_div(a.T, p.chunk);
  p.logits = a.logits;
  p.topk = a.topk_idx;
  p.mask = a.mask;
  p.off = a.offset;
  p.share = (float)((double)a.E / (double)a.k);
  p.coef_b = (float)a.coef_balance;
  p.coef_z = (float)a.coef_z;
  p.status = a.status;
  return p;
}

// Calls f with the lanes per row and values per lane of E experts.
template <class F>
usaf_status by_width(int E, F f) {
  using std::integral_constant;
#define USAF_W(L, N) f(integral_constant<int, L>(), integral_constant<int, N>())
  if (E <= 8) return USAF_W(8, 1);
  if (E <= 16) return USAF_W(16, 1);
  if (E <= 32) return USAF_W(32, 1);
  if (E <= 64) return USAF_W(32, 2);
  if (E <= 128) return USAF_W(32, 4);
  if (E <= 256) return USAF_W(32, 8);
  if (E <= 512) return USAF_W(32, 16);
  return USAF_W(32, 32);
#undef USAF_W
}

}  // namespace

// Tokens of a chunk: eight warps of the block that owns it, at most about two chunks per SM.
int64_t aux_chunk_tokens(int64_t T) {
  const int64_t per = ceil_div(T, 2 * 152);
  const int64_t c = round_up(per, 32);
  return c < 32 ? 32 : c;
}

void aux_ws_layout(int64_t T, int64_t E, int64_t G, Carver& c, AuxWs& w) {
  const int64_t slots = ceil_div(T, aux_chunk_tokens(T)) + G - 1;
  w.prob = c.take<float>(slots * E);
  w.count = c.take<int32_t>(slots * E);
  w.n = c.take<int32_t>(slots);
  w.z = c.take<float>(slots);
}

usaf_status aux_fwd_launch(const AuxArgs& a, int32_t* count, float* prob_sum, int32_t* n_tok,
                           float* loss, const AuxWs& w, cudaStream_t st) {
  const AuxParams p = make_params(a);
  const size_t smem = (size_t)(AUX_WARPS + 1) * a.E * 4 + p.chunk;
  const bool one = p.nchunks == 1;
  USAF_TRY(by_width(a.E, [&](auto lpr, auto nv) {
    USAF_TRACE("router_aux_part", st);
    auto go = [&](auto kernel) {
      if (smem > 48 * 1024 &&
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
              cudaSuccess)
        return USAF_ERR_CUDA;
      kernel<<<p.nchunks, AUX_THREADS, smem, st>>>(p, w, count, prob_sum, n_tok, loss);
      USAF_CHECK_LAUNCH();
      return USAF_OK;
    };
    return one ? go(aux_part_kernel<lpr.value, nv.value, true>)
               : go(aux_part_kernel<lpr.value, nv.value, false>);
  }));
  if (one) return USAF_OK;
  USAF_TRACE("router_aux_final", st);
  const int wd = (a.E + FIN_CTAS - 1) / FIN_CTAS;
  int el = 1;
  while (el < wd) el *= 2;
  int sl = 1;
  const int64_t per_group = ceil_div(p.nchunks, a.G) + 1;
  while (sl * 2 <= FIN_THREADS / el && sl < per_group) sl *= 2;
  aux_final_kernel<<<FIN_CTAS, FIN_THREADS, 0, st>>>(p, w, el, sl, count, prob_sum, n_tok, loss);
  USAF_CHECK_LAUNCH();
  return USAF_OK;
}

usaf_status aux_bwd_launch(const AuxArgs& a, const int32_t* count, const int32_t* n_tok,
                           const float* d_loss, float* dlogit, int64_t ld_out, int accumulate,
                           cudaStream_t st) {
  const AuxParams p = make_params(a);
  USAF_TRACE("router_aux_bwd", st);
  return by_width(a.E, [&](auto lpr, auto nv) {
    constexpr int RPW = 32 / lpr.value;
    // rows per lane group: enough blocks for every SM first, then rows that share a count load
    const int64_t lanes = (int64_t)AUX_WARPS * RPW;
    int rows = 1;
    while (rows < 8 && ceil_div(a.T, lanes * rows * 2) >= 4 * 152) rows *= 2;
    const unsigned grid = (unsigned)ceil_div(a.T, lanes * rows);
    aux_bwd_kernel<lpr.value, nv.value><<<grid, AUX_THREADS, 0, st>>>(
        p, count, n_tok, d_loss, dlogit, ld_out, accumulate, rows);
    USAF_CHECK_LAUNCH();
    return USAF_OK;
  });
}

}  // namespace usaf
