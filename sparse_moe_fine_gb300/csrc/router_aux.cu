// Load-balance loss, z-loss and per-expert counts of a router's logits, and their gradient
// (usaf_router_aux_fwd / _bwd). Softmax statistics and sums are fp32, counts integers.
//
// A row of E logits is held by LPR neighbouring lanes, NV values each, so a softmax is one read of
// the row, two butterflies and no shared memory. Few lanes with many values beat the other way round:
// a butterfly step costs the same for every lane of the warp, so four rows of eight lanes share what
// one row of 32 would pay alone (and have two steps fewer). Only routers of more than 128 experts
// use more lanes.
//
// A forward reads the logits once (2 MB for 4,096 tokens of 128 experts, 0.3 us of DRAM time), so the
// calls are bound by launches and by the latency of one round to memory: forward and backward
// together 14 us for 128 tokens of 8 experts (two launches; the host takes as long to issue them),
// 17 us for 4,096 of 128 (three), 26 us for 16,383 masked tokens of 128 in 37 packed sequences.
#include <type_traits>

#include "train.cuh"

namespace usaf {

namespace {

constexpr int AUX_WARPS = 8;
constexpr int AUX_THREADS = 32 * AUX_WARPS;
constexpr int FIN_WARPS = 32;
constexpr int FIN_THREADS = 32 * FIN_WARPS;
// Rows that a lane has in flight: 16 values at most.
template <int NV>
constexpr int ROWS = NV <= 4 ? 4 : (NV <= 8 ? 2 : 1);
constexpr int MAX_CHUNK = 4096;  // a token's flag is a byte of shared memory
// Blocks of an SM: four (64 registers a thread) hold the chunks of 16,383 tokens in one wave, where
// the compiler's own choice needs two (28.7 -> 26.7 us); 32 values a lane need the registers.
template <int NV>
constexpr int BLOCKS = NV <= 16 ? 4 : 2;
// The expert of a lane's i-th value: four neighbours at a time, whether or not the rows' alignment
// lets them be read as one vector, so that sums have one order and results do not depend on strides.
template <int LPR, int NV>
__device__ __forceinline__ int expert(int sub, int i) {
  return NV >= 4 ? 4 * (sub + LPR * (i / 4)) + i % 4 : sub + LPR * i;
}

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

// The group offsets as a kernel looks them up: in shared memory where they fit (a binary search is
// then a few cycles a step instead of a cache miss a step), else in place.
constexpr int OFF_CAP = 1024;
struct Groups {
  const AuxParams& p;
  const int32_t* s_off;
  // fills s_off (all threads of the block, a barrier before its use) and checks its share
  __device__ __forceinline__ Groups(const AuxParams& p_, int32_t* s) : p(p_), s_off(s) {
    if (!p.off) return;
    bool bad = false;
    if (p.G < OFF_CAP) {
      for (int i = threadIdx.x; i <= p.G; i += blockDim.x) {
        const int o = p.off[i];
        bad |= o < 0 || o > p.T || (i < p.G && p.off[i + 1] < o);
        s[i] = o < 0 ? 0 : (o > p.T ? (int32_t)p.T : o);
      }
    } else {
      for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i <= p.G;
           i += (int64_t)gridDim.x * blockDim.x) {
        const int o = p.off[i];
        bad |= o < 0 || o > p.T || (i < p.G && p.off[i + 1] < o);
      }
    }
    if (bad) flag_status(p.status, USAF_DEV_BAD_INDEX);
  }
  __device__ __forceinline__ int64_t at(int g) const {
    if (!p.off) return g == 0 ? 0 : p.T;
    return p.G < OFF_CAP ? s_off[g] : clamp_off(p, g);
  }
  // the group of token t (at(g) <= t < at(g + 1)), or -1
  __device__ __forceinline__ int of(int64_t t) const {
    if (!p.off) return 0;
    int lo = 0, hi = p.G + 1;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (at(mid) <= t) lo = mid + 1;
      else hi = mid;
    }
    return lo - 1 < p.G ? lo - 1 : -1;
  }
  // the first group that ends after token t, G if none does
  __device__ __forceinline__ int first_ending_after(int64_t t) const {
    int lo = 0, hi = p.G;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (at(mid + 1) <= t) lo = mid + 1;
      else hi = mid;
    }
    return lo;
  }
  // the last group that starts before token t, -1 if none does
  __device__ __forceinline__ int last_starting_before(int64_t t) const {
    int lo = 0, hi = p.G;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (at(mid) < t) lo = mid + 1;
      else hi = mid;
    }
    return lo - 1;
  }
};

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

// The row of token t, -inf where there is none; the mask is read beside it, not before it.
// VEC: E and the row stride are multiples of four, the rows 16-byte aligned.
template <int LPR, int NV, bool VEC>
__device__ __forceinline__ void load_row(const AuxParams& p, int64_t t, bool in, int sub,
                                         float (&v)[NV]) {
  const float* row = p.logits + t * p.ld;
  const bool keep = !(p.mask && in) || p.mask[t] != 0;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < NV; i += 4) {
      const int e = expert<LPR, NV>(sub, i);
      const float4 f = in && e < p.E ? *reinterpret_cast<const float4*>(row + e)
                                     : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      v[i] = f.x, v[i + 1] = f.y, v[i + 2] = f.z, v[i + 3] = f.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = expert<LPR, NV>(sub, i);
      v[i] = in && e < p.E ? row[e] : -INFINITY;
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = keep ? v[i] : -INFINITY;
}

// The loss from the sums over groups and experts. fp32: the sums are of positive terms (a double
// costs this GPU 64 times a float, and a division in doubles was once a third of a small call).
__device__ __forceinline__ void write_loss(const AuxParams& p, float bal, float z, int64_t n,
                                           float* loss) {
  const float inv = n > 0 ? 1.f / (float)n : 0.f;
  const float b = n > 0 ? p.share * inv * bal : 0.f;
  const float zz = n > 0 ? inv * z : 0.f;
  const float tot = (p.coef_b != 0.f ? p.coef_b * b : 0.f) + (p.coef_z != 0.f ? p.coef_z * zz : 0.f);
  loss[0] = tot;
  loss[1] = b;
  loss[2] = zz;
  if (!finite_f(b) || !finite_f(zz)) flag_status(p.status, USAF_DEV_NONFINITE);
}

// One block per chunk of tokens; its sums go to a slot per group that the chunk meets. One or two
// groups: the block's warps share each group's rows, summed in registers, then over the rows of a
// warp and over the warps in a fixed order. More (short packed sequences): each warp takes groups of
// its own, so that no barrier stands between them.
// ONE: the only chunk; the block also forms the outputs and the loss (one launch).
template <int LPR, int NV, bool VEC, bool ONE>
__global__ void __launch_bounds__(AUX_THREADS, BLOCKS<NV>)
    aux_part_kernel(const AuxParams p, AuxWs w, int32_t* __restrict__ count_out,
                    float* __restrict__ prob_out, int32_t* __restrict__ n_out,
                    float* __restrict__ loss) {
  extern __shared__ float sm[];
  float* s_prob = sm;                                                   // [AUX_WARPS][E]
  int32_t* s_cnt = reinterpret_cast<int32_t*>(sm + AUX_WARPS * p.E);    // [E]
  uint8_t* s_live = reinterpret_cast<uint8_t*>(s_cnt + p.E);            // [chunk]
  __shared__ int32_t s_off[OFF_CAP];
  __shared__ float s_z[AUX_WARPS];
  __shared__ int s_n[AUX_WARPS];
  __shared__ float s_bal[AUX_WARPS], s_za[AUX_WARPS];
  __shared__ int64_t s_na[AUX_WARPS];
  constexpr int RPW = 32 / LPR, U = ROWS<NV>, PRE = 4;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int sub = lane % LPR, rw = lane / LPR;
  const int64_t t0 = (int64_t)blockIdx.x * p.chunk, t1 = min(p.T, t0 + p.chunk);
  dep_launch();
  const Groups groups(p, s_off);
  for (int e = threadIdx.x; e < p.E; e += AUX_THREADS) s_cnt[e] = 0;
  if (!ONE && blockIdx.x == 0 && threadIdx.x == 0) *w.arrived = 0;  // for the final kernel
  if constexpr (ONE) {
    for (int64_t i = threadIdx.x; i < (int64_t)p.G * p.E; i += AUX_THREADS) {
      count_out[i] = 0;
      prob_out[i] = 0.f;
    }
    for (int i = threadIdx.x; i < p.G; i += AUX_THREADS) n_out[i] = 0;
  }
  float bal_all = 0.f, z_all = 0.f;  // ONE: this thread's share of the loss
  int64_t n_all = 0;
  bool badidx = false;
  __syncthreads();
  const int g0 = groups.first_ending_after(t0), g1 = groups.last_starting_before(t1);
  const bool alone = g1 - g0 >= 2;  // a warp on its own takes a group

  // Rows base, base + step, ... below te: sums of this lane's experts, of the squared logsumexps and
  // of the tokens that take part, whose flags go to s_live.
  float acc[NV], z;
  int n;
  auto rows = [&](int64_t base, int64_t te, int step) {
#pragma unroll
    for (int i = 0; i < NV; ++i) acc[i] = 0.f;
    z = 0.f;
    n = 0;
    for (; base < te; base += step * U) {
      float v[U][NV];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t tok = base + u * step + rw;
        load_row<LPR, NV, VEC>(p, tok, tok < te, sub, v[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t tok = base + u * step + rw;
        float lse;
        const bool alive = row_softmax<LPR, NV>(v[u], lse);
#pragma unroll
        for (int i = 0; i < NV; ++i) acc[i] += v[u][i];
        if (sub == 0) {
          z += lse * lse;
          n += alive ? 1 : 0;
          if (tok < te) s_live[tok - t0] = alive ? 1 : 0;
        }
      }
    }
#pragma unroll
    for (int o = 16; o >= LPR; o >>= 1)
#pragma unroll
      for (int i = 0; i < NV; ++i) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
    z = row_sum<32>(z);
#pragma unroll
    for (int o = 16; o; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  };
  auto add = [&](int32_t* cnt, int64_t q, int e) {  // slot q went to expert e
    if (!s_live[(int)(q - t0 * p.k) / p.k]) return;
    if (e >= 0 && e < p.E) atomicAdd(&cnt[e], 1);
    else badidx = true;
  };
  float* po = ONE ? prob_out : w.prob;
  int32_t* co = ONE ? count_out : w.count;
  auto totals = [&](int g, int64_t slot, int ng, float zg) {
    if constexpr (ONE) {
      n_out[g] = ng;
      n_all += ng;
      z_all += zg;
    } else {
      w.n[slot] = ng;
      w.z[slot] = zg;
    }
  };

  if (alone) {
    int32_t* cnt = reinterpret_cast<int32_t*>(s_prob) + wid * p.E;
    for (int e = lane; e < p.E; e += 32) cnt[e] = 0;
    for (int g = g0 + wid; g <= g1; g += AUX_WARPS) {
      const int64_t t = max(t0, groups.at(g)), te = min(t1, groups.at(g + 1));
      if (te <= t) continue;
      const int64_t slot = ONE ? g : (int64_t)blockIdx.x + g;
      rows(t, te, RPW);
      __syncwarp();  // the flags are set, the counts clear
      for (int64_t q = t * p.k + lane; q < te * p.k; q += 32) add(cnt, q, p.topk[q]);
      __syncwarp();
      if (rw == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int e = expert<LPR, NV>(sub, i);
          if (e >= p.E) continue;
          const int c = cnt[e];
          cnt[e] = 0;
          po[slot * p.E + e] = acc[i];
          co[slot * p.E + e] = c;
          if (ONE && n > 0) bal_all += (float)c * acc[i] / (float)n;
        }
      }
      if (lane == 0) totals(g, slot, n, z);
      __syncwarp();
    }
  } else {
    for (int g = g0; g <= g1; ++g) {
      const int64_t t = max(t0, groups.at(g)), te = min(t1, groups.at(g + 1));
      if (te <= t) continue;
      const int64_t slot = ONE ? g : (int64_t)blockIdx.x + g;
      // the group's first expert indices, on their way while the rows are read
      const int64_t q0 = t * p.k + threadIdx.x, q1 = te * p.k;
      int ids[PRE];
#pragma unroll
      for (int u = 0; u < PRE; ++u)
        ids[u] = q0 + u * AUX_THREADS < q1 ? p.topk[q0 + u * AUX_THREADS] : 0;
      rows(t + wid * RPW, te, AUX_WARPS * RPW);
      if (rw == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int e = expert<LPR, NV>(sub, i);
          if (e < p.E) s_prob[wid * p.E + e] = acc[i];
        }
      }
      if (lane == 0) {
        s_z[wid] = z;
        s_n[wid] = n;
      }
      __syncthreads();
#pragma unroll
      for (int u = 0; u < PRE; ++u)
        if (q0 + u * AUX_THREADS < q1) add(s_cnt, q0 + u * AUX_THREADS, ids[u]);
      for (int64_t q = q0 + PRE * AUX_THREADS; q < q1; q += AUX_THREADS) add(s_cnt, q, p.topk[q]);
      __syncthreads();
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
        if (ONE && ng > 0) bal_all += (float)c * s / (float)ng;
      }
      if (threadIdx.x == 0) {
        float s = 0.f;
#pragma unroll
        for (int u = 0; u < AUX_WARPS; ++u) s += s_z[u];
        totals(g, slot, ng, s);
      }
      __syncthreads();  // the shared sums are read
    }
  }
  if (badidx) flag_status(p.status, USAF_DEV_BAD_INDEX);
  if constexpr (ONE) {
    for (int o = 16; o; o >>= 1) {
      bal_all += __shfl_xor_sync(0xffffffffu, bal_all, o);
      z_all += __shfl_xor_sync(0xffffffffu, z_all, o);
      n_all += __shfl_xor_sync(0xffffffffu, n_all, o);
    }
    if (lane == 0) {
      s_bal[wid] = bal_all;
      s_za[wid] = z_all;
      s_na[wid] = n_all;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int u = 1; u < AUX_WARPS; ++u) {
        bal_all += s_bal[u];
        z_all += s_za[u];
        n_all += s_na[u];
      }
      write_loss(p, bal_all, z_all, n_all, loss);
    }
  }
}

// Sums the chunks' partials of `el` experts of a group: threads are (slot lane, expert). Where there
// are several blocks, the one that arrives last (a counter that the partials' kernel cleared) adds the
// blocks' shares of the loss in their order.
__global__ void __launch_bounds__(FIN_THREADS)
    aux_final_kernel(const AuxParams p, AuxWs w, int el, int nb, int32_t* __restrict__ count,
                     float* __restrict__ prob, int32_t* __restrict__ n_tok,
                     float* __restrict__ loss) {
  __shared__ float s_p[FIN_THREADS], s_z[FIN_WARPS], s_b[FIN_WARPS];
  __shared__ int32_t s_c[FIN_THREADS], s_n[FIN_WARPS];
  __shared__ bool s_last;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int tx = threadIdx.x % el, ls = threadIdx.x / el, sl = FIN_THREADS / el;
  const int g = blockIdx.x / nb, eb = blockIdx.x % nb, e = eb * el + tx;
  float a = 0.f, z = 0.f;
  int32_t c = 0, n = 0;
  dep_launch();
  dep_wait();
  const int64_t o0 = clamp_off(p, g), o1 = clamp_off(p, g + 1);
  const int64_t ch0 = o0 / p.chunk, ch1 = o1 > o0 ? (o1 - 1) / p.chunk : ch0 - 1;
  if (e < p.E) {
    const float* pp = w.prob + (ch0 + ls + g) * p.E + e;
    const int32_t* pc = w.count + (ch0 + ls + g) * p.E + e;
#pragma unroll 8
    for (int64_t ch = ch0 + ls; ch <= ch1; ch += sl, pp += (int64_t)sl * p.E, pc += (int64_t)sl * p.E) {
      a += *pp;
      c += *pc;
    }
  }
  for (int64_t ch = ch0 + threadIdx.x; ch <= ch1; ch += FIN_THREADS) {
    n += w.n[ch + g];
    z += w.z[ch + g];
  }
  s_p[threadIdx.x] = a;
  s_c[threadIdx.x] = c;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    n += __shfl_xor_sync(0xffffffffu, n, o);
    z += __shfl_xor_sync(0xffffffffu, z, o);
  }
  if (lane == 0) {
    s_n[wid] = n;
    s_z[wid] = z;
  }
  __syncthreads();
  // every warp needs the group's tokens; warps of slot lane 0 add the lanes
  n = s_n[lane];
  z = s_z[lane];
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    n += __shfl_xor_sync(0xffffffffu, n, o);
    z += __shfl_xor_sync(0xffffffffu, z, o);
  }
  float bal = 0.f;
  if (ls == 0) {
    for (int u = 1; u < sl; ++u) {
      a += s_p[u * el + tx];
      c += s_c[u * el + tx];
    }
    if (e < p.E) {
      prob[(int64_t)g * p.E + e] = a;
      count[(int64_t)g * p.E + e] = c;
      if (n > 0) bal = (float)c * a / (float)n;
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) bal += __shfl_xor_sync(0xffffffffu, bal, o);
  if (lane == 0) s_b[wid] = bal;
  __syncthreads();
  if (wid != 0) {
    if (gridDim.x == 1) return;
  } else {
    bal = s_b[lane];
#pragma unroll
    for (int o = 16; o; o >>= 1) bal += __shfl_xor_sync(0xffffffffu, bal, o);
    if (lane == 0) {
      if (eb == 0) n_tok[g] = n;
      if (gridDim.x == 1) {
        write_loss(p, bal, z, n, loss);
      } else {
        w.bal[blockIdx.x] = bal;
        if (eb == 0) w.group_z[g] = z;
        __threadfence();
        s_last = atomicAdd(w.arrived, 1u) == gridDim.x - 1;
      }
    }
    if (gridDim.x == 1) return;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();
  // fixed order: thread t its share of the blocks and groups, then a tree
  __shared__ int64_t r_n[FIN_WARPS];
  float sb = 0.f, sz = 0.f;
  int64_t sn = 0;
  for (int64_t i = threadIdx.x; i < gridDim.x; i += FIN_THREADS) sb += __ldcg(w.bal + i);
  for (int i = threadIdx.x; i < p.G; i += FIN_THREADS) {
    sz += __ldcg(w.group_z + i);
    sn += __ldcg(n_tok + i);
  }
  auto tree = [&] {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      sb += __shfl_xor_sync(0xffffffffu, sb, o);
      sz += __shfl_xor_sync(0xffffffffu, sz, o);
      sn += __shfl_xor_sync(0xffffffffu, sn, o);
    }
  };
  tree();
  if (lane == 0) {
    s_b[wid] = sb;
    s_z[wid] = sz;
    r_n[wid] = sn;
  }
  __syncthreads();
  if (wid != 0) return;
  sb = s_b[lane];
  sz = s_z[lane];
  sn = r_n[lane];
  tree();
  if (lane == 0) write_loss(p, sb, sz, sn, loss);
}

// The gradient: each row is read once, its group's counts stay in registers while the group lasts.
template <int LPR, int NV, bool VEC>
__global__ void __launch_bounds__(AUX_THREADS, BLOCKS<NV>)
    aux_bwd_kernel(const AuxParams p, const int32_t* __restrict__ count,
                   const int32_t* __restrict__ n_tok, const float* __restrict__ d_loss, float* out,
                   int64_t ld_out, int accumulate, int rows_per_lane) {
  __shared__ int64_t s_n[AUX_WARPS];
  constexpr int RPW = 32 / LPR, U = ROWS<NV>;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int sub = lane % LPR, rw = lane / LPR;
  __shared__ int32_t s_off[OFF_CAP];
  dep_wait();
  dep_launch();
  const int64_t first = ((int64_t)blockIdx.x * AUX_WARPS + wid) * RPW * rows_per_lane;
  float v[U][NV];
  auto load = [&](int r0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t tok = first + (r0 + u) * RPW + rw;
      load_row<LPR, NV, VEC>(p, tok, r0 + u < rows_per_lane && tok < p.T, sub, v[u]);
    }
  };
  load(0);  // on their way while the counts are looked up
  const Groups groups(p, s_off);
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
  int cur = -2;       // group whose counts are in c
  int64_t cur_end = 0;
  float c[NV], cg = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) c[i] = 0.f;
  bool bad = false;
  for (int r0 = 0; r0 < rows_per_lane; r0 += U) {
    if (first + r0 * RPW >= p.T) break;
    if (r0 > 0) load(r0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t tok = first + (r0 + u) * RPW + rw;
      const bool in = r0 + u < rows_per_lane && tok < p.T;
      if (in && (cur == -2 || tok >= cur_end)) {
        cur = groups.of(tok);
        cur_end = cur >= 0 ? groups.at(cur + 1) : (tok < groups.at(0) ? groups.at(0) : p.T);
        const int ng = cur >= 0 ? n_tok[cur] : 0;
        cg = p.coef_b != 0.f && ng > 0 ? up * p.coef_b * p.share * inv_n / (float)ng : 0.f;
        if (cur >= 0) {
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int e = expert<LPR, NV>(sub, i);
            c[i] = e < p.E ? (float)count[(int64_t)cur * p.E + e] : 0.f;
          }
        }
      }
      if (cur < 0)  // a token of no group takes no part
#pragma unroll
        for (int i = 0; i < NV; ++i) v[u][i] = -INFINITY;
      float lse;
      row_softmax<LPR, NV>(v[u], lse);
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) s = fmaf(v[u][i], c[i], s);
      s = row_sum<LPR>(s);
      const float zt = zc * lse;
      if (in) {
        float* o = out + tok * ld_out;
        // 0 where p is 0, also under an upstream gradient whose factor is not finite
        if (fabsf(cg) < 1e28f && fabsf(zt) < 1e38f) {  // counts are below 2^31
#pragma unroll
          for (int i = 0; i < NV; ++i) v[u][i] *= fmaf(cg, c[i] - s, zt);
        } else {
#pragma unroll
          for (int i = 0; i < NV; ++i)
            if (v[u][i] != 0.f) v[u][i] *= fmaf(cg, c[i] - s, zt);
        }
        if constexpr (VEC) {
#pragma unroll
          for (int i = 0; i < NV; i += 4) {
            const int e = expert<LPR, NV>(sub, i);
            if (e >= p.E) continue;
            float4* at = reinterpret_cast<float4*>(o + e);
            float4 d = make_float4(v[u][i], v[u][i + 1], v[u][i + 2], v[u][i + 3]);
            if (accumulate) {
              const float4 old = *at;
              d.x += old.x, d.y += old.y, d.z += old.z, d.w += old.w;
            }
            *at = d;
            bad |= !finite_f(d.x) || !finite_f(d.y) || !finite_f(d.z) || !finite_f(d.w);
          }
        } else {
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int e = expert<LPR, NV>(sub, i);
            if (e >= p.E) continue;
            float d = v[u][i];
            if (accumulate) d += o[e];
            o[e] = d;
            bad |= !finite_f(d);
          }
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
  p.chunk = (int)aux_chunk_tokens(a.T, a.E);
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

// Calls f with the lanes per row and values per lane of E experts, and whether 16-byte vectors serve
// (`vec`: the rows allow them).
template <class F>
usaf_status by_width(int E, bool vec, F f) {
#define USAF_W(L, N)                                                                              \
  do {                                                                                            \
    if constexpr (N >= 4)                                                                         \
      if (vec)                                                                                    \
        return f(std::integral_constant<int, L>(), std::integral_constant<int, N>(),              \
                 std::true_type());                                                               \
    return f(std::integral_constant<int, L>(), std::integral_constant<int, N>(),                  \
             std::false_type());                                                                  \
  } while (0)
  if (E <= 8) USAF_W(8, 1);
  if (E <= 16) USAF_W(8, 2);
  if (E <= 32) USAF_W(8, 4);
  if (E <= 64) USAF_W(8, 8);
  if (E <= 128) USAF_W(8, 16);
  if (E <= 256) USAF_W(16, 16);
  if (E <= 512) USAF_W(32, 16);
  USAF_W(32, 32);
#undef USAF_W
}

bool rows_vec(const float* base, int64_t ld, int E) {
  return E % 4 == 0 && ld % 4 == 0 && (reinterpret_cast<uintptr_t>(base) & 15) == 0;
}

}  // namespace

// Tokens of a chunk. A batch of at most four rounds of the block's warps is one chunk, whose block forms the
// outputs itself (one launch); longer ones have up to four chunks per SM.
int64_t aux_chunk_tokens(int64_t T, int64_t E) {
  const int64_t rows = E <= 128 ? 4 : (E <= 256 ? 2 : 1);  // of a warp at a time
  if (T <= 4 * AUX_WARPS * rows) return T;
  const int64_t c = round_up(ceil_div(T, 4 * 152), 32);
  return c < 32 ? 32 : (c > MAX_CHUNK ? MAX_CHUNK : c);
}

void aux_ws_layout(int64_t T, int64_t E, int64_t G, Carver& c, AuxWs& w) {
  const int64_t slots = ceil_div(T, aux_chunk_tokens(T, E)) + G - 1;
  w.prob = c.take<float>(slots * E);
  w.count = c.take<int32_t>(slots * E);
  w.n = c.take<int32_t>(slots);
  w.z = c.take<float>(slots);
  w.bal = c.take<float>(G * ceil_div(E, 32));
  w.group_z = c.take<float>(G);
  w.arrived = c.take<uint32_t>(1);
}

usaf_status aux_fwd_launch(const AuxArgs& a, int32_t* count, float* prob_sum, int32_t* n_tok,
                           float* loss, const AuxWs& w, cudaStream_t st) {
  const AuxParams p = make_params(a);
  const size_t smem = (size_t)(AUX_WARPS + 1) * a.E * 4 + p.chunk;  // at most 40 KB
  // one block for everything, while it also clears the outputs of every group in little time
  const bool one = p.nchunks == 1 && a.G * a.E <= (1 << 16);
  USAF_TRY(by_width(a.E, rows_vec(a.logits, a.ld, a.E), [&](auto lpr, auto nv, auto vec) {
    USAF_TRACE("router_aux_part", st);
    auto go = [&](auto kernel) {
      kernel<<<p.nchunks, AUX_THREADS, smem, st>>>(p, w, count, prob_sum, n_tok, loss);
      USAF_CHECK_LAUNCH();
      return USAF_OK;
    };
    return one ? go(aux_part_kernel<lpr.value, nv.value, vec.value, true>)
               : go(aux_part_kernel<lpr.value, nv.value, vec.value, false>);
  }));
  if (one) return USAF_OK;
  USAF_TRACE("router_aux_final", st);
  // experts of a block: all of a common router's at once while that leaves a thread at most 20 chunks
  // (a batch of 4,096 tokens then needs one block and no counter), else fewer and more chunk lanes
  const int el = ceil_div(p.nchunks, a.G) <= 160 && a.E > 32 ? 128 : 32;
  const int nb = (int)ceil_div(a.E, el);
  return launch_dep(aux_final_kernel, dim3((unsigned)(nb * a.G)), FIN_THREADS, 0, st, p, w, el, nb,
                    count, prob_sum, n_tok, loss);
}

usaf_status aux_bwd_launch(const AuxArgs& a, const int32_t* count, const int32_t* n_tok,
                           const float* d_loss, float* dlogit, int64_t ld_out, int accumulate,
                           cudaStream_t st) {
  const AuxParams p = make_params(a);
  USAF_TRACE("router_aux_bwd", st);
  const bool rows_ok = rows_vec(a.logits, a.ld, a.E) && rows_vec(dlogit, ld_out, a.E);
  return by_width(a.E, rows_ok, [&](auto lpr, auto nv, auto vec) {
    constexpr int RPW = 32 / lpr.value;
    // rows per lane group: enough blocks for every SM first, then rows that share a count load
    const int64_t lanes = (int64_t)AUX_WARPS * RPW;
    int rows = 1;
    while (rows < 8 && ceil_div(a.T, lanes * rows * 2) >= 4 * 152) rows *= 2;
    const unsigned grid = (unsigned)ceil_div(a.T, lanes * rows);
    return launch_dep(aux_bwd_kernel<lpr.value, nv.value, vec.value>, dim3(grid), AUX_THREADS, 0, st, p, count,
                      n_tok, d_loss, dlogit, ld_out, accumulate, rows);
  });
}

}  // namespace usaf
