// Routing rules beyond softmax top-k: what follows the choice of experts (gate_select.cuh) in usaf_gate_topk,
// the gradient of the weights (usaf_gate_bwd) and the step of the balancing bias (usaf_gate_balance).
#include <algorithm>

#include "gate.cuh"

namespace usaf {

namespace {

constexpr int GATE_WARPS = 8;

GateParams params(const GateArgs& a) {
  GateParams p;
  p.T = a.T;
  p.ld = a.ld;
  p.E = a.E;
  p.k = a.k;
  p.G = a.gate.n_group;
  p.per = a.E / a.gate.n_group;
  p.keep = a.gate.topk_group;
  p.top = a.gate.group_top;
  p.sigmoid = a.gate.score == USAF_GATE_SIGMOID;
  p.renorm = a.gate.renorm;
  p.scale = a.gate.scale;
  p.logits = a.logits;
  p.bias = a.bias;
  p.status = a.status;
  return p;
}

// Lane = expert, the block's warps share the chunks: before[c][e] = slots of expert e in the chunks before c,
// total[e] = all of them. Bound by two rounds to L2 (512 chunks of 256 experts: 4 us).
__global__ void __launch_bounds__(1024) gate_scan_kernel(const uint32_t* __restrict__ masks, int E,
                                                         int nchunks, int32_t* __restrict__ before,
                                                         int32_t* __restrict__ total) {
  __shared__ int32_t part[32][33];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int e = blockIdx.x * 32 + lane;
  const int per = (nchunks + 31) / 32, c0 = warp * per, c1 = min(nchunks, c0 + per);
  dep_launch();
  dep_wait();
  // a warp's chunks: up to KEEP of them are read once, all in flight
  constexpr int KEEP = 16;
  int32_t n[KEEP], sum = 0;
  if (e < E) {
#pragma unroll
    for (int i = 0; i < KEEP; ++i) n[i] = c0 + i < c1 ? (int)masks[(int64_t)(c0 + i) * E + e] : 0;
#pragma unroll
    for (int i = 0; i < KEEP; ++i) sum += n[i] = __popc(n[i]);
#pragma unroll 8
    for (int c = c0 + KEEP; c < c1; ++c) sum += __popc(masks[(int64_t)c * E + e]);
  }
  part[warp][lane] = sum;
  __syncthreads();
  int32_t at = 0, all = 0;
#pragma unroll
  for (int w = 0; w < 32; ++w) {
    if (w == warp) at = all;
    all += part[w][lane];
  }
  if (e >= E) return;
  if (warp == 0) total[e] = all;
#pragma unroll
  for (int i = 0; i < KEEP; ++i) {
    if (c0 + i < c1) before[(int64_t)(c0 + i) * E + e] = at;
    at += n[i];
  }
#pragma unroll 8
  for (int c = c0 + KEEP; c < c1; ++c) {
    before[(int64_t)c * E + e] = at;
    at += __popc(masks[(int64_t)c * E + e]);
  }
}

// Slots of a block's chunk of tokens: n of them from s0 on.
struct ChunkSlots {
  int64_t s0;
  int n;
  __device__ __forceinline__ ChunkSlots(int64_t T, int k)
      : s0((int64_t)blockIdx.x * GATE_CHUNK * k),
        n((int)min((int64_t)GATE_CHUNK * k, T * k - (int64_t)blockIdx.x * GATE_CHUNK * k)) {}
};
// slot i's rank among its expert's slots of the chunk
__device__ __forceinline__ int rank_in_chunk(const uint32_t* masks, int E, int e, int tok) {
  return __popc(masks[(int64_t)blockIdx.x * E + e] & ((1u << tok) - 1));
}
__device__ __forceinline__ void write_slot(const GateTables& o, const ChunkSlots& c, int i, int tok,
                                           int32_t pos) {
  o.perm_tok[pos] = (int32_t)(blockIdx.x * GATE_CHUNK + tok);
  o.perm_slot[pos] = (int32_t)(c.s0 + i);
  o.slot_row[c.s0 + i] = pos;
}
// The rows behind each expert's, and behind all of them: a block's share.
template <class Total>
__device__ __forceinline__ void fill_rest(int E, const GateTables& o, const int32_t* s_off, Total total) {
  for (int64_t e = blockIdx.x; e < E; e += gridDim.x) {
    if (threadIdx.x < USAF_ROW_ALIGN)
      fill_padding(o, s_off[e] + total(e), s_off[e + 1], threadIdx.x, USAF_ROW_ALIGN);
    if (threadIdx.x == 0) {
      o.count[e] = total(e);
      o.offset[e] = s_off[e];
      if (e == E - 1) o.offset[E] = s_off[E];
    }
  }
  fill_tail(o, s_off[E], o.cap, (int64_t)blockIdx.x * blockDim.x + threadIdx.x,
            (int64_t)gridDim.x * blockDim.x);
}

__global__ void __launch_bounds__(256) gate_fill_kernel(int64_t T, int E, int k, const GateTables o,
                                                        const uint32_t* __restrict__ masks,
                                                        const int32_t* __restrict__ before,
                                                        const int32_t* __restrict__ total) {
  extern __shared__ int32_t smem[];
  int32_t* s_off = smem;           // [E + 1]
  int32_t* s_warp = smem + E + 1;  // [8]
  dep_launch();
  dep_wait();
  const ChunkSlots c(T, k);
  const auto look = [&](int i, int& e) {  // slot i's place among its expert's
    e = o.topk_idx[c.s0 + i];
    return before[(int64_t)blockIdx.x * E + e] + rank_in_chunk(masks, E, e, i / k);
  };
  // the thread's first slot is looked up while the offsets are formed
  int e1 = 0, at1 = 0;
  if ((int)threadIdx.x < c.n) at1 = look(threadIdx.x, e1);
  const auto tot = [&](int64_t e) { return total[e]; };
  expert_offsets(E, tot, s_off, s_warp);
  if ((int)threadIdx.x < c.n) write_slot(o, c, threadIdx.x, threadIdx.x / k, s_off[e1] + at1);
  for (int i = threadIdx.x + blockDim.x; i < c.n; i += blockDim.x) {
    int e;
    const int at = look(i, e);
    write_slot(o, c, i, i / k, s_off[e] + at);
  }
  fill_rest(E, o, s_off, tot);
}

// The same for batches of few chunks, without gate_scan_kernel before it: each block counts all chunks' words
// itself, from L2, `slices` threads an expert. What it reads grows with the square of the chunks, and what a
// thread reads with chunks * E: it is the faster one up to some 100 chunks, and to 12 to 20 K words (us, without
// and with the scan; the launch that it saves costs the host some 2 us besides):
//   E   8:  64 chunks 8.2, 8.3;   128 9.8, 9.2;     160 11.7, 9.3;   512 23.0, 15.2;  2,048 112.6, 48.7
//   E  64: 128 chunks 9.4, 10.0;  192 13.3, 11.4    E 128: 96 chunks 11.4, 11.5;  128 11.7, 11.7;  192 15.7, 12.9
//   E 160:  76 chunks 11.6, 11.6; 102 12.8, 11.7    E 256: 64 chunks 12.8, 13.4;  80 15.2, 13.2
//   E 512:  40 chunks 21.2, 21.3;  64 21.0, 20.3    E 1,024: 24 chunks 43.1, 43.5; 48 43.5, 41.5
constexpr int64_t FEW_CHUNKS = 128;
constexpr int64_t FEW_WORDS = 16384;
__global__ void __launch_bounds__(1024) gate_fill_few_kernel(int64_t T, int E, int k,
                                                             const GateTables o,
                                                             const uint32_t* __restrict__ masks,
                                                             int nchunks, int slices) {
  extern __shared__ int32_t smem[];
  int32_t* s_off = smem;                 // [E + 1]
  int32_t* s_warp = s_off + E + 1;       // [32]
  int32_t* s_total = s_warp + 32;        // [slices][E]
  int32_t* s_before = s_total + slices * E;
  dep_launch();
  dep_wait();
  const int width = (int)blockDim.x / slices, e0 = threadIdx.x % width, slice = threadIdx.x / width;
  for (int e = e0; e < E; e += width) {
    int32_t all = 0, mine = 0;
#pragma unroll 8
    for (int c = slice; c < nchunks; c += slices) {
      const int n = __popc(masks[(int64_t)c * E + e]);
      all += n;
      mine += c < (int)blockIdx.x ? n : 0;
    }
    s_total[slice * E + e] = all;
    s_before[slice * E + e] = mine;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x)
    for (int i = 1; i < slices; ++i) {
      s_total[e] += s_total[i * E + e];
      s_before[e] += s_before[i * E + e];
    }
  __syncthreads();
  const auto tot = [&](int64_t e) { return s_total[e]; };
  expert_offsets(E, tot, s_off, s_warp);
  const ChunkSlots c(T, k);
  for (int i = threadIdx.x; i < c.n; i += blockDim.x) {
    const int e = o.topk_idx[c.s0 + i], tok = i / k;
    write_slot(o, c, i, tok, s_off[e] + s_before[e] + rank_in_chunk(masks, E, e, tok));
  }
  fill_rest(E, o, s_off, tot);
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
  return v;
}

// ------------------------------------------------------------------------------------------------
// Gradient of the weights. One warp per token, lane j with its j-th slot. Where only the k experts' logits
// have a gradient, a row is cleared in wide stores and lane j writes its entry behind them, or, to add to
// what is there, touches nothing but its entry; a softmax over all experts writes -s u everywhere first.
// Bound by the launch and by memory: 16,383 tokens of 256 experts added to in 6 us (24 MB of DRAM reads; a
// form that read and wrote every entry took 11), 5,001 tokens of 160 experts, dense, 3 us.
// ------------------------------------------------------------------------------------------------

// Slot `lane` of a token: its expert (-1 for none), and what the weight's gradient puts there. Slots of one
// expert twice (no routing call makes them) are added up by the first of them.
struct Slot {
  int e;
  float w, d;  // 0 for slots that are constants
  float u;     // of the token
  __device__ __forceinline__ Slot(const GateParams& p, const int32_t* topk_idx, const float* topk_w,
                                  const float* dw, int64_t t, int lane, bool& bad_index)
      : e(-1), w(0.f), d(0.f) {
    if (lane < p.k) {
      e = topk_idx[t * p.k + lane];
      w = topk_w[t * p.k + lane];
      d = dw[t * p.k + lane];
      if (e < 0 || e >= p.E) {
        bad_index = true;
        e = -1;
      }
      if (e < 0 || w == 0.f) w = d = 0.f;
    }
    // renormalised weights sum to scale, so a single one has no gradient whatever its rounding
    u = warp_sum(p.renorm ? (w / p.scale) * d : w * d);
  }
  // v summed over the slots of the lane's expert; false for all but the first of them
  __device__ __forceinline__ bool first(int lane, float& v) const {
    const unsigned same = __match_any_sync(FULL, e < 0 ? -1 - lane : e);
    if (__any_sync(FULL, (same & (same - 1)) != 0)) {
      float sum = 0.f;
      for (int j = 0; j < 32; ++j) {
        const float x = __shfl_sync(FULL, v, j);
        if ((same >> j) & 1u) sum += x;
      }
      v = sum;
    }
    return e >= 0 && (same & ((1u << lane) - 1)) == 0;
  }
};

__global__ void __launch_bounds__(32 * GATE_WARPS)
    gate_bwd_kernel(const GateParams p, const int32_t* __restrict__ topk_idx,
                    const float* __restrict__ topk_w, const float* __restrict__ dw, float* dlogit,
                    int64_t ld_out, int accumulate) {
  const int lane = threadIdx.x % 32;
  const int64_t t = (int64_t)blockIdx.x * GATE_WARPS + threadIdx.x / 32;
  dep_launch();
  dep_wait();
  if (t >= p.T) return;
  bool bad_index = false;
  const Slot s(p, topk_idx, topk_w, dw, t, lane, bad_index);
  float pull = 0.f;
  if (s.w != 0.f) {
    pull = s.w * (p.renorm ? s.d - s.u : s.d);
    if (p.sigmoid) pull /= 1.f + expf(p.logits[t * p.ld + s.e]);  // 1 - s = 1 / (1 + exp(l))
  }
  const bool bad = !finite_f(pull);
  const bool mine = s.first(lane, pull);
  float* row = dlogit + t * ld_out;
  if (accumulate) {
    if (mine) row[s.e] += pull;
  } else {
    __syncwarp();  // the logits, which may be this row, are read
    if (((reinterpret_cast<uintptr_t>(row) | (uintptr_t)p.E * 4) & 15) == 0) {
      for (int e = 4 * lane; e < p.E; e += 128)
        *reinterpret_cast<float4*>(row + e) = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
      for (int e = lane; e < p.E; e += 32) row[e] = 0.f;
    }
    __syncwarp();
    if (mine) row[s.e] = pull;
  }
  flag_status_warp(p.status, bad, USAF_DEV_NONFINITE);
  flag_status_warp(p.status, bad_index, USAF_DEV_BAD_INDEX);
}

// Four neighbours of a row, by one access where `vec`.
__device__ __forceinline__ void row_load(const float* row, int e, int E, bool vec, float rest,
                                         float (&v)[4]) {
  if (vec && e < E) {
    const float4 q = *reinterpret_cast<const float4*>(row + e);
    v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = e + j < E ? row[e + j] : rest;
  }
}

// Softmax over all experts without renormalising: every logit has a gradient. Lane l has the NV groups of
// four logits 128 i + 4 l.
template <int NV>
__global__ void __launch_bounds__(32 * GATE_WARPS)
    gate_bwd_dense_kernel(const GateParams p, const int32_t* __restrict__ topk_idx,
                          const float* __restrict__ topk_w, const float* __restrict__ dw,
                          float* dlogit, int64_t ld_out, int accumulate) {
  const int lane = threadIdx.x % 32;
  const int64_t t = (int64_t)blockIdx.x * GATE_WARPS + threadIdx.x / 32;
  dep_launch();
  dep_wait();
  if (t >= p.T) return;
  const float* row = p.logits + t * p.ld;
  float* out = dlogit + t * ld_out;
  const bool vec = ((reinterpret_cast<uintptr_t>(row) | (uintptr_t)p.E * 4) & 15) == 0;
  const bool vec_out = ((reinterpret_cast<uintptr_t>(out) | (uintptr_t)p.E * 4) & 15) == 0;
  float l[NV][4];
#pragma unroll
  for (int i = 0; i < NV; ++i) row_load(row, 128 * i + 4 * lane, p.E, vec, -INFINITY, l[i]);
  bool bad_index = false;
  const Slot s(p, topk_idx, topk_w, dw, t, lane, bad_index);
  float own = s.e >= 0 ? row[s.e] : -INFINITY;
  const float old = s.e >= 0 && accumulate ? out[s.e] : 0.f;
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (isnan(l[i][j])) l[i][j] = -INFINITY;
      mx = fmaxf(mx, l[i][j]);
    }
  mx = warp_max(mx);
  const float ref = mx == -INFINITY ? 0.f : mx;
  float total = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) total += l[i][j] = expf(l[i][j] - ref);
  total = warp_sum(total);
  const float inv = 1.f / total;  // (a row of -inf alone has no scores to multiply)
  float got = s.w != 0.f ? p.scale * s.d : 0.f;
  const bool mine = s.first(lane, got);
  bool bad = false;
  __syncwarp();  // the rows, which may be one, are read
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = 128 * i + 4 * lane;
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[j] = l[i][j] != 0.f ? l[i][j] * inv * (0.f - s.u) : 0.f;
      bad |= !finite_f(v[j]);
    }
    if (e >= p.E) continue;
    if (accumulate) {
      float q[4];
      row_load(out, e, p.E, vec_out, 0.f, q);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += q[j];
    }
    if (vec_out) {
      *reinterpret_cast<float4*>(out + e) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (e + j < p.E) out[e + j] = v[j];
    }
  }
  __syncwarp();
  if (mine) {
    if (isnan(own)) own = -INFINITY;
    const float ex = expf(own - ref);
    const float v = ex != 0.f ? ex * inv * (got - s.u) : 0.f;
    bad |= !finite_f(v);
    out[s.e] = old + v;
  }
  flag_status_warp(p.status, bad, USAF_DEV_NONFINITE);
  flag_status_warp(p.status, bad_index, USAF_DEV_BAD_INDEX);
}

// One block, 3 us, most of it the launch: thread e sums expert e's counts; E * c[e] is compared with the
// total, so that no division decides a sign.
__global__ void __launch_bounds__(1024) gate_balance_kernel(int E, const int32_t* __restrict__ count,
                                                            int64_t n, float rate,
                                                            float* __restrict__ bias,
                                                            const uint32_t* status) {
  __shared__ long long sums[32];
  const int e = threadIdx.x;
  dep_launch();
  dep_wait();
  if (status && (*(volatile const uint32_t*)status & USAF_DEV_SKIP_MASK)) return;
  long long c = 0;
  if (e < E)
    for (int64_t i = 0; i < n; ++i) c += count[i * E + e];
  const long long part = warp_sum(c);
  if (e % 32 == 0) sums[e / 32] = part;
  __syncthreads();
  long long total = 0;
  for (int i = 0; i < (int)blockDim.x / 32; ++i) total += sums[i];
  if (e < E && total != E * c) bias[e] += total > E * c ? rate : -rate;
}

}  // namespace

void gate_ws_layout(const usaf_moe_shape& s, Carver& c, GateWs& w) {
  const int64_t n = ceil_div(s.T, GATE_CHUNK);
  w.masks = c.take<uint32_t>(n > 1 ? n * s.E : 0);
  w.before = c.take<int32_t>(n > 1 ? n * s.E : 0);
  w.total = c.take<int32_t>(s.E);
}

usaf_status gate_topk_launch(const GateArgs& a, const usaf_routing& rt, int64_t cap, const GateWs& w,
                             cudaStream_t st) {
  const GateParams p = params(a);
  const GateTables o{rt.topk_idx, rt.expert_count, rt.expert_offset, rt.perm_tok, rt.perm_slot,
                     rt.slot_row, rt.topk_w, cap};
  const int64_t n = ceil_div(a.T, GATE_CHUNK);
  {
    USAF_TRACE("gate_select", st);
    USAF_TRY(p.sigmoid ? gate_select_sigmoid(p, o, w.masks, n, st)
                       : gate_select_softmax(p, o, w.masks, n, st));
  }
  if (n == 1) return USAF_OK;
  if (n <= FEW_CHUNKS && n * a.E <= FEW_WORDS) {
    USAF_TRACE("gate_fill", st);
    // threads for as many slices as there are chunks, at most 1024
    const int width = (int)round_up(a.E, 32);
    const int slices = (int)std::max<int64_t>(1, std::min<int64_t>(1024 / width, n));
    const size_t smem = (a.E + 1 + 32 + 2 * (size_t)slices * a.E) * sizeof(int32_t);
    return launch_dep(gate_fill_few_kernel, dim3((unsigned)n), (unsigned)(slices * width), smem, st,
                      a.T, a.E, a.k, o, w.masks, (int)n, slices);
  }
  {
    USAF_TRACE("gate_scan", st);
    USAF_TRY(launch_dep(gate_scan_kernel, dim3((unsigned)ceil_div(a.E, 32)), 1024, 0, st, w.masks, a.E,
                        (int)n, w.before, w.total));
  }
  USAF_TRACE("gate_fill", st);
  return launch_dep(gate_fill_kernel, dim3((unsigned)n), 256, (a.E + 1 + 8) * sizeof(int32_t), st, a.T,
                    a.E, a.k, o, w.masks, w.before, w.total);
}

usaf_status gate_bwd_launch(const GateArgs& a, const int32_t* topk_idx, const float* topk_w,
                            const float* dw, float* dlogit, int64_t ld_out, int accumulate,
                            cudaStream_t st) {
  USAF_TRACE("gate_bwd", st);
  const GateParams p = params(a);
  const dim3 grid((unsigned)ceil_div(a.T, GATE_WARPS));
  constexpr unsigned threads = 32 * GATE_WARPS;
  if (p.sigmoid || p.renorm)
    return launch_dep(gate_bwd_kernel, grid, threads, 0, st, p, topk_idx, topk_w, dw, dlogit, ld_out,
                      accumulate);
  const auto go = [&](auto kernel) {
    return launch_dep(kernel, grid, threads, 0, st, p, topk_idx, topk_w, dw, dlogit, ld_out,
                      accumulate);
  };
  if (a.E <= 128) return go(gate_bwd_dense_kernel<1>);
  if (a.E <= 256) return go(gate_bwd_dense_kernel<2>);
  if (a.E <= 512) return go(gate_bwd_dense_kernel<4>);
  return go(gate_bwd_dense_kernel<8>);
}

usaf_status gate_balance_launch(int E, const int32_t* count, int64_t n, float rate, float* bias,
                                const uint32_t* status, cudaStream_t st) {
  USAF_TRACE("gate_balance", st);
  return launch_dep(gate_balance_kernel, dim3(1), (unsigned)round_up(E, 32), 0, st, E, count, n, rate,
                    bias, status);
}

}  // namespace usaf
