// The two products of a dense router gradient for bf16 tokens on tcgen05 tensor cores.
//
//   g_router[e, h] = g_in + sum_t dlogit[t, e] x[t, h]     (contraction over tokens)
//   dx[t, h]       = dx_in + sum_e dlogit[t, e] w[e, h]    (contraction over experts)
//
// dlogit and w are fp32; the tensor cores take bf16. Cutting a float to its upper 16 bits and doing
// the same with what is left gives three bf16 numbers whose sum is exactly the float (8 bits each of
// its 24), and a product of two bf16 numbers is exact in fp32. g_router uses all three parts of dlogit
// (x is bf16 already). dx uses all three parts of both operands and the six of their nine products that
// reach 2^-24 of the whole: a softmax's gradient sums to zero over the experts, so what the rows of w
// have in common cancels, and an error relative to w itself does not. (With two parts and three
// products, 2^-16, rows that differ by a thousandth of what they share gave 1% of error in dx, with
// six 3e-5, fp32 arithmetic 1e-4.) A first kernel writes the parts (6 bytes a logit, which stay in L2);
// the products' kernels are then fed by TMA alone. (Converting in the products' own kernels cost more:
// every feature group's CTA converts again.)
//
// Measured, both products with dx_in: T 4096, E 128, H 2048 31 us (54 MB; 8 us at the copy rate);
// T 8192, E 8, H 4096 46 us (202 MB; 30 us); T 16,383, E 128, H 2048 73 us (212 MB, 31 us; the bf16
// products alone are 40 us of tensor time). With dx's three products of two parts they were 29, 49 and
// 64 us. What bounds them is at each kernel.
#include "tc_ptx.cuh"
#include "train.cuh"

namespace usaf {

using namespace tcx;

namespace {

// How the parts lie in memory. Routers of at most 40 experts: rows of three parts side by side, part
// q from column q * part_cols(E) on. Others: blocks of 32 tokens x 64 experts (what a product's shared
// memory holds as one box), for each 32 tokens the blocks of the first 128 experts' three parts, then
// the next 128's, so that g_router's kernel takes a block of tokens with one copy instead of six
// (T = 16,383: 68 -> 65 us for both products). Columns past E hold zeros.
__host__ __device__ constexpr int part_cols(int E) { return (E + 7) / 8 * 8; }
__host__ __device__ constexpr bool side_by_side(int E) { return part_cols(E) <= 40; }
__host__ __device__ constexpr int halves(int E) { return E > 64 ? 2 : 1; }  // blocks of 128 experts
__host__ __device__ constexpr int blocks_of(int E) { return (E + 127) / 128 * 3 * halves(E); }
// the block of part q, experts [64 kb, 64 kb + 64)
__host__ __device__ constexpr int block_at(int E, int q, int kb) {
  return (kb / halves(E) * 3 + q) * halves(E) + kb % halves(E);
}
__host__ __device__ constexpr int split_cols(int E) {  // columns that the split writes of a part
  return side_by_side(E) ? part_cols(E) : (E + 127) / 128 * halves(E) * 64;
}
__host__ __device__ constexpr int64_t split_rows(int64_t T, int E) {
  return side_by_side(E) ? T : (T + 31) / 32 * 32;
}
constexpr int64_t parts_size(int64_t T, int E) {
  return split_rows(T, E) * (side_by_side(E) ? 3 * part_cols(E) : 64 * blocks_of(E));
}
// dx of at most 16 experts: the three parts' columns, side by side, are one axis of the contraction (a
// box of 64 columns holds them), and w's rows are repeated for each part.
__host__ __device__ constexpr bool stacked(int E) { return 3 * part_cols(E) <= 64; }
// Rows of w's parts: whole steps of the contraction, zero past the experts.
__host__ __device__ constexpr int w_rows(int E) {
  return ((stacked(E) ? 3 * part_cols(E) : E) + 15) / 16 * 16;
}

// ------------------------------------------------------------------------------ parts
__device__ __forceinline__ uint4 take_part(float (&v)[8]) {
  uint4 p;
  p.x = trunc_bf16x2(v[0], v[1]);
  p.y = trunc_bf16x2(v[2], v[3]);
  p.z = trunc_bf16x2(v[4], v[5]);
  p.w = trunc_bf16x2(v[6], v[7]);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = trunc_rest(v[i]);
  return p;
}

// One thread per eight logits of a token, then one per eight columns of w (when w is given).
__global__ void __launch_bounds__(256)
    router_grad_split_kernel(const float* __restrict__ dl, int64_t ld, int64_t T, int E, int vec,
                             __nv_bfloat16* __restrict__ parts, const float* __restrict__ w, int H,
                             __nv_bfloat16* __restrict__ wparts) {
  dep_launch();
  const int ec = split_cols(E) / 8, hc = H / 8;
  const int64_t rows = split_rows(T, E);
  int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  float v[8];
  if (i < rows * ec) {
    const int64_t t = i / ec;
    const int e = (int)(i - t * ec) * 8;
    const float* row = dl + t * ld + e;
    if (vec && t < T && e + 8 <= E) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(row));
      const float4 b = __ldg(reinterpret_cast<const float4*>(row) + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = t < T && e + j < E ? __ldg(row + j) : 0.f;
    }
    if (side_by_side(E)) {
      uint4* to = reinterpret_cast<uint4*>(parts + t * 3 * part_cols(E) + e);
#pragma unroll
      for (int q = 0; q < 3; ++q) to[q * ec] = take_part(v);
    } else {
      uint4* to = reinterpret_cast<uint4*>(
          parts + ((t / 32 * blocks_of(E) + block_at(E, 0, e / 64)) * 32 + t % 32) * 64 + e % 64);
#pragma unroll
      for (int q = 0; q < 3; ++q) to[q * halves(E) * (32 * 64 / 8)] = take_part(v);
    }
    return;
  }
  i -= rows * ec;
  if (!w || i >= (int64_t)w_rows(E) * hc) return;
  const int row = (int)(i / hc);
  const int64_t c = i - (int64_t)row * hc;
  const int e = stacked(E) ? (row < 3 * part_cols(E) ? row % part_cols(E) : E) : row;
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.f;
  if (e < E) {
    const float4* from = reinterpret_cast<const float4*>(w + (int64_t)e * H) + 2 * c;
    const float4 a = __ldg(from), b = __ldg(from + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  uint4* to = reinterpret_cast<uint4*>(wparts) + i;
#pragma unroll
  for (int q = 0; q < 3; ++q) to[q * (int64_t)w_rows(E) * hc] = take_part(v);
}

// ------------------------------------------------------------------------------ g_router
// A CTA owns 128 expert rows (M) by 256 features (N) over one stretch of the tokens (K). A = dlogit's
// parts, 32 tokens x 128 experts, experts contiguous (MN-major); B = x, 32 tokens x 256 features
// (MN-major). Routers of at most 40 experts have their three parts side by side in one 128-row A
// (STACK): one MMA instead of three, the rows added at the end. Otherwise the leading part and the
// two smaller ones have accumulators of their own.
// The tensor core adds to its accumulator with truncation, an error that grows with the number of
// additions (1.8e-8 a step here), so the leading accumulator is emptied every FLUSH blocks (16
// steps) into fp32 registers of the epilogue warps, which round to nearest. The smaller parts' sums
// are 2^-8 of it and need no such care; their MMAs run while it is read. (STACK: two accumulators
// take turns.) Error in norm against 64 bits at 16,383 tokens: 1.0e-6 without, 3e-7 with.
// T 4096, E 128, H 2048: 13 us, of which 2 us until the first block has come, 4 us of MMAs (28% of
// the tensor pipe over the kernel) and 4 us to bring out 128 KB a CTA. T 16,383: 23 us; a block of
// 40 KB takes 1,100-1,300 cycles where its MMAs take 800, with 200 KB in flight on every SM.
namespace gw {
constexpr int BK = 32;
constexpr int N = 256;
constexpr int BOX = 64 * BK * 2;
constexpr int B_BYTES = 4 * BOX;
constexpr int FLUSH = 8;
constexpr int EPI_WARPS = 16;  // of each 32 lanes by 64 columns
constexpr int OUT_PITCH = N + 4;  // floats per row of the tile in the epilogue
constexpr int THREADS = 64 + 32 * EPI_WARPS;
template <bool STACK>
struct Cfg {
  static constexpr int PARTS = STACK ? 1 : 3;
  static constexpr int NS = STACK ? 8 : 5;
  static constexpr int A_BYTES = PARTS * 2 * BOX;
  static constexpr int STAGE = A_BYTES + B_BYTES;
  static constexpr int RING = NS * STAGE;
  static constexpr int SMEM = RING + 1024 + 256;
  static_assert(128 * OUT_PITCH * 4 <= RING, "output tile in the ring");
  static_assert(SMEM <= 232448, "shared memory");
};
struct Params {
  int64_t T;
  int E, H;
  int64_t per_split;
  const float* g_in;
  float* out;      // g_router, or the stretches' sums [splits][E][H]
  int whole;       // one stretch: out is g_router
  uint32_t* status;
};
}  // namespace gw

template <bool STACK>
__global__ void __launch_bounds__(gw::THREADS, 1)
    router_grad_w_tc_kernel(const __grid_constant__ CUtensorMap tm_d,
                            const __grid_constant__ CUtensorMap tm_x, const gw::Params p) {
  using C = gw::Cfg<STACK>;
  using namespace gw;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::RING);
  // full[NS], empty[NS], taken[2] (accumulator complete), given[2] (accumulator read), done
  const uint32_t full = smem_u32(bars), empty = full + 8 * C::NS, taken = empty + 8 * C::NS,
                 given = taken + 16, done = given + 16;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * C::NS + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  constexpr uint32_t COLS = 2 * N;  // STACK: two accumulators; else leading part | smaller parts
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int h0 = blockIdx.x * N, e0 = blockIdx.y * 128;
  const int64_t t0 = blockIdx.z * p.per_split;
  const int64_t t1 = min(p.T, t0 + p.per_split);
  const int nkb = (int)((t1 - t0 + BK - 1) / BK);
  const int nbox = min(4, (p.H - h0) / 64);
  const int ep = STACK ? part_cols(p.E) : min(part_cols(p.E) - e0, 128);
  const int na = STACK ? (3 * ep > 64 ? 2 : 1) : halves(p.E);  // 64-expert boxes of a part

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(taken + 8 * i, 1);
      mbar_init(given + 8 * i, EPI_WARPS);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  dep_wait();    // the parts are written
  dep_launch();  // dx's kernel may be set up beside this one

  if (warp == 0) {
    if (lane == 0) {  // ------------------------------------------------ loads
      int issued = 0;
      bool ok = true;
      for (int kb = 0; kb < nkb; ++kb) {
        const int s = kb % C::NS;
        ok = mbar_wait(empty + 8 * s, ((kb / C::NS) & 1) ^ 1, abort_flag);
        if (!ok) break;
        const uint32_t a = smem_u32(smem + s * C::STAGE), b = a + C::A_BYTES, fb = full + 8 * s;
        const int t = (int)(t0 + (int64_t)kb * BK);
        mbar_expect_tx(fb, C::PARTS * na * BOX + B_BYTES);
        if constexpr (STACK) {
          for (int i = 0; i < na; ++i) tma_load_2d(a + i * BOX, &tm_d, fb, 64 * i, t);
        } else {
          tma_load_4d(a, &tm_d, fb, 0, 0, blockIdx.y * 3 * na, t / BK);
        }
        tma_load_3d(b, &tm_x, fb, 0, t, h0 / 64);  // four boxes, zeros past the last feature
        ++issued;
      }
      if (!ok) *abort_flag = 1;
      const long long deadline = clock64() + TIMEOUT_CYCLES;  // every copy lands before the end
      for (int s = 0; s < C::NS && s < issued; ++s) {
        const int last = issued - 1 - ((issued - 1 - s) % C::NS);
        mbar_drain(full + 8 * s, (last / C::NS) & 1, deadline);
      }
    }
  } else if (warp == 1) {
    {  // ------------------------------------------------------------ MMAs
      const bool leader = elect_one();
      const uint32_t idesc = idesc_bf16(64 * nbox, true, true);
      const uint64_t ad0 = sdesc(smem_u32(smem), BOX, 1024);
      const uint64_t bd0 = sdesc(smem_u32(smem) + C::A_BYTES, BOX, 1024);
      bool ok = true;
      for (int kb = 0; kb < nkb; ++kb) {
        const int s = kb % C::NS;
        ok = mbar_wait_all(full + 8 * s, (kb / C::NS) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint64_t a = ad0 + ((s * C::STAGE) >> 4), b = bd0 + ((s * C::STAGE) >> 4);
        auto part = [&](uint32_t d, int q, bool fresh) {
          if (!leader) return;
#pragma unroll
          for (int ks = 0; ks < BK / 16; ++ks)
            umma_bf16(d, a + ((q * na * BOX + ks * 2048) >> 4), b + ((ks * 2048) >> 4), idesc,
                      fresh && ks == 0 ? 0u : 1u);
        };
        if constexpr (!STACK) {
          part(tmem + N, 1, kb == 0);
          part(tmem + N, 2, false);
        }
        const int turn = kb / FLUSH, acc = STACK ? turn & 1 : 0;
        const bool fresh = kb % FLUSH == 0;
        if (fresh) {  // the accumulator's last sums have been read
          const int use = STACK ? turn >> 1 : turn;  // how often it has been used before
          ok = mbar_wait_all(given + 8 * acc, (use & 1) ^ 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
        }
        part(tmem + acc * N, 0, fresh);
        if (leader) {
          umma_commit(empty + 8 * s);
          if (kb % FLUSH == FLUSH - 1 || kb == nkb - 1) umma_commit(taken + 8 * acc);
        }
        __syncwarp();
      }
      if (!ok) *abort_flag = 1;
      if (leader) {
        umma_commit(done);
        mbar_drain(done, 0, clock64() + TIMEOUT_CYCLES);
      }
      __syncwarp();
    }
  } else {  // ---------------------------------------------------- epilogue
    const int q = warp & 3, col = (warp - 2) >> 2;  // lanes' quarter, box of columns
    const uint32_t ta = tmem + ((uint32_t)(q * 32) << 16) + col * 64;
    const bool mine = q * 32 < (STACK ? 3 * ep : ep) && col < nbox;
    float sum[2][32];  // this lane's row, 64 columns
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int j = 0; j < 32; ++j) sum[c][j] = 0.f;
    auto add = [&](uint32_t from) {
      if (!mine) return;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float d[16];
        tmem_ld16(from + c * 16, d);
#pragma unroll
        for (int j = 0; j < 16; ++j) sum[c / 2][c % 2 * 16 + j] += d[j];
      }
    };
    bool ok = true;
    for (int turn = 0; turn * FLUSH < nkb; ++turn) {
      const int acc = STACK ? turn & 1 : 0, use = STACK ? turn >> 1 : turn;
      ok = mbar_wait_warp(taken + 8 * acc, use & 1, abort_flag);
      if (!ok) break;
      tc_fence_after();
      add(ta + acc * N);
      if ((turn + 1) * FLUSH >= nkb) break;  // the last: every MMA is complete
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(given + 8 * acc);
    }
    if (ok) {
      if constexpr (!STACK) add(ta + N);
      // registers -> the ring (free after the last MMA), for whole rows of global memory
      float* tile = reinterpret_cast<float*>(smem) + (q * 32 + lane) * OUT_PITCH + col * 64;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (!mine) break;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          reinterpret_cast<float4*>(tile + c * 32)[j] = make_float4(
              sum[c][4 * j], sum[c][4 * j + 1], sum[c][4 * j + 2], sum[c][4 * j + 3]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    if (threadIdx.x == 0) flag_status(p.status, USAF_DEV_TIMEOUT);
  } else {
    float* tile = reinterpret_cast<float*>(smem);
    const int ne = min(p.E - e0, 128), w4 = nbox * 16;
    bool bad = false;
    if (STACK || p.whole)
      for (int i = threadIdx.x; i < ne * w4; i += THREADS) {
        const int e = i / w4, c = (i - e * w4) * 4;
        float4 a = *reinterpret_cast<const float4*>(tile + e * OUT_PITCH + c);
        if constexpr (STACK) {
#pragma unroll
          for (int part = 1; part < 3; ++part) {
            const float4 b =
                *reinterpret_cast<const float4*>(tile + (e + part * ep) * OUT_PITCH + c);
            a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
          }
        }
        if (!p.whole) {
          *reinterpret_cast<float4*>(tile + e * OUT_PITCH + c) = a;
          continue;
        }
        const int64_t o = (int64_t)(e0 + e) * p.H + h0 + c;
        float r[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // g_in and g_router need no alignment
          if (p.g_in) r[j] += p.g_in[o + j];
          bad |= !finite_f(r[j]);
          p.out[o + j] = r[j];
        }
      }
    flag_status_warp(p.status, bad, USAF_DEV_NONFINITE);
    if (!p.whole) {  // rows of the tile by the copy engine
      fence_async_smem();
      __syncthreads();
      if (threadIdx.x < ne) {
        bulk_store(p.out + blockIdx.z * (int64_t)p.E * p.H + (int64_t)(e0 + threadIdx.x) * p.H + h0,
                   smem_u32(tile + threadIdx.x * OUT_PITCH), nbox * 256);
        bulk_commit();
        bulk_wait();
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free(tmem, COLS);
  }
}

// g_router = g_in + the stretches' sums in their order: thread i of n
__device__ __forceinline__ void reduce_parts(const float* part, int splits, int64_t count,
                                             const float* g_in, float* g, uint32_t* status,
                                             int64_t i0, int64_t n) {
  bool bad = false;
  for (int64_t i = i0 * 4; i < count; i += n * 4) {  // count = E H is a multiple of 64
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int U = 10;  // loads in flight
    for (int s0 = 0; s0 < splits; s0 += U) {
      float4 d[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (s0 + u < splits) d[u] = __ldcg(reinterpret_cast<const float4*>(part + (s0 + u) * count + i));
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (s0 + u < splits) v.x += d[u].x, v.y += d[u].y, v.z += d[u].z, v.w += d[u].w;
    }
    float r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {  // g_in and g_router need no alignment
      if (g_in) r[j] += g_in[i + j];
      bad |= !finite_f(r[j]);
      g[i + j] = r[j];
    }
  }
  flag_status_warp(status, bad, USAF_DEV_NONFINITE);
}
__global__ void __launch_bounds__(256)
    router_grad_sum_kernel(const float* part, int splits, int64_t count, const float* g_in,
                           float* g, uint32_t* status) {
  dep_wait();
  reduce_parts(part, splits, count, g_in, g, status, (int64_t)blockIdx.x * 256 + threadIdx.x,
               (int64_t)gridDim.x * 256);
}

// ------------------------------------------------------------------------------ dx
// A CTA owns 128 features and walks token tiles of 128: A = dlogit's three parts (K-major, 64 experts
// a block), B = w's three parts, accumulators in tensor memory, twice. A block's parts come one by one
// through a ring of 16 KB slots, the leading one first, and each slot is free again after the products
// that use it: three, two and one. RES: B for all experts stays in shared memory (at most 160 experts);
// else its blocks come through the ring ahead of A's. STACK (RES, at most 16 experts): all parts of a
// tile are one slot, whose products are w's three parts (T 8192, E 8, H 4096: both products 57 us with
// three mostly empty slots a tile). dx_in comes and dx goes by TMA through a ring of
// 128 x 64 boxes in which the epilogue adds, so token rows are read and written in whole lines while
// later tiles are on their way. The shared memory that B leaves goes to boxes first (eight, four or
// two), then to the ring.
// The same launch adds up g_router's stretches (`sum`): its epilogue warps do so while the first
// tiles are on their way, which saves a launch and hides most of the sum.
// T 16,383, E 128, H 2048: each of the 16 feature groups reads dlogit's parts, 201 MB between L2 and the
// SMs beside 134 MB of dx_in and dx, with 64 KB of parts and 64 KB of boxes in flight on an SM; that
// bounds it (two parts instead of three: 10 us less).
namespace gx {
constexpr int TM = 128;      // tokens of a tile
constexpr int NH = 128;      // features of a CTA
constexpr int KB = 64;       // experts of a block
constexpr int SLOT = TM * KB * 2;  // a part of A (128 tokens x 64 experts) or B (64 x 128 features)
constexpr int BOX = TM * 64 * 2;
constexpr int MAX_RES = 160;
constexpr int MAX_RING = 10;
constexpr int MAX_SLOTS = 8;
constexpr int EPI_WARPS = 16;  // two boxes of a tile by two tiles by four quarters of lanes
constexpr int THREADS = 96 + 32 * EPI_WARPS;
constexpr int SMEM_MAX = 232448;
constexpr int EXTRA = 1024 + 512;  // alignment, barriers
__host__ __device__ constexpr int b_bytes(int ke) {  // of the resident parts
  return ke <= MAX_RES ? 3 * 2 * ke * 128 : 0;
}
__host__ __device__ constexpr int fit(int ke, int boxes) {  // ring slots beside that many boxes
  return (SMEM_MAX - EXTRA - b_bytes(ke) - boxes * BOX) / SLOT;
}
// Boxes of the staging ring. A wait by parity tells a phase only from its neighbours, so a box's
// barriers serve one epilogue group, whose tiles use the box in turn: with two groups a box (tiles
// of either parity) that takes a multiple of four; where fewer fit, one group does all tiles.
__host__ __device__ constexpr int slots(int ke) {
  if (ke > MAX_RES) return 4;
  return fit(ke, 8) >= 3 ? 8 : (fit(ke, 4) >= 4 ? 4 : 2);
}
__host__ __device__ constexpr int ring(int ke) {
  return fit(ke, slots(ke)) < MAX_RING ? fit(ke, slots(ke)) : MAX_RING;
}
static_assert(slots(64) == 8 && slots(128) == 4 && slots(MAX_RES) == 2, "boxes");
// streamed B: a block's six parts and more
static_assert(ring(64) >= 3 && ring(128) >= 4 && ring(MAX_RES) >= 4 && ring(1024) >= 7, "ring");
struct Params {
  int64_t T;
  int E, H, ke;
  int ring, slots;
  int per_group;   // CTAs that share a feature group
  int add;         // dx_in is there
  uint32_t* status;
  const float* sum;  // g_router's stretches to add up, or null
  int splits;
  const float* g_in;
  float* g_router;
};
}  // namespace gx

template <bool RES, bool STACK>
__global__ void __launch_bounds__(gx::THREADS, 1)
    router_grad_x_tc_kernel(const __grid_constant__ CUtensorMap tm_d,
                            const __grid_constant__ CUtensorMap tm_w,
                            const __grid_constant__ CUtensorMap tm_in,
                            const __grid_constant__ CUtensorMap tm_out, const gx::Params p) {
  using namespace gx;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  static_assert(RES || !STACK, "stacked parts of few experts are resident");
  constexpr int PARTS = STACK ? 1 : 3;  // slots of a block of A
  const int ke = p.ke, NS = p.slots, NA = p.ring;
  uint8_t* sRing = smem;
  uint8_t* sStage = smem + NA * SLOT;
  uint8_t* sB = sStage + NS * BOX;  // RES: [part][feature group of 64][expert][64 features]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sB + b_bytes(ke));
  // full[], empty[] of the ring, tfull[2], tempty[2], loaded[], added[], freed[] of the boxes, done,
  // wfull
  const uint32_t full = smem_u32(bars), empty = full + 8 * MAX_RING, tfull = empty + 8 * MAX_RING,
                 tempty = tfull + 16, loaded = tempty + 16, added = loaded + 8 * MAX_SLOTS,
                 freed = added + 8 * MAX_SLOTS, done = freed + 8 * MAX_SLOTS, wfull = done + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * MAX_RING + 4 + 3 * MAX_SLOTS + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  constexpr uint32_t COLS = 2 * NH;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int groups = gridDim.x / p.per_group;
  const int h0 = (blockIdx.x % groups) * NH;
  const int first = blockIdx.x / groups;
  const int tiles = (int)((p.T + TM - 1) / TM);
  const int nbox = min(2, (p.H - h0) / 64);
  const int nkb = (ke + KB - 1) / KB;
  const int part_b = 2 * ke * 128;  // RES: bytes of a part of B

  if (threadIdx.x == 0) {
    for (int i = 0; i < NA; ++i) {
      mbar_init(full + 8 * i, 1);
      mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(tfull + 8 * i, 1);
      mbar_init(tempty + 8 * i, 4 * nbox);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(loaded + 8 * i, 1);
      mbar_init(added + 8 * i, 4);
      mbar_init(freed + 8 * i, 1);
    }
    mbar_init(done, 1);
    mbar_init(wfull, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // Every thread waits, the loading ones too: that g_router's kernel has seen the parts written orders
  // nothing for this grid, only that kernel's end does.
  dep_wait();
  bool bad = false;

  if (warp == 0) {
    if (lane == 0) {  // ------------------------------------------------ A and B parts
      bool ok = true;
      int it = 0, s = 0;  // slots filled, the next one
      uint32_t ph = 1;
      auto acquire = [&](uint32_t bytes) {
        ok = mbar_wait(empty + 8 * s, ph, abort_flag);
        if (ok) mbar_expect_tx(full + 8 * s, bytes);
        return ok;
      };
      auto advance = [&] {
        ++it;
        if (++s == NA) s = 0, ph ^= 1;
      };
      if constexpr (RES) {
        mbar_expect_tx(wfull, 3 * nbox * ke * 128);
        for (int q = 0; q < 3; ++q)
          for (int i = 0; i < nbox; ++i)
            tma_load_2d(smem_u32(sB + q * part_b + i * ke * 128), &tm_w, wfull, h0 + 64 * i,
                        q * ke);
      }
      for (int t = first; t < tiles && ok; t += p.per_group)
        for (int kb = 0; kb < nkb && ok; ++kb) {
          if constexpr (!RES)
            for (int q = 0; q < 3 && acquire(nbox * KB * 128); ++q, advance())
              for (int i = 0; i < nbox; ++i)
                tma_load_2d(smem_u32(sRing + s * SLOT + i * KB * 128), &tm_w, full + 8 * s,
                            h0 + 64 * i, q * ke + kb * KB);
          for (int q = 0; ok && q < PARTS && acquire(SLOT); ++q, advance()) {
            const uint32_t a = smem_u32(sRing + s * SLOT), fb = full + 8 * s;
            if (side_by_side(p.E))
              tma_load_2d(a, &tm_d, fb, q * part_cols(p.E), t * TM);
            else
              tma_load_4d(a, &tm_d, fb, 0, 0, block_at(p.E, q, kb), t * (TM / 32));
          }
        }
      if (!ok) *abort_flag = 1;
      const long long deadline = clock64() + TIMEOUT_CYCLES;
      if constexpr (RES) mbar_drain(wfull, 0, deadline);
      for (int i = 0; i < NA && i < it; ++i) {
        const int last = it - 1 - ((it - 1 - i) % NA);
        mbar_drain(full + 8 * i, (last / NA) & 1, deadline);
      }
    }
  } else if (warp == 1) {
    {  // ------------------------------------------------------------ MMAs
      const bool leader = elect_one();
      const uint32_t idesc = idesc_bf16(64 * nbox, false, true);
      const uint64_t ad0 = sdesc(smem_u32(sRing), 16, 1024);
      const uint64_t bd0 = RES ? sdesc(smem_u32(sB), ke * 128, 1024)
                               : sdesc(smem_u32(sRing), KB * 128, 1024);
      int n = 0, s = 0;
      uint32_t ph = 0;
      bool ok = true;
      auto arrived = [&] {  // the next slot of the ring
        ok = mbar_wait_all(full + 8 * s, ph, abort_flag);
        if (ok) tc_fence_after();
        return ok;
      };
      auto advance = [&] {
        if (++s == NA) s = 0, ph ^= 1;
      };
      if constexpr (RES) ok = mbar_wait_all(wfull, 0, abort_flag);
      for (int t = first; t < tiles && ok; t += p.per_group, ++n) {
        ok = mbar_wait_all(tempty + 8 * (n & 1), ((n >> 1) & 1) ^ 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tmem + (n & 1) * NH;
        for (int kb = 0; kb < nkb && ok; ++kb) {
          uint64_t b[3];
          int sb[3];
#pragma unroll
          for (int q = 0; q < 3; ++q) {
            if constexpr (RES) {
              b[q] = bd0 + ((q * part_b + kb * KB * 128) >> 4);
            } else {
              if (!ok || !arrived()) break;
              sb[q] = s;
              b[q] = bd0 + ((s * SLOT) >> 4);
              advance();
            }
          }
          const int steps = min(KB / 16, ke / 16 - kb * (KB / 16));
#pragma unroll
          for (int q = 0; q < PARTS; ++q) {  // dlogit's part q by w's parts 0 to 2 - q
            if (!ok || !arrived()) break;
            if (leader) {
              const uint64_t a = ad0 + ((s * SLOT) >> 4);
#pragma unroll
              for (int r = 0; r < 3 - q; ++r)
                for (int ks = 0; ks < steps; ++ks)
                  umma_bf16(d, a + ((ks * 32) >> 4), b[r] + ((ks * 2048) >> 4), idesc,
                            kb > 0 || q > 0 || r > 0 || ks > 0 ? 1u : 0u);
              umma_commit(empty + 8 * s);
            }
            __syncwarp();
            advance();
          }
          if constexpr (!RES)
            if (ok && leader)
              for (int q = 0; q < 3; ++q) umma_commit(empty + 8 * sb[q]);
        }
        if (ok && leader) umma_commit(tfull + 8 * (n & 1));
        __syncwarp();
      }
      if (!ok) *abort_flag = 1;
      if (leader) {
        umma_commit(done);
        mbar_drain(done, 0, clock64() + TIMEOUT_CYCLES);
      }
      __syncwarp();
    }
  } else if (warp == 2) {
    if (lane == 0) {  // ------------------------------------------------ dx_in boxes
      int u = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += p.per_group)
        for (int b = 0; b < nbox && ok; ++b) {
          const int s = u % NS;
          ok = mbar_wait(freed + 8 * s, ((u / NS) & 1) ^ 1, abort_flag);
          if (!ok) break;
          if (p.add) {
            mbar_expect_tx(loaded + 8 * s, BOX);
            tma_load_2d(smem_u32(sStage + s * BOX), &tm_in, loaded + 8 * s, h0 + 64 * b, t * TM);
          } else {
            mbar_arrive(loaded + 8 * s);
          }
          ++u;
        }
      if (!ok) *abort_flag = 1;
      const long long deadline = clock64() + TIMEOUT_CYCLES;
      for (int s = 0; s < NS && s < u; ++s) {
        const int last = u - 1 - ((u - 1 - s) % NS);
        mbar_drain(loaded + 8 * s, (last / NS) & 1, deadline);
      }
    }
  } else {  // ---------------------------------------------------- epilogue: add and store
    // lanes' quarter, box of the tile, tiles of one parity (and so one accumulator)
    const int q = warp & 3, b = ((warp - 3) >> 2) & 1, par = (warp - 3) >> 3;
    const int pars = NS >= 4 ? 2 : 1;
    const bool issuer = ((warp - 3) & 3) == 0 && lane == 0;
    const int row = q * 32 + lane;
    if (p.sum) {
      constexpr int N = 32 * EPI_WARPS;
      reduce_parts(p.sum, p.splits, (int64_t)p.E * p.H, p.g_in, p.g_router, p.status,
                   (int64_t)blockIdx.x * N + threadIdx.x - 96, (int64_t)gridDim.x * N);
      __syncwarp();
    }
    if (b < nbox && par < pars) {
      for (int n = par, t = first + par * p.per_group; t < tiles;
           t += pars * p.per_group, n += pars) {
        const int u = n * nbox + b, s = u % NS;
        const uint32_t ph = (u / NS) & 1;
        if (!mbar_wait_warp(loaded + 8 * s, ph, abort_flag)) break;
        if (!mbar_wait_warp(tfull + 8 * (n & 1), (n >> 1) & 1, abort_flag)) break;
        tc_fence_after();
        uint8_t* box = sStage + s * BOX + row * 128;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float d[32];
          tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + (n & 1) * NH + b * 64 + half * 32, d);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint4* at = reinterpret_cast<uint4*>(box + (((half * 4 + c) ^ (row & 7)) << 4));
            if (p.add) {
              const uint4 in = *at;
              const uint32_t w[4] = {in.x, in.y, in.z, in.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                d[8 * c + 2 * j] += __uint_as_float(w[j] << 16);
                d[8 * c + 2 * j + 1] += __uint_as_float(w[j] & 0xFFFF0000u);
              }
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)  // from there on bf16 rounds to infinity; NaN too
              bad |= !(fabsf(d[8 * c + j]) < 0x1.FFp127f);
            *at = make_uint4(pack_bf16x2(d[8 * c], d[8 * c + 1]),
                             pack_bf16x2(d[8 * c + 2], d[8 * c + 3]),
                             pack_bf16x2(d[8 * c + 4], d[8 * c + 5]),
                             pack_bf16x2(d[8 * c + 6], d[8 * c + 7]));
          }
        }
        tc_fence_before();
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(tempty + 8 * (n & 1));
          mbar_arrive(added + 8 * s);
        }
        if (issuer) {
          if (mbar_wait(added + 8 * s, ph, abort_flag)) {
            tma_store_2d(&tm_out, smem_u32(sStage + s * BOX), h0 + 64 * b, t * TM);
            bulk_commit();
            bulk_wait_read();
            mbar_arrive(freed + 8 * s);
          } else {
            *abort_flag = 1;
          }
        }
        __syncwarp();
      }
      if (issuer) bulk_wait();
      __syncwarp();
    }
  }
  flag_status_warp(p.status, bad, USAF_DEV_NONFINITE);
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag) flag_status(p.status, USAF_DEV_TIMEOUT);
  if (warp == 1) {
    tc_fence_after();
    tmem_free(tmem, COLS);
  }
}

// The parts in boxes of `tokens` x 64 experts side by side, else of `blocks` blocks by `tokens` / 32
// blocks of 32 tokens.
bool map_parts(CUtensorMap* m, const void* parts, int64_t T, int E, uint32_t blocks,
               uint32_t tokens) {
  if (side_by_side(E)) return map_bf16_2d(m, parts, 3 * part_cols(E), T, 64, tokens);
  const uint64_t dims[4] = {64, 32, (uint64_t)blocks_of(E), (uint64_t)(split_rows(T, E) / 32)};
  const uint64_t pitch[3] = {128, 128 * 32, 128 * 32 * dims[2]};
  const uint32_t box[4] = {64, 32, blocks, tokens / 32};
  return map_bf16(m, parts, 4, dims, pitch, box);
}

template <class K>
bool grow_smem(OncePerDevice& once, K kernel, int bytes) {
  return once([&] {
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) ==
           cudaSuccess;
  });
}

template <bool STACK>
usaf_status launch_w(const CUtensorMap& d, const CUtensorMap& x, const gw::Params& p, dim3 grid,
                     cudaStream_t st) {
  USAF_TRACE("router_grad_w", st);
  using C = gw::Cfg<STACK>;
  static OncePerDevice once;
  if (!grow_smem(once, router_grad_w_tc_kernel<STACK>, C::SMEM)) return USAF_ERR_CUDA;
  return launch_dep(router_grad_w_tc_kernel<STACK>, grid, gw::THREADS, C::SMEM, st, d, x, p);
}

template <bool RES, bool STACK>
usaf_status launch_x(const CUtensorMap& d, const CUtensorMap& w, const CUtensorMap& in,
                     const CUtensorMap& out, const gx::Params& p, unsigned grid, cudaStream_t st) {
  USAF_TRACE("router_grad_x", st);
  static OncePerDevice once;
  if (!grow_smem(once, router_grad_x_tc_kernel<RES, STACK>, gx::SMEM_MAX)) return USAF_ERR_CUDA;
  const int smem = p.ring * gx::SLOT + p.slots * gx::BOX + gx::b_bytes(p.ke) + gx::EXTRA;
  return launch_dep(router_grad_x_tc_kernel<RES, STACK>, dim3(grid), gx::THREADS, smem, st, d, w, in, out,
                    p);
}

// Tokens of a stretch of g_router's sum: about one CTA per SM, whole blocks, at least 128 tokens.
int64_t stretch(int64_t T, int64_t E, int64_t H) {
  const int64_t tiles = ceil_div(H, gw::N) * ceil_div(E, 128);
  const int64_t s = tiles < 152 ? 152 / tiles : 1;
  const int64_t per = round_up(ceil_div(T, s), gw::BK);
  return per < 128 ? 128 : per;
}

}  // namespace

void router_grad_tc_layout(int64_t T, int64_t E, int64_t H, Carver& c, RouterGradWs& w) {
  w.parts = c.take<uint16_t>(parts_size(T, (int)E));
  w.w_parts = c.take<uint16_t>(3 * w_rows((int)E) * H);
  const int64_t s = ceil_div(T, stretch(T, E, H));
  w.g_part = c.take<float>(s > 1 ? s * E * H : 1);
}

usaf_status router_grad_tc(const RouterGradArgs& a, const RouterGradWs& ws, cudaStream_t st) {
  const int E = (int)a.E, H = (int)a.H, ke = w_rows(E);
  __nv_bfloat16* parts = static_cast<__nv_bfloat16*>(ws.parts);
  __nv_bfloat16* wparts = static_cast<__nv_bfloat16*>(ws.w_parts);
  {
    USAF_TRACE("router_grad_split", st);
    const int64_t n = split_rows(a.T, E) * (split_cols(E) / 8) + (a.dx ? (int64_t)ke * (H / 8) : 0);
    const int vec = a.ld % 4 == 0 && (reinterpret_cast<uintptr_t>(a.dlogit) & 15) == 0;
    router_grad_split_kernel<<<(unsigned)ceil_div(n, 256), 256, 0, st>>>(
        a.dlogit, a.ld, a.T, E, vec, parts, a.dx ? a.w_router : nullptr, H, wparts);
    USAF_CHECK_LAUNCH();
  }
  const int64_t per = stretch(a.T, E, H), splits = ceil_div(a.T, per);
  if (a.g_router) {
    CUtensorMap d, x;
    // x as (64 features, token, group of 64 features)
    const uint64_t dims[3] = {64, (uint64_t)a.T, (uint64_t)H / 64}, pitch[2] = {(uint64_t)H * 2, 128};
    const uint32_t box[3] = {64, gw::BK, gw::N / 64};
    if (!map_parts(&d, parts, a.T, E, 3 * halves(E), gw::BK) ||
        !map_bf16(&x, a.x, 3, dims, pitch, box))
      return USAF_ERR_CUDA;
    gw::Params p{};
    p.T = a.T;
    p.E = E;
    p.H = H;
    p.per_split = per;
    p.g_in = a.g_in;
    p.whole = splits == 1;
    p.out = p.whole ? a.g_router : ws.g_part;
    p.status = a.status;
    const dim3 grid((unsigned)ceil_div(H, gw::N), (unsigned)ceil_div(E, 128), (unsigned)splits);
    // three parts fit the 128 rows of one A
    USAF_TRY(side_by_side(E) ? launch_w<true>(d, x, p, grid, st) : launch_w<false>(d, x, p, grid, st));
  }
  const bool sum = a.g_router && splits > 1;
  if (!a.dx) {
    if (!sum) return USAF_OK;
    USAF_TRACE("router_grad_sum", st);
    return launch_dep(router_grad_sum_kernel, dim3(grid_dim_for(a.E * a.H / 4)), 256, 0, st,
                      ws.g_part, (int)splits, a.E * a.H, a.g_in, a.g_router, a.status);
  }
  CUtensorMap d, w, in, out;
  const uint32_t wrows = ke <= gx::MAX_RES ? ke : gx::KB;
  const int64_t groups = ceil_div(H, gx::NH), tiles = ceil_div(a.T, gx::TM);
  if (!map_parts(&d, parts, a.T, E, 1, gx::TM) ||
      !map_bf16_2d(&w, wparts, H, 3 * ke, 64, wrows) ||
      !map_bf16_2d(&out, a.dx, H, a.T, 64, gx::TM) ||
      !map_bf16_2d(&in, a.dx_in ? a.dx_in : a.dx, H, a.T, 64, gx::TM))
    return USAF_ERR_CUDA;
  gx::Params p{};
  p.T = a.T;
  p.E = E;
  p.H = H;
  p.ke = ke;
  p.ring = gx::ring(ke);
  p.slots = gx::slots(ke);
  p.add = a.dx_in != nullptr;
  p.status = a.status;
  p.sum = sum ? ws.g_part : nullptr;
  p.splits = (int)splits;
  p.g_in = a.g_in;
  p.g_router = a.g_router;
  int64_t most = device_sm_count() / groups;
  if (most < 1) most = 1;
  p.per_group = (int)(most < tiles ? most : tiles);
  const unsigned grid = (unsigned)(groups * p.per_group);
  if (stacked(E)) return launch_x<true, true>(d, w, in, out, p, grid, st);
  return ke <= gx::MAX_RES ? launch_x<true, false>(d, w, in, out, p, grid, st)
                           : launch_x<false, false>(d, w, in, out, p, grid, st);
}

}  // namespace usaf
