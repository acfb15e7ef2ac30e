// The two products of a dense router gradient for bf16 tokens on tcgen05 tensor cores.
//
//   g_router[e, h] = g_in + sum_t dlogit[t, e] x[t, h]     (contraction over tokens)
//   dx[t, h]       = dx_in + sum_e dlogit[t, e] w[e, h]    (contraction over experts)
//
// dlogit and w are fp32; the tensor cores take bf16. Cutting a float to its upper 16 bits and doing
// the same with what is left gives three bf16 numbers whose sum is exactly the float (8 bits each of
// its 24), and a product of two bf16 numbers is exact in fp32. g_router, an fp32 result, uses all
// three parts of dlogit (x is bf16 already). dx is rounded to bf16 at the end, so two parts of
// dlogit and of w (2^-16 each) and three of their four products are enough. The converting warps
// read dlogit as fp32 and write the parts into shared memory in the layout the MMA reads, so no
// split copy ever goes through memory.
#include "tc_ptx.cuh"
#include "train.cuh"

namespace usaf {

using namespace tcx;

namespace {

constexpr int CONV_WARPS = 8;  // converting warps of either kernel; g_router's then run the epilogue

// Eight neighbouring logits' gradients, zero past the experts' end or for a row that is not there.
__device__ __forceinline__ void load8(const float* row, bool in, int e, int E, bool vec,
                                      float (&v)[8]) {
  if (in && vec && e + 8 <= E) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(row + e));
    const float4 b = __ldg(reinterpret_cast<const float4*>(row + e + 4));
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = in && e + i < E ? __ldg(row + e + i) : 0.f;
  }
}
// The next truncated part of eight values; they become what it leaves.
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
__device__ __forceinline__ uint4 round_part(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// ------------------------------------------------------------------------------ g_router
// A CTA owns 128 expert rows (M) by 256 features (N) over one part of the tokens (K).
// A = dlogit's parts, 64 tokens x 128 experts each, experts contiguous (MN-major); B = x boxes of 64
// features x 64 tokens by TMA (MN-major). Routers of at most 40 experts put the three parts side by
// side into one 128-row A (STACK): one MMA instead of three, the rows added in the epilogue.
// Otherwise the leading parts' products and the smaller ones have accumulators of their own.
namespace gw {
constexpr int BK = 64;
constexpr int N = 256;
constexpr int PART_BYTES = 128 * BK * 2;
constexpr int BOX_BYTES = 64 * BK * 2;
constexpr int B_BYTES = 4 * BOX_BYTES;
constexpr int NA = 2;
constexpr int OUT_PITCH = N + 4;  // floats per row of the tile in the epilogue
constexpr int THREADS = 64 + 32 * CONV_WARPS;
template <bool STACK>
struct Cfg {
  static constexpr int PARTS = STACK ? 1 : 3;
  static constexpr int NB = STACK ? 5 : 3;
  static constexpr int A_BYTES = PARTS * PART_BYTES;
  static constexpr int RING = NA * A_BYTES + NB * B_BYTES;
  static constexpr int SMEM = RING + 1024 + 256;
  static_assert(128 * OUT_PITCH * 4 <= RING, "output tile in the rings");
  static_assert(SMEM <= 232448, "shared memory");
};
struct Params {
  int64_t T, ld;
  int E, H;
  int64_t per_split;
  const float* dl;
  const float* g_in;
  float* out;      // g_router, or the parts' sums [splits][E][H]
  int whole;       // one split: out is g_router
  int vec;         // dlogit's rows allow 16-byte loads
  uint32_t* status;
};
}  // namespace gw

template <bool STACK>
__global__ void __launch_bounds__(gw::THREADS, 1)
    router_grad_w_tc_kernel(const __grid_constant__ CUtensorMap tm_x, const gw::Params p) {
  using C = gw::Cfg<STACK>;
  using namespace gw;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + NA * C::A_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::RING);
  // fullA[NA], emptyA[NA], fullB[NB], emptyB[NB], done
  const uint32_t fullA = smem_u32(bars), emptyA = fullA + 8 * NA, fullB = emptyA + 8 * NA,
                 emptyB = fullB + 8 * C::NB, done = emptyB + 8 * C::NB;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * NA + 2 * C::NB + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  constexpr uint32_t COLS = STACK ? N : 2 * N;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int h0 = blockIdx.x * N, e0 = blockIdx.y * 128;
  const int64_t t0 = blockIdx.z * p.per_split;
  const int64_t t1 = min(p.T, t0 + p.per_split);
  const int nkb = (int)((t1 - t0 + BK - 1) / BK);
  const int nbox = min(4, (p.H - h0) / 64);
  const int ep = (min(p.E - e0, 128) + 7) / 8 * 8;  // experts of the tile, in whole chunks of 8

  if (threadIdx.x == 0) {
    for (int i = 0; i < NA; ++i) {
      mbar_init(fullA + 8 * i, CONV_WARPS);
      mbar_init(emptyA + 8 * i, 1);
    }
    for (int i = 0; i < C::NB; ++i) {
      mbar_init(fullB + 8 * i, 1);
      mbar_init(emptyB + 8 * i, 1);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), COLS);
  // expert rows that no conversion writes (past the router's end, past the stacked parts) are zero
  if (STACK || ep < 128)
    for (int i = threadIdx.x; i < NA * C::A_BYTES / 16; i += THREADS)
      reinterpret_cast<uint4*>(sA)[i] = make_uint4(0, 0, 0, 0);
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    if (lane == 0) {  // ------------------------------------------------ x boxes
      int issued = 0;
      bool ok = true;
      for (int kb = 0; kb < nkb; ++kb) {
        const int s = kb % C::NB;
        ok = mbar_wait(emptyB + 8 * s, ((kb / C::NB) & 1) ^ 1, abort_flag);
        if (!ok) break;
        mbar_expect_tx(fullB + 8 * s, nbox * BOX_BYTES);
        for (int b = 0; b < nbox; ++b)
          tma_load_2d(smem_u32(sB + s * B_BYTES + b * BOX_BYTES), &tm_x, fullB + 8 * s,
                      h0 + 64 * b, (int)(t0 + (int64_t)kb * BK));
        ++issued;
      }
      if (!ok) *abort_flag = 1;
      const long long deadline = clock64() + TIMEOUT_CYCLES;  // every copy lands before the end
      for (int s = 0; s < C::NB && s < issued; ++s) {
        const int last = issued - 1 - ((issued - 1 - s) % C::NB);
        mbar_drain(fullB + 8 * s, (last / C::NB) & 1, deadline);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {  // ------------------------------------------------ MMAs
      const uint32_t idesc = idesc_bf16(64 * nbox, true, true);
      const uint64_t ad0 = sdesc(smem_u32(sA), 8192, 1024);
      const uint64_t bd0 = sdesc(smem_u32(sB), BOX_BYTES, 1024);
      bool ok = true;
      for (int kb = 0; kb < nkb; ++kb) {
        const int sa = kb % NA, sb = kb % C::NB;
        ok = mbar_wait(fullA + 8 * sa, (kb / NA) & 1, abort_flag) &&
             mbar_wait(fullB + 8 * sb, (kb / C::NB) & 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint64_t a = ad0 + ((sa * C::A_BYTES) >> 4), b = bd0 + ((sb * B_BYTES) >> 4);
#pragma unroll
        for (int part = 0; part < C::PARTS; ++part)
#pragma unroll
          for (int ks = 0; ks < BK / 16; ++ks)
            umma_bf16(tmem + (part ? N : 0), a + ((part * PART_BYTES + ks * 2048) >> 4),
                      b + ((ks * 2048) >> 4), idesc,
                      kb > 0 || ks > 0 || part == 2 ? 1u : 0u);
        umma_commit(emptyA + 8 * sa);
        umma_commit(emptyB + 8 * sb);
      }
      if (!ok) *abort_flag = 1;
      umma_commit(done);
      mbar_drain(done, 0, clock64() + TIMEOUT_CYCLES);
    }
  } else {  // ---------------------------------------------------- parts of dlogit
    const int ct = threadIdx.x - 64;
    const int chunks = ep / 8;                  // chunks of eight experts per token
    const int per = (BK * chunks + 255) / 256;  // chunks per thread, at most 4
    float v[4][8];
    auto load = [&](int kb) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = ct + 256 * u;
        if (u >= per || i >= BK * chunks) continue;
        const int tk = i / chunks, c = i - tk * chunks;
        const int64_t t = t0 + (int64_t)kb * BK + tk;
        load8(p.dl + t * p.ld, t < t1, e0 + 8 * c, p.E, p.vec != 0, v[u]);
      }
    };
    bool ok = true;
    if (nkb > 0) load(0);
    for (int kb = 0; kb < nkb; ++kb) {
      const int sa = kb % NA;
      ok = mbar_wait_warp(emptyA + 8 * sa, ((kb / NA) & 1) ^ 1, abort_flag);
      if (!ok) break;
      uint8_t* a = sA + sa * C::A_BYTES;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = ct + 256 * u;
        if (u >= per || i >= BK * chunks) continue;
        const int tk = i / chunks, c = i - tk * chunks;
#pragma unroll
        for (int part = 0; part < 3; ++part) {
          // chunk of the 128 rows; 64 rows to a box, the chunk's place swizzled by the token
          const int m = STACK ? c + part * chunks : c;
          uint8_t* dst = a + (STACK ? 0 : part * PART_BYTES) + (m >> 3) * 8192 + tk * 128 +
                         (((m & 7) ^ (tk & 7)) << 4);
          *reinterpret_cast<uint4*>(dst) = take_part(v[u]);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(fullA + 8 * sa);
      if (kb + 1 < nkb) load(kb + 1);
    }
    // ---------------------------------------------------------------- epilogue
    // tensor memory -> the rings (free after the last MMA) -> whole rows of global memory
    float* tile = reinterpret_cast<float*>(smem);
    const int q = warp & 3, half = (warp - 2) >> 2;
    const int row = q * 32 + lane;
    if (ok) ok = mbar_wait_warp(done, 0, abort_flag);
    if (ok && *abort_flag == 0) {
      tc_fence_after();
      const int rows = STACK ? 3 * ep : ep;
      for (int ch = half * 4; ch < half * 4 + 4; ++ch) {
        if (ch * 32 >= nbox * 64) break;
        if (q * 32 < rows) {
          float d[32];
          const uint32_t ta = tmem + ((uint32_t)(q * 32) << 16) + ch * 32;
          tmem_ld32(ta, d);
          if constexpr (!STACK) {
            float lo[32];
            tmem_ld32(ta + N, lo);
#pragma unroll
            for (int j = 0; j < 32; ++j) d[j] += lo[j];
          }
          float4* dst = reinterpret_cast<float4*>(tile + row * OUT_PITCH + ch * 32);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            dst[j] = make_float4(d[4 * j], d[4 * j + 1], d[4 * j + 2], d[4 * j + 3]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    if (threadIdx.x == 0) flag_status(p.status, USAF_DEV_TIMEOUT);
  } else {
    const float* tile = reinterpret_cast<const float*>(smem);
    const int ne = min(p.E - e0, 128), w4 = nbox * 16;
    float* out = p.whole ? p.out : p.out + blockIdx.z * (int64_t)p.E * p.H;
    bool bad = false;
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
      const int64_t o = (int64_t)(e0 + e) * p.H + h0 + c;
      float r[4] = {a.x, a.y, a.z, a.w};
      if (p.whole) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (p.g_in) r[j] += p.g_in[o + j];
          bad |= !finite_f(r[j]);
          out[o + j] = r[j];
        }
      } else {
        *reinterpret_cast<float4*>(out + o) = make_float4(r[0], r[1], r[2], r[3]);
      }
    }
    flag_status_warp(p.status, bad, USAF_DEV_NONFINITE);
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_free(tmem, COLS);
  }
}

// ------------------------------------------------------------------------------ dx
// A CTA keeps the router's columns [h0, h0 + 128) in shared memory, two bf16 parts, and walks token
// tiles of 128: A = dlogit's two parts (K-major, 64 experts a block) through a ring, accumulators in
// tensor memory, twice. dx_in comes and dx goes by TMA through a ring of 128 x 64 boxes in which the
// epilogue adds: the token rows are read and written in whole lines while the next tile converts.
namespace gx {
constexpr int TM = 128;      // tokens of a tile
constexpr int NH = 128;      // features of a CTA
constexpr int KB = 64;       // experts of an A block
constexpr int A_PART = TM * KB * 2;
constexpr int A_BYTES = 2 * A_PART;
constexpr int NA = 2;
constexpr int BOX = TM * 64 * 2;
constexpr int MAX_E = 256;
constexpr int MAX_SLOTS = 6;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 64 + 32 * (EPI_WARPS + CONV_WARPS);
constexpr int SMEM_MAX = 232448;
// bytes of the router's two parts for ke experts (a multiple of 16): two groups of 64 features
__host__ __device__ constexpr int b_bytes(int ke) { return 2 * 2 * ke * 128; }
__host__ __device__ constexpr int slots(int ke) {
  const int s = (SMEM_MAX - 1024 - 512 - NA * A_BYTES - b_bytes(ke)) / BOX;
  return s < MAX_SLOTS ? s : MAX_SLOTS;
}
static_assert(slots(MAX_E) >= 2, "staging for one tile");
struct Params {
  int64_t T, ld;
  int E, H, ke;
  int slots;
  int per_group;   // CTAs that share a feature group
  const float* dl;
  const float* w;
  int add;         // dx_in is there
  int vec;
  uint32_t* status;
};
}  // namespace gx

__global__ void __launch_bounds__(gx::THREADS, 1)
    router_grad_x_tc_kernel(const __grid_constant__ CUtensorMap tm_in,
                            const __grid_constant__ CUtensorMap tm_out, const gx::Params p) {
  using namespace gx;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int ke = p.ke, NS = p.slots;
  uint8_t* sA = smem;
  uint8_t* sStage = smem + NA * A_BYTES;
  uint8_t* sB = sStage + NS * BOX;  // [part][feature group of 64][expert][64 features]
  uint64_t* bars = reinterpret_cast<uint64_t*>(sB + b_bytes(ke));
  // fullA[NA], emptyA[NA], tfull[2], tempty[2], loaded[NS], added[NS], freed[NS], done
  const uint32_t fullA = smem_u32(bars), emptyA = fullA + 8 * NA, tfull = emptyA + 8 * NA,
                 tempty = tfull + 16, loaded = tempty + 16, added = loaded + 8 * MAX_SLOTS,
                 freed = added + 8 * MAX_SLOTS, done = freed + 8 * MAX_SLOTS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * NA + 4 + 3 * MAX_SLOTS + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  constexpr uint32_t COLS = 2 * NH;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int groups = gridDim.x / p.per_group;
  const int h0 = (blockIdx.x % groups) * NH;
  const int first = blockIdx.x / groups;
  const int tiles = (int)((p.T + TM - 1) / TM);
  const int nbox = min(2, (p.H - h0) / 64);
  const int nkb = (ke + KB - 1) / KB;
  const int part_b = 2 * ke * 128;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NA; ++i) {
      mbar_init(fullA + 8 * i, CONV_WARPS);
      mbar_init(emptyA + 8 * i, 1);
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
    *abort_flag = 0;
    mbar_init_fence();
  }
  if (warp == 1) tmem_alloc(smem_u32(tmem_slot), COLS);
  // the router's columns: expert row of 128 bytes (64 features), 16-byte chunks swizzled by the row
  for (int i = threadIdx.x; i < ke * 16; i += THREADS) {
    const int e = i >> 4, c = i & 15;
    float v[8];
    const int h = h0 + 8 * c;
    if (e < p.E && h < p.H) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(p.w + (int64_t)e * p.H + h));
      const float4 b = __ldg(reinterpret_cast<const float4*>(p.w + (int64_t)e * p.H + h + 4));
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
      v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.f;
    }
    uint8_t* dst = sB + (c >> 3) * ke * 128 + e * 128 + (((c & 7) ^ (e & 7)) << 4);
    *reinterpret_cast<uint4*>(dst) = take_part(v);
    *reinterpret_cast<uint4*>(dst + part_b) = round_part(v);
  }
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  bool bad = false;

  if (warp == 0) {
    if (lane == 0) {  // ------------------------------------------------ dx_in boxes
      int u = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += p.per_group)
        for (int b = 0; b < nbox && ok; ++b, ++u) {
          const int s = u % NS;
          ok = mbar_wait(freed + 8 * s, ((u / NS) & 1) ^ 1, abort_flag);
          if (!ok) break;
          if (p.add) {
            mbar_expect_tx(loaded + 8 * s, BOX);
            tma_load_2d(smem_u32(sStage + s * BOX), &tm_in, loaded + 8 * s, h0 + 64 * b, t * TM);
          } else {
            mbar_arrive(loaded + 8 * s);
          }
        }
      if (!ok) *abort_flag = 1;
      const int issued = u;  // boxes 0 .. u - 1
      const long long deadline = clock64() + TIMEOUT_CYCLES;
      for (int s = 0; s < NS && s < issued; ++s) {
        const int last = issued - 1 - ((issued - 1 - s) % NS);
        mbar_drain(loaded + 8 * s, (last / NS) & 1, deadline);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {  // ------------------------------------------------ MMAs
      const uint32_t idesc = idesc_bf16(64 * nbox, false, true);
      const uint64_t ad0 = sdesc(smem_u32(sA), 16, 1024);
      const uint64_t bd0 = sdesc(smem_u32(sB), ke * 128, 1024);
      int n = 0, kc = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += p.per_group, ++n) {
        ok = mbar_wait(tempty + 8 * (n & 1), ((n >> 1) & 1) ^ 1, abort_flag);
        if (!ok) break;
        const uint32_t d = tmem + (n & 1) * NH;
        for (int kb = 0; kb < nkb; ++kb, ++kc) {
          const int sa = kc % NA;
          ok = mbar_wait(fullA + 8 * sa, (kc / NA) & 1, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint64_t a = ad0 + ((sa * A_BYTES) >> 4);
          const int steps = min(KB / 16, ke / 16 - kb * (KB / 16));
          for (int ks = 0; ks < steps; ++ks) {
            const uint64_t ah = a + ((ks * 32) >> 4), am = ah + (A_PART >> 4);
            const uint64_t bh = bd0 + (((kb * 4 + ks) * 2048) >> 4), bm = bh + (part_b >> 4);
            umma_bf16(d, ah, bh, idesc, kb > 0 || ks > 0 ? 1u : 0u);
            umma_bf16(d, ah, bm, idesc, 1u);
            umma_bf16(d, am, bh, idesc, 1u);
          }
          umma_commit(emptyA + 8 * sa);
        }
        if (ok) umma_commit(tfull + 8 * (n & 1));
      }
      if (!ok) *abort_flag = 1;
      umma_commit(done);
      mbar_drain(done, 0, clock64() + TIMEOUT_CYCLES);
    }
  } else if (warp < 2 + EPI_WARPS) {  // ------------------------- epilogue: add and store
    const int q = warp & 3, b = (warp - 2) >> 2;  // lanes' quarter, box of the tile
    const bool issuer = ((warp - 2) & 3) == 0 && lane == 0;
    const int row = q * 32 + lane;
    if (b < nbox) {
      int n = 0;
      for (int t = first; t < tiles; t += p.per_group, ++n) {
        const int u = n * nbox + b, s = u % NS;
        const uint32_t ph = (u / NS) & 1;
        if (!mbar_wait_warp(loaded + 8 * s, ph, abort_flag)) break;
        if (!mbar_wait_warp(tfull + 8 * (n & 1), (n >> 1) & 1, abort_flag)) break;
        tc_fence_after();
        const bool live = (int64_t)t * TM + row < p.T;
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
            for (int j = 0; j < 8; ++j) bad |= live && !finite_f(d[8 * c + j]);
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
  } else {  // ---------------------------------------------------- dlogit's parts
    const int ct = threadIdx.x - 64 - 32 * EPI_WARPS;
    // 128 tokens x 8 chunks of eight experts: four a thread
    float v[4][8];
    auto load = [&](int t, int kb) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = ct + 256 * u, tk = i >> 3, c = i & 7;
        const int64_t tok = (int64_t)t * TM + tk;
        const int e = kb * KB + 8 * c;
        if (e < ke) load8(p.dl + tok * p.ld, tok < p.T, e, p.E, p.vec != 0, v[u]);
      }
    };
    int kc = 0;
    bool ok = true;
    if (first < tiles) load(first, 0);
    for (int t = first; t < tiles && ok; t += p.per_group)
      for (int kb = 0; kb < nkb; ++kb, ++kc) {
        const int sa = kc % NA;
        ok = mbar_wait_warp(emptyA + 8 * sa, ((kc / NA) & 1) ^ 1, abort_flag);
        if (!ok) break;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = ct + 256 * u, tk = i >> 3, c = i & 7;
          if (kb * KB + 8 * c >= ke) continue;
          uint8_t* dst = sA + sa * A_BYTES + tk * 128 + ((c ^ (tk & 7)) << 4);
          *reinterpret_cast<uint4*>(dst) = take_part(v[u]);
          *reinterpret_cast<uint4*>(dst + A_PART) = round_part(v[u]);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(fullA + 8 * sa);
        if (kb + 1 < nkb) load(t, kb + 1);
        else if (t + p.per_group < tiles) load(t + p.per_group, 0);
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

bool rows_vec(const RouterGradArgs& a) {
  return a.ld % 4 == 0 && (reinterpret_cast<uintptr_t>(a.dlogit) & 15) == 0;
}

template <bool STACK>
usaf_status launch_w(const CUtensorMap& tm, const gw::Params& p, dim3 grid, cudaStream_t st) {
  USAF_TRACE("router_grad_w", st);
  using C = gw::Cfg<STACK>;
  if (cudaFuncSetAttribute(router_grad_w_tc_kernel<STACK>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
    return USAF_ERR_CUDA;
  router_grad_w_tc_kernel<STACK><<<grid, gw::THREADS, C::SMEM, st>>>(tm, p);
  USAF_CHECK_LAUNCH();
  return USAF_OK;
}

}  // namespace

// Tokens of a split of g_router's sum: about one CTA per SM, whole blocks of 64 tokens, at least two.
int64_t router_grad_tc_split(int64_t T, int64_t E, int64_t H) {
  const int64_t tiles = ceil_div(H, gw::N) * ceil_div(E, 128);
  const int64_t s = tiles < 152 ? 152 / tiles : 1;
  const int64_t per = round_up(ceil_div(T, s), gw::BK);
  return per < 2 * gw::BK ? 2 * gw::BK : per;
}

usaf_status router_grad_w_tc(const RouterGradArgs& a, float* part, int64_t per_split,
                             cudaStream_t st) {
  CUtensorMap tm;
  if (!map_bf16_2d(&tm, a.x, a.H, a.T, 64, gw::BK)) return USAF_ERR_CUDA;
  const int64_t splits = ceil_div(a.T, per_split);
  gw::Params p{};
  p.T = a.T;
  p.ld = a.ld;
  p.E = (int)a.E;
  p.H = (int)a.H;
  p.per_split = per_split;
  p.dl = a.dlogit;
  p.g_in = a.g_in;
  p.whole = splits == 1;
  p.out = p.whole ? a.g_router : part;
  p.vec = rows_vec(a);
  p.status = a.status;
  const dim3 grid((unsigned)ceil_div(a.H, gw::N), (unsigned)ceil_div(a.E, 128), (unsigned)splits);
  // three parts of round_up(E, 8) rows fit the 128 of one A
  return round_up(a.E, 8) <= 40 ? launch_w<true>(tm, p, grid, st) : launch_w<false>(tm, p, grid, st);
}

bool router_grad_x_tc_ok(int64_t E) { return E <= gx::MAX_E; }

usaf_status router_grad_x_tc(const RouterGradArgs& a, cudaStream_t st) {
  USAF_TRACE("router_grad_x", st);
  CUtensorMap in, out;
  if (!map_bf16_2d(&out, a.dx, a.H, a.T, 64, gx::TM) ||
      !map_bf16_2d(&in, a.dx_in ? a.dx_in : a.dx, a.H, a.T, 64, gx::TM))
    return USAF_ERR_CUDA;
  gx::Params p{};
  p.T = a.T;
  p.ld = a.ld;
  p.E = (int)a.E;
  p.H = (int)a.H;
  p.ke = (int)round_up(a.E, 16);
  p.slots = gx::slots(p.ke);
  p.dl = a.dlogit;
  p.w = a.w_router;
  p.add = a.dx_in != nullptr;
  p.vec = rows_vec(a);
  p.status = a.status;
  const int64_t groups = ceil_div(a.H, gx::NH), tiles = ceil_div(a.T, gx::TM);
  int64_t per = device_sm_count() / groups;
  if (per < 1) per = 1;
  if (per > tiles) per = tiles;
  p.per_group = (int)per;
  const int smem = gx::NA * gx::A_BYTES + p.slots * gx::BOX + gx::b_bytes(p.ke) + 1024 + 512;
  if (cudaFuncSetAttribute(router_grad_x_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           gx::SMEM_MAX) != cudaSuccess)
    return USAF_ERR_CUDA;
  router_grad_x_tc_kernel<<<(unsigned)(groups * per), gx::THREADS, smem, st>>>(in, out, p);
  USAF_CHECK_LAUNCH();
  return USAF_OK;
}

}  // namespace usaf
