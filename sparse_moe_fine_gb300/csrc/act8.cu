// Activations in 8 bits between a layer's forward and its backward (usaf_act8_save / _restore):
// blocks of 16 values share a power-of-two scale, so that coding and decoding are exact up to the
// one rounding of each code, and every decoded value is a bf16 number (a code has 7 bits).
//
// Both directions are bound by memory traffic: every value is read once and written once, whole
// 16-byte vectors a lane, neighbouring lanes neighbouring vectors. The arithmetic stays at a few
// instructions a value by two uses of fp32's exact integers: adding 1.5 * 2^23 leaves a rounded
// (to nearest even) code in the low byte, and a code byte put into 2^23's mantissa is the code plus
// a constant.
//
// Blocks of 16 with a power of two: on Gaussian values int8 codes are off by 0.73% in norm (0.47%
// with an exact scale, whose codes and values would have to be rounded twice), 8-bit floats of three
// mantissa bits by 2.6%. The exponent byte adds 1/16 to the store.
// Measured (Qwen3-30B-A3B-shaped layer: T 4096, top 8, H 2048, I 768): bf16 save 33 us for 179 MB,
// restore 73 us for 365 MB, of which 302 MB are written; fp32 save 53 us, restore 176 us (297 and 666
// MB). Mixtral-8x7B-shaped (T 8192, I 14336, bf16): both 582 us for 3.69 GB, 93% of the copy rate.
// The small restore is at no rate of the memory (DRAM 58% busy, L2 50%, 1.2 GB of writes go at 4.5 TB/s,
// its 302 MB at 4.1): its gather blocks come first and wait for the rows they gather, and the blocks
// that stream come after them.
#include "tc_ptx.cuh"
#include "train.cuh"

namespace usaf {

namespace {

constexpr int BLK = USAF_ACT8_BLOCK;
constexpr int THREADS = 256;
constexpr float MAX_CODED = 127.f * 2.6584559915698317e36f;  // 127 * 2^121

// exponent byte of a block from its largest magnitude's fp32 bits: amax = m 2^q with 1 <= m < 2 is
// covered by 127 * 2^(q - 6) while m <= 127 / 64; 0 for zeros, 255 for NaN and infinities
__device__ __forceinline__ int exp_byte(uint32_t amax_bits) {
  if (amax_bits == 0) return 0;
  if (amax_bits >= 0x7F800000u) return 255;
  const int b = (int)(amax_bits >> 23) - 6 + ((amax_bits & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
  return b < 1 ? 1 : (b > 248 ? 248 : b);
}
// 2^-(byte - 127), the factor of the codes; 0 for blocks whose codes are 0
__device__ __forceinline__ float code_factor(int byte) {
  return byte == 0 || byte == 255 ? 0.f : __uint_as_float((uint32_t)(254 - byte) << 23);
}
// 2^(byte - 127); 0 for byte 0, infinity (0 times which is NaN) for byte 255
__device__ __forceinline__ float value_factor(int byte) {
  return __uint_as_float((uint32_t)byte << 23);
}

// ------------------------------------------------------------------------------ coding
// v * f rounded to an integer, in the low byte (v * f is exact: f is a power of two)
__device__ __forceinline__ uint32_t code_bits(float v, float f) {
  return __float_as_uint(fmaf(v, f, 12582912.f));
}
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
__device__ __forceinline__ float clamp_coded(float v) {
  return fminf(fmaxf(v, -MAX_CODED), MAX_CODED);
}

template <typename T>
struct Vec;
// 16 bytes: eight bf16 values, half a block (two lanes share it), eight codes
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  using Codes = uint2;
  static __device__ __forceinline__ uint32_t amax(const uint4& r) {
    const uint32_t k = __vmaxu2(__vmaxu2(r.x & 0x7FFF7FFFu, r.y & 0x7FFF7FFFu),
                                __vmaxu2(r.z & 0x7FFF7FFFu, r.w & 0x7FFF7FFFu));
    const uint32_t m = __vmaxu2(k, __shfl_xor_sync(0xffffffffu, k, 1));
    return max(m >> 16, m & 0xFFFFu) << 16;
  }
  template <bool RARE>
  static __device__ __forceinline__ Codes encode(const uint4& r, int byte) {
    const float f = code_factor(byte);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xFFFF0000u);
      if (RARE) lo = clamp_coded(lo), hi = clamp_coded(hi);
      c[2 * i] = code_bits(lo, f);
      c[2 * i + 1] = code_bits(hi, f);
    }
    if (RARE && byte == 255) return make_uint2(0, 0);
    return make_uint2(pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7]));
  }
};
// four fp32 values, a quarter of a block, four codes
template <>
struct Vec<float> {
  static constexpr int N = 4;
  using Codes = uint32_t;
  static __device__ __forceinline__ uint32_t amax(const uint4& r) {
    uint32_t k = max(max(r.x & 0x7FFFFFFFu, r.y & 0x7FFFFFFFu),
                     max(r.z & 0x7FFFFFFFu, r.w & 0x7FFFFFFFu));
    k = max(k, __shfl_xor_sync(0xffffffffu, k, 1));
    return max(k, __shfl_xor_sync(0xffffffffu, k, 2));
  }
  template <bool RARE>
  static __device__ __forceinline__ Codes encode(const uint4& r, int byte) {
    const float f = code_factor(byte);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v = __uint_as_float(w[i]);
      if (RARE) v = clamp_coded(v);
      c[i] = code_bits(v, f);
    }
    return RARE && byte == 255 ? 0u : pack4(c[0], c[1], c[2], c[3]);
  }
};

// The warp's 32 x U vectors of src from vector i0 on, of which those below n are there (n whole
// blocks); every lane takes part. True where a block was not finite. Blocks at the top of fp32's
// range, whose codes have to be clamped, and blocks that are not finite are coded on a path of
// their own: their tests would cost the others a third more instructions.
template <typename T, int U>
__device__ __forceinline__ bool encode_run(const T* src, int64_t i0, int64_t n, int8_t* code,
                                           uint8_t* ex) {
  using V = Vec<T>;
  using Codes = typename V::Codes;
  constexpr int LB = BLK / V::N;
  const int lane = threadIdx.x & 31;
  const int left = (int)min((int64_t)(32 * U), n - i0) - lane;  // vector 32 u + lane is there
  const uint4* from = reinterpret_cast<const uint4*>(src) + i0 + lane;
  Codes* to = reinterpret_cast<Codes*>(code) + i0 + lane;
  uint8_t* eto = ex + (i0 + lane) / LB;
  uint4 r[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    r[u] = 32 * u < left ? __ldg(from + 32 * u) : make_uint4(0, 0, 0, 0);
  int b[U];
  int top = 0;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    b[u] = exp_byte(V::amax(r[u]));
    top = max(top, b[u]);
  }
  const bool rare = __any_sync(0xffffffffu, top >= 248);
#pragma unroll
  for (int u = 0; u < U; ++u) {
    Codes c;
    if (!rare) c = V::template encode<false>(r[u], b[u]);
    else c = V::template encode<true>(r[u], b[u]);
    if (32 * u < left) {
      to[32 * u] = c;
      if (lane % LB == 0) eto[32 / LB * u] = (uint8_t)b[u];
    }
  }
  return top == 255;
}

// One block of n <= 16 values, a thread each: rows whose length is not a multiple of 16.
template <typename T>
__device__ __forceinline__ bool encode_block(const T* src, int n, int8_t* code, uint8_t* ex) {
  float v[BLK];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < BLK; ++i) {
    v[i] = i < n ? to_f32(src[i]) : 0.f;
    amax = max(amax, abs_key(v[i]));
  }
  const int b = exp_byte(amax);
  const float f = code_factor(b);
#pragma unroll
  for (int i = 0; i < BLK; ++i)
    if (i < n) code[i] = b == 255 ? (int8_t)0 : (int8_t)code_bits(clamp_coded(v[i]), f);
  *ex = (uint8_t)b;
  return b == 255;
}

constexpr int SAVE_U = 4;  // vectors of a lane in flight

// A warp per run of a feature's rows, all blocks the machine holds at once: 34 us for 117 MB in and
// 62 MB out on the Qwen3-shaped layer (issue slots 67% busy, DRAM 60%).

template <typename T>
__global__ void __launch_bounds__(THREADS)
    act8_save_kernel(const Act8Args a, const T* __restrict__ x, const T* __restrict__ h,
                     uint32_t* status) {
  constexpr int VW = Vec<T>::N, RUN = 32 * SAVE_U;  // vectors of a warp's run
  const int64_t warps = (int64_t)gridDim.x * (THREADS / 32);
  const int64_t wg = (int64_t)blockIdx.x * (THREADS / 32) + threadIdx.x / 32;
  bool bad = false;
  // h: each feature's rows that experts own, in runs
  const int64_t nv = a.rt.expert_offset[a.s.E] / VW, pitch = a.R_cap / BLK;
  const int64_t runs = (nv + RUN - 1) / RUN;
  for (int64_t i = wg; i < 2 * a.s.I * runs; i += warps) {
    const int64_t j = i / runs, r = i - j * runs;
    bad |= encode_run<T, SAVE_U>(h + j * a.R_cap, r * RUN, nv, a.h_code + j * a.R_cap,
                                 a.h_exp + j * pitch);
  }
  // x: tokens of whole blocks are one run of vectors
  if (a.s.H % BLK == 0) {
    const int64_t n = a.s.T * a.s.H / VW;
    for (int64_t i = wg * RUN; i < n; i += warps * RUN)
      bad |= encode_run<T, SAVE_U>(x, i, n, a.x_code, a.x_exp);
  } else {
    const int64_t nbx = (a.s.H + BLK - 1) / BLK;
    for (int64_t i = (int64_t)blockIdx.x * THREADS + threadIdx.x; i < a.s.T * nbx;
         i += (int64_t)gridDim.x * THREADS) {
      const int64_t t = i / nbx, b = i - t * nbx;
      const int64_t o = t * a.s.H + b * BLK;
      bad |= encode_block(x + o, (int)min((int64_t)BLK, a.s.H - b * BLK), a.x_code + o,
                          a.x_exp + i);
    }
  }
  flag_status_warp(status, bad, USAF_DEV_NONFINITE);
}

// ------------------------------------------------------------------------------ decoding
// the four codes of a word as floats: byte q ^ 0x80 in the mantissa of 2^23 is 2^23 + 128 + code
__device__ __forceinline__ void decode4(uint32_t w, float s, float* v) {
  const uint32_t u = w ^ 0x80808080u;
  v[0] = (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7440)) - 8388736.f) * s;
  v[1] = (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7441)) - 8388736.f) * s;
  v[2] = (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7442)) - 8388736.f) * s;
  v[3] = (__uint_as_float(__byte_perm(u, 0x4B000000u, 0x7443)) - 8388736.f) * s;
}
template <typename T>
__device__ __forceinline__ void decode(const typename Vec<T>::Codes& c, float s,
                                       float (&v)[Vec<T>::N]) {
  if constexpr (Vec<T>::N == 8) {
    decode4(c.x, s, v);
    decode4(c.y, s, v + 4);
  } else {
    decode4(c, s, v);
  }
}
template <typename T>
__device__ __forceinline__ uint4 to_vec(const float (&v)[Vec<T>::N]) {
  if constexpr (Vec<T>::N == 8) {
    return make_uint4(tcx::pack_bf16x2(v[0], v[1]), tcx::pack_bf16x2(v[2], v[3]),
                      tcx::pack_bf16x2(v[4], v[5]), tcx::pack_bf16x2(v[6], v[7]));
  } else {
    return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                      __float_as_uint(v[3]));
  }
}

// silu by exp(-|g|), which does not overflow: far negative gates keep their tiny values. bf16
// results are rounded to 8 bits (2^-9), so the fast exponential and quotient serve them: the first is
// documented to 2 + 1.17 |g| units of 2^-23, below 2^-16 for |g| up to 87, where the result leaves
// fp32's normal numbers; the second to 2 units.
template <typename T>
__device__ __forceinline__ float silu_tail(float g) {
  if constexpr (sizeof(T) == 2) {
    const float e = __expf(-fabsf(g));
    return g * (g >= 0.f ? 1.f : e) * __fdividef(1.f, 1.f + e);
  } else {
    const float e = expf(-fabsf(g));
    return g * (g >= 0.f ? 1.f : e) / (1.f + e);
  }
}

// Rows [seg, seg + 32 vectors) of up to 64 features from feature `f0` on, one warp a feature: h
// decoded, wa formed again. The lanes' routing weights stay in registers over the features. With x:
// 43 us for 226 MB (Qwen3-shaped layer), 5.3 TB/s.
constexpr int ROW_FEATURES = 64;  // features of a block: eight per warp
template <typename T>
__device__ __forceinline__ void restore_rows(const Act8Args& a, int64_t seg, int64_t f0, T* h,
                                             T* wa) {
  using V = Vec<T>;
  constexpr int VW = V::N;
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int64_t rows = a.rt.expert_offset[a.s.E], r = seg + lane * VW;
  if (seg >= rows) return;
  const bool in = r < rows;  // rows is a multiple of 16: a vector is whole or not there
  float w[VW];
#pragma unroll
  for (int q = 0; q < VW; q += 4) {
    const int4 sl = in ? *reinterpret_cast<const int4*>(a.rt.perm_slot + r + q)
                       : make_int4(-1, -1, -1, -1);
    w[q] = sl.x >= 0 ? a.rt.topk_w[sl.x] : 0.f;
    w[q + 1] = sl.y >= 0 ? a.rt.topk_w[sl.y] : 0.f;
    w[q + 2] = sl.z >= 0 ? a.rt.topk_w[sl.z] : 0.f;
    w[q + 3] = sl.w >= 0 ? a.rt.topk_w[sl.w] : 0.f;
  }
  if (!in) return;
  using Codes = typename V::Codes;
  constexpr int U = 2;  // features of a warp in flight (1 and 4: 9% and 13% slower)
  // the lane's places in the gate's row of this warp's first feature
  const int fw = __shfl_sync(__activemask(), wid, 0);
  const int64_t i0 = f0 + fw, pitch = a.R_cap / BLK;
  const int8_t* gc = a.h_code + i0 * a.R_cap + r;
  const uint8_t* ge = a.h_exp + i0 * pitch + r / BLK;
  T* gh = h + i0 * a.R_cap + r;
  T* gw = wa + i0 * a.R_cap + r;
  const int64_t up_c = a.s.I * a.R_cap, up_e = a.s.I * pitch;
  const int nf = (int)min((int64_t)ROW_FEATURES, a.s.I - f0);
#pragma unroll 1
  for (int f = fw; f < nf; f += 8 * U) {
    Codes cg[U], cu[U];
    int sg[U], su[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (f + 8 * u >= nf) break;
      cg[u] = __ldg(reinterpret_cast<const Codes*>(gc + 8 * u * a.R_cap));
      cu[u] = __ldg(reinterpret_cast<const Codes*>(gc + 8 * u * a.R_cap + up_c));
      sg[u] = __ldg(ge + 8 * u * pitch);
      su[u] = __ldg(ge + 8 * u * pitch + up_e);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (f + 8 * u >= nf) break;
      float g[VW], up[VW];
      decode<T>(cg[u], value_factor(sg[u]), g);
      *reinterpret_cast<uint4*>(gh + 8 * u * a.R_cap) = to_vec<T>(g);
#pragma unroll
      for (int q = 0; q < VW; ++q) g[q] = w[q] * silu_tail<T>(g[q]);
      decode<T>(cu[u], value_factor(su[u]), up);
      *reinterpret_cast<uint4*>(gh + 8 * u * a.R_cap + up_c) = to_vec<T>(up);
#pragma unroll
      for (int q = 0; q < VW; ++q) g[q] *= up[q];
      *reinterpret_cast<uint4*>(gw + 8 * u * a.R_cap) = to_vec<T>(g);
    }
    gc += 8 * U * a.R_cap;
    ge += 8 * U * pitch;
    gh += 8 * U * a.R_cap;
    gw += 8 * U * a.R_cap;
  }
}

constexpr int X_VECTORS = 4 * THREADS;  // vectors of a block of the decoded x
template <typename T>
__device__ __forceinline__ void restore_x(const Act8Args& a, int64_t blk, T* x) {
  using V = Vec<T>;
  if (a.s.H % BLK == 0) {
    const int64_t n = a.s.T * a.s.H / V::N;
    typename V::Codes c[4];
    float s[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t i = blk * X_VECTORS + u * THREADS + threadIdx.x;
      if (i < n) {
        c[u] = __ldg(reinterpret_cast<const typename V::Codes*>(a.x_code) + i);
        s[u] = value_factor(__ldg(a.x_exp + i / (BLK / V::N)));
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t i = blk * X_VECTORS + u * THREADS + threadIdx.x;
      if (i >= n) break;
      float v[V::N];
      decode<T>(c[u], s[u], v);
      reinterpret_cast<uint4*>(x)[i] = to_vec<T>(v);
    }
  } else {
    const int64_t nbx = (a.s.H + BLK - 1) / BLK, lo = blk * X_VECTORS * V::N;
    const int64_t hi = min(a.s.T * a.s.H, lo + X_VECTORS * V::N);
    constexpr int U = 8;  // loads in flight; 4,000 bf16 tokens, H 1,000: 63.9 us with one, 55.8 with eight
    for (int64_t i0 = lo + threadIdx.x; i0 < hi; i0 += U * THREADS) {
      int code[U], e[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t i = i0 + u * THREADS;
        if (i >= hi) break;
        const int64_t t = i / a.s.H, c = i - t * a.s.H;
        code[u] = __ldg(a.x_code + i);
        e[u] = __ldg(a.x_exp + t * nbx + c / BLK);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t i = i0 + u * THREADS;
        if (i >= hi) break;
        x[i] = from_f32<T>((float)code[u] * value_factor(e[u]));
      }
    }
  }
}

// x_perm[f, row] = the decoded x of the row's token, 0 in padding and tail rows: 256 rows x 64
// features at a time, stored by TMA as four boxes of 64 rows x 64 features. A lane decodes eight rows
// x eight features and packs the transpose as it converts (a bf16 pair is one feature of two rows).
// The eight lanes of a quarter-warp write eight row chunks of one feature, so every 16-byte store
// into the 128-byte swizzled box is free of bank conflicts, and a row's four feature groups are one
// 32-byte sector of codes. A block keeps its rows' tokens over G_STEPS feature tiles; the copy engine
// reads a tile while the next one's codes are on their way. H a multiple of 64. 38 us for 134 MiB
// written (Qwen3-shaped layer); wider and taller tiles were no faster.
constexpr int G_ROWS = 256, G_FEATURES = 64, G_STEPS = 4;
constexpr int G_SMEM = 4 * 8192 + 1024;
__device__ __forceinline__ void gather_bf16(const CUtensorMap& tm, const Act8Args& a, int rb,
                                            int fb0, uint8_t* tile) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
  const int c = lane & 7, box = wid >> 1;
  const int f = (wid & 1) * 32 + (lane >> 3) * 8;  // first feature within the tile's 64
  const int64_t r = (int64_t)rb * G_ROWS + box * 64 + c * 8;
  const int rows = a.rt.expert_offset[a.s.E], H = (int)a.s.H;
  uint32_t at[8];  // the token's first vector of eight codes, NONE without one
  constexpr uint32_t NONE = 0xFFFFFFFFu;
  {
    const int4 t0 = *reinterpret_cast<const int4*>(a.rt.perm_tok + r);
    const int4 t1 = *reinterpret_cast<const int4*>(a.rt.perm_tok + r + 4);
    const int4 s0 = *reinterpret_cast<const int4*>(a.rt.perm_slot + r);
    const int4 s1 = *reinterpret_cast<const int4*>(a.rt.perm_slot + r + 4);
    const int tt[8] = {t0.x, t0.y, t0.z, t0.w, t1.x, t1.y, t1.z, t1.w};
    const int ss[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i)
      at[i] = r < rows && ss[i] >= 0 ? (uint32_t)tt[i] * (uint32_t)(H / 8) : NONE;
  }
  uint8_t* bx = tile + box * 8192 + f * 128;
  const int steps = min(G_STEPS, H / G_FEATURES - fb0);
  const uint2* xc = reinterpret_cast<const uint2*>(a.x_code) + (fb0 * G_FEATURES + f) / 8;
  const uint8_t* xe = a.x_exp + (fb0 * G_FEATURES + f) / BLK;
#pragma unroll 1
  for (int st = 0; st < steps; ++st) {
    uint2 code[8];
    int s[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const bool live = at[i] != NONE;
      code[i] = live ? __ldg(xc + at[i]) : make_uint2(0, 0);
      s[i] = live ? __ldg(xe + (at[i] >> 1)) : 0;  // an exponent per two vectors
    }
    xc += G_FEATURES / 8;
    xe += G_FEATURES / BLK;
    if (st > 0) {  // the last tile has been read out of shared memory
      if (threadIdx.x == 0) tcx::bulk_wait_read();
      __syncthreads();
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {  // four features of the eight rows
      uint32_t out[4][4];                   // [feature][pair of rows]
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        float v0[4], v1[4];
        decode4(half ? code[2 * p].y : code[2 * p].x, value_factor(s[2 * p]), v0);
        decode4(half ? code[2 * p + 1].y : code[2 * p + 1].x, value_factor(s[2 * p + 1]), v1);
#pragma unroll
        for (int k = 0; k < 4; ++k) out[k][p] = tcx::pack_bf16x2(v0[k], v1[k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int fk = half * 4 + k;
        *reinterpret_cast<uint4*>(bx + fk * 128 + ((c ^ fk) << 4)) =
            make_uint4(out[k][0], out[k][1], out[k][2], out[k][3]);
      }
    }
    tcx::fence_async_smem();
    __syncthreads();
    if (threadIdx.x == 0) {
      const uint32_t src = tcx::smem_u32(tile);
      for (int b = 0; b < 4; ++b)
        tcx::tma_store_2d(&tm, src + b * 8192, rb * G_ROWS + b * 64, (fb0 + st) * G_FEATURES);
      tcx::bulk_commit();
    }
  }
  if (threadIdx.x == 0) tcx::bulk_wait();
}

// The same for fp32 tokens and for widths that are no multiple of 64: 128 rows x 64 features through
// shared memory. Each code's address waits on its row's token and each thread has only bytes to load, so
// latency bounds it: the tokens are read once per tile and eight values of a thread are on their way at
// a time (restore of 4,096 fp32 tokens, 128 experts, top 8, H 2,048: 242 us with one at a time, 176 us so).
constexpr int XG_ROWS = 128;
template <typename T>
__global__ void __launch_bounds__(THREADS) act8_gather_kernel(const Act8Args a, T* x_perm) {
  __shared__ T tile[64][XG_ROWS + 1];
  __shared__ int s_tok[XG_ROWS];  // the rows' tokens, -1 without one
  const int64_t r0 = (int64_t)blockIdx.x * XG_ROWS;
  // the widest tokens have more tiles than the second axis may (one axis and a division: 11% slower)
  const int64_t h0 = ((int64_t)blockIdx.z * gridDim.y + blockIdx.y) * 64;
  if (h0 >= a.s.H) return;
  const int64_t end = a.rt.expert_offset[a.s.E], nbx = (a.s.H + BLK - 1) / BLK;
  for (int r = threadIdx.x; r < XG_ROWS; r += THREADS)
    s_tok[r] = r0 + r < end && a.rt.perm_slot[r0 + r] >= 0 ? a.rt.perm_tok[r0 + r] : -1;
  __syncthreads();
  constexpr int U = 8;
  const int f = threadIdx.x % 64;
  const int64_t c = h0 + f;
  for (int r1 = threadIdx.x / 64; r1 < XG_ROWS; r1 += U * (THREADS / 64)) {
    int code[U], e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = s_tok[r1 + u * (THREADS / 64)];
      const bool live = t >= 0 && c < a.s.H;
      code[u] = live ? __ldg(a.x_code + t * a.s.H + c) : 0;
      e[u] = live ? __ldg(a.x_exp + t * nbx + c / BLK) : 0;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      tile[f][r1 + u * (THREADS / 64)] = from_f32<T>((float)code[u] * value_factor(e[u]));
  }
  __syncthreads();
  for (int v = threadIdx.x; v < XG_ROWS * 64; v += THREADS) {
    const int fo = v / XG_ROWS, r = v % XG_ROWS;
    if (h0 + fo < a.s.H) x_perm[(h0 + fo) * a.R_cap + r0 + r] = tile[fo][r];
  }
}

// The blocks of one launch: gather tiles (GATHER), then rows of h and wa, then x.
struct RestoreGrid {
  int64_t gather_rows, gather, row_segs, rows, x;
};

template <typename T, bool GATHER>
__global__ void __launch_bounds__(THREADS, 4)
    act8_restore_kernel(const __grid_constant__ CUtensorMap tm, const Act8Args a,
                        const RestoreGrid g, T* x_out, T* h, T* wa) {
  extern __shared__ uint8_t raw[];
  int64_t b = blockIdx.x;
  if constexpr (GATHER) {
    if (b < g.gather) {
      uint8_t* tile = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                                 ~uintptr_t(1023));
      const int fb = (int)(b / g.gather_rows);
      gather_bf16(tm, a, (int)(b - fb * g.gather_rows), fb * G_STEPS, tile);
      return;
    }
    b -= g.gather;
  }
  if (b < g.rows) {
    const int64_t fb = b / g.row_segs;
    restore_rows<T>(a, (b - fb * g.row_segs) * 32 * Vec<T>::N, fb * ROW_FEATURES, h, wa);
    return;
  }
  restore_x<T>(a, b - g.rows, x_out);
}

template <typename T>
usaf_status restore(const Act8Args& a, void* x_out, void* x_perm, void* h, void* wa,
                    cudaStream_t st) {
  CUtensorMap tm{};
  RestoreGrid g{};
  // (the tiles' vectors of codes are indexed in 32 bits)
  const bool tiles = sizeof(T) == 2 && a.s.H % G_FEATURES == 0 && a.s.T * a.s.H < (int64_t(1) << 34);
  if (tiles) {
    if (!tcx::map_bf16_2d(&tm, x_perm, a.R_cap, a.s.H, 64, 64)) return USAF_ERR_CUDA;
    g.gather_rows = a.R_cap / G_ROWS;
    g.gather = g.gather_rows * ceil_div(a.s.H / G_FEATURES, G_STEPS);
  }
  g.row_segs = ceil_div(a.R_cap, 32 * Vec<T>::N);
  g.rows = g.row_segs * ceil_div(a.s.I, ROW_FEATURES);
  g.x = x_out ? ceil_div(a.s.T * a.s.H, X_VECTORS * Vec<T>::N) : 0;
  const int64_t blocks = g.gather + g.rows + g.x;
  if (blocks >= (int64_t(1) << 31)) return USAF_ERR_UNSUPPORTED;
  {
    USAF_TRACE("act8_restore", st);
    T *xo = static_cast<T*>(x_out), *ho = static_cast<T*>(h), *wo = static_cast<T*>(wa);
    if constexpr (sizeof(T) == 2) {
      if (tiles) {
        // four blocks' tiles per SM; the rest of the shared memory stays L1
        static OncePerDevice once;
        if (!once([] {
              return cudaFuncSetAttribute(act8_restore_kernel<T, true>,
                                          cudaFuncAttributePreferredSharedMemoryCarveout,
                                          66) == cudaSuccess;
            }))
          return USAF_ERR_CUDA;
        act8_restore_kernel<T, true><<<(unsigned)blocks, THREADS, G_SMEM, st>>>(tm, a, g, xo, ho,
                                                                                wo);
      } else {
        act8_restore_kernel<T, false><<<(unsigned)blocks, THREADS, 0, st>>>(tm, a, g, xo, ho, wo);
      }
    } else {
      act8_restore_kernel<T, false><<<(unsigned)blocks, THREADS, 0, st>>>(tm, a, g, xo, ho, wo);
    }
    USAF_CHECK_LAUNCH();
  }
  if (tiles) return USAF_OK;
  USAF_TRACE("act8_gather", st);
  const int64_t wide = ceil_div(a.s.H, 64), most = 32768;
  const dim3 grid((unsigned)(a.R_cap / XG_ROWS), (unsigned)(wide < most ? wide : most),
                  (unsigned)ceil_div(wide, most));
  act8_gather_kernel<T><<<grid, THREADS, 0, st>>>(a, static_cast<T*>(x_perm));
  USAF_CHECK_LAUNCH();
  return USAF_OK;
}

}  // namespace

usaf_status act8_save_launch(const Act8Args& a, const void* x, const void* h, uint32_t* status,
                             cudaStream_t st) {
  USAF_TRACE("act8_save", st);
  const int64_t vw = a.dt == USAF_BF16 ? 8 : 4;
  const int64_t runs = 2 * a.s.I * ceil_div(a.R_cap / vw, 32 * SAVE_U) + ceil_div(a.s.T * a.s.H, 32 * SAVE_U * vw);
  const int64_t most = 8 * 152;  // eight blocks of 256 threads fill an SM
  const int64_t want = ceil_div(runs, THREADS / 32);
  const unsigned grid = (unsigned)(want < most ? want : most);
  if (a.dt == USAF_BF16)
    act8_save_kernel<__nv_bfloat16><<<grid, THREADS, 0, st>>>(
        a, static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(h), status);
  else
    act8_save_kernel<float><<<grid, THREADS, 0, st>>>(a, static_cast<const float*>(x),
                                                      static_cast<const float*>(h), status);
  USAF_CHECK_LAUNCH();
  return USAF_OK;
}

usaf_status act8_restore_launch(const Act8Args& a, void* x_out, void* x_perm, void* h, void* wa,
                                cudaStream_t st) {
  return a.dt == USAF_BF16 ? restore<__nv_bfloat16>(a, x_out, x_perm, h, wa, st)
                           : restore<float>(a, x_out, x_perm, h, wa, st);
}

}  // namespace usaf
