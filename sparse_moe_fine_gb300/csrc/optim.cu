// AdamW over a list of tensors with states in 32 or 8 bits (usaf_adamw_step) and the norm of their
// gradients (usaf_grad_norm). The list travels in the kernel's arguments: no table in device memory has
// to be kept or copied, and a captured call holds its own.
#include <cuda_fp8.h>

#include <algorithm>
#include <type_traits>

#include "gate.cuh"

namespace usaf {

namespace {

constexpr int THREADS = 256;
constexpr int BLOCK8 = USAF_ADAMW_BLOCK;
constexpr int WARPS = THREADS / 32;
// Blocks of 128 elements that a warp takes, by the elements of a list: few for short ones, which have too few
// for every SM otherwise; more for long ones, whose every block looks for its tensor first. 8-bit states need
// four to have two pairs in flight. (us by 1, 2, 4 and 8 blocks, tensors of equal sizes; in brackets with bf16
// gradients:)
//   32 bits, 16 tensors:  256 K elements 3.4, 3.9, 4.9, 6.7;  1 M 6.9, 6.7, 7.0, 9.1;  4 M 20.2, 19.5, 19.8, 21.3;
//                         8 M 36.9, 36.3, 36.7, 37.6;  128 M 544, 529, 533, 538 (521, 491, 495, 501)
//           300 tensors:  4.7 M 51, 30, 24, 21;  8.6 M 92, 54, 43, 42;  300 M 2,937, 1,692, 1,251, 1,252
//   8 bits, 16 tensors:   256 K 3.0, 3.9, 4.9, 6.5 (3.3, 4.4, 5.7, 6.9);  0.5 M 6.7, 6.0, 7.1, 7.5 (6.2, 6.7, 7.4, 7.6);
//                         1 M 9.0, 7.3, 6.0, 8.2 (7.6, 7.3, 7.3, 10.9);  4 M 28.8, 21.7, 18.5, 17.9 (22.1, 18.1,
//                         15.9, 16.7);  8 M 54.5, 39.0, 31.5, 30.4 (41.8, 32.1, 27.6, 26.8)
//           300 tensors:  1.2 M 19, 13, 10, 11;  4.7 M 57, 36, 25, 20;  8.6 M 109, 66, 50, 38
constexpr int64_t K = 1024;
int step_per(int64_t n, int bits) {
  if (n < 512 * K) return 1;
  if (bits == 32) return n < 8 * K * K ? 2 : 4;
  return n < 4 * K * K ? 4 : 8;
}
// Groups of four that a thread of the norm takes (us by 4, 8, 16 and 32; in brackets of bf16 gradients):
//    16 tensors:  1 M 5.6, 5.3, 6.4, 8.7 (5.3, 4.7, 5.1, 6.5);  2 M 6.0, 6.1, 6.7, 8.9 (6.2, 6.0, 5.8, 6.6);
//                 8 M 9.8, 9.3, 9.4, 10.3 (8.9, 7.4, 8.5, 8.7);  128 M 80.3, 78.4, 77.5, 77.7 (69.1, 46.9, 44.3, 43.0)
//   300 tensors:  1.2 M 9.1, 9.5, 9.7, 9.5;  4.7 M 18.4, 14.0, 9.6, 11.7;  8.6 M 29.8, 19.9, 16.8, 15.6
int norm_per(int64_t n) { return n < 4 * K * K ? 4 : 16; }

struct Desc {
  const void* g;
  float* p;
  void *w, *m, *v;
  float *ms, *vs;
  int64_t n;
  uint64_t first;
  float step, decay;  // a / (1 - beta1^t), 1 - a * weight_decay
  int32_t vec;        // every array is aligned for four elements at once
};
// Tensors of one launch: kernel arguments may take 32,764 bytes.
template <int CAP>
struct Table {
  int count, per;      // tensors; blocks of a warp, or groups of a thread
  uint32_t end[CAP];  // blocks of threads up to and with tensor i
  Desc d[CAP];
};
constexpr int CAP_SMALL = 64, CAP_LARGE = 336;

// The tensor of a block of threads: a warp looks at 32 ends at once, as a search one after the other
// would wait for the arguments to arrive each time.
template <int CAP>
__device__ __forceinline__ int tensor_of(const Table<CAP>& tab, uint32_t block) {
  int before = 0;
  for (int i = 0; i < tab.count; i += 32) {
    const int t = i + threadIdx.x % 32;
    const unsigned done = __ballot_sync(FULL, t < tab.count && tab.end[t < CAP ? t : 0] <= block);
    before += __popc(done);
    if (done != FULL) break;
  }
  return before;
}

struct Hyper {
  float b1, b2, om_b1, om_b2, inv_bc2, eps;  // inv_bc2 = 1 / sqrt(1 - beta2^t)
  const float* g_scale;
  const uint32_t* status;
  uint32_t seed_lo, seed_hi;
  int skip;
};

// 32 random bits of place q (usaf_optim.h): all steps behind the first product.
__device__ __forceinline__ uint32_t random_from(uint32_t r, const Hyper& h) {
  r = (r ^ (r >> 16)) * 0x6a09e667u;
  r = (r ^ (r >> 15)) + h.seed_hi;
  r *= 0xbb67ae85u;
  return r ^ (r >> 16);
}
constexpr uint32_t FIRST_FACTOR = 0x9e3779b9u;
__device__ __forceinline__ uint32_t random_at(uint64_t q, const Hyper& h) {
  return random_from(((uint32_t)q ^ (uint32_t)(q >> 32) * 0x6a09e667u) * FIRST_FACTOR + h.seed_lo, h);
}

// x * inv as an e4m3 code, up or down at random. Codes are the bits of a float with three mantissa
// bits; times 2^-120 their smallest normal value is fp32's, and what is below it is evenly spaced in both:
// the code is what the lowest 20 bits of the fp32 number leave, after the random number was added to them.
// (x * inv may be a rounding above 448, which these 20 bits hold too.)
__device__ __forceinline__ uint32_t ladder(float x, float inv, uint32_t rnd20) {
  return __float_as_uint(__fmul_rn(__fmul_rn(x, inv), 0x1p-120f)) + rnd20;
}
// ...for any x; a positive r has a code of one at least
__device__ __forceinline__ uint32_t encode(float x, float inv, uint32_t rnd20) {
  const uint32_t w = ladder(x, inv, rnd20);
  return finite_f(x) ? (w >> 20 & 0x7f) | (w >> 24 & ~0x7fu) : 0x7fu;
}
__device__ __forceinline__ uint32_t encode_root(float r, float inv, uint32_t rnd20) {
  const uint32_t c = encode(r, inv, rnd20);
  return c == 0 && r > 0.f && inv > 0.f ? 1u : c;
}
__device__ __forceinline__ uint32_t rnd_m(uint32_t rnd) { return (rnd & 0xffff) << 4; }
__device__ __forceinline__ uint32_t rnd_r(uint32_t rnd) { return (rnd & 0xffff0000u) >> 12; }
__device__ __forceinline__ float decode(uint8_t c) {
  __nv_fp8_e4m3 q;
  q.__x = c;
  return (float)q;
}
__device__ __forceinline__ float amax_finite(float x) { return finite_f(x) ? fabsf(x) : 0.f; }
__device__ __forceinline__ float warp_amax(float v) {
  return __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(v)));  // not negative: ordered as bits
}
constexpr float TINY = 0x1p-100f;
__device__ __forceinline__ float inverse(float top) { return top >= TINY ? 448.f * __frcp_rn(top) : 0.f; }
__device__ __forceinline__ float scale_of(float top) { return top >= TINY ? top * (1.f / 448.f) : 0.f; }

__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// One entry: the new moments, and p's step. Moments are formed without fused products, so that their 8-bit
// codes are a function of the formula alone.
__device__ __forceinline__ void adamw_one(float g, float& p, float& m, float& v, float& r,
                                          float step, float decay, const Hyper& h) {
  m = __fadd_rn(__fmul_rn(h.b1, m), __fmul_rn(h.om_b1, g));
  v = __fadd_rn(__fmul_rn(h.b2, v), __fmul_rn(__fmul_rn(h.om_b2, g), g));
  r = sqrtf(v);
  // (the divisor is at least eps, which is a normal number)
  p = p * decay - step * (m * rcp_fast(r * h.inv_bc2 + h.eps));
}

// Four elements of an array as they are in memory: neighbours by one access where VEC, else 32 apart.
template <class T, bool VEC>
struct Raw4;
template <bool VEC>
struct Raw4<float, VEC> {
  float4 q;
  __device__ __forceinline__ void load(const float* p) {
    q = VEC ? __ldcs(reinterpret_cast<const float4*>(p)) : make_float4(p[0], p[32], p[64], p[96]);
  }
  __device__ __forceinline__ void get(float (&v)[4]) const {
    v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
  }
};
template <bool VEC>
struct Raw4<__nv_bfloat16, VEC> {
  uint2 q;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    if (VEC) {
      q = __ldcs(reinterpret_cast<const uint2*>(p));
    } else {
      const uint16_t* u = reinterpret_cast<const uint16_t*>(p);
      q = make_uint2(u[0] | (uint32_t)u[32] << 16, u[64] | (uint32_t)u[96] << 16);
    }
  }
  __device__ __forceinline__ void get(float (&v)[4]) const {
    v[0] = __uint_as_float(q.x << 16), v[1] = __uint_as_float(q.x & 0xffff0000u);
    v[2] = __uint_as_float(q.y << 16), v[3] = __uint_as_float(q.y & 0xffff0000u);
  }
};
template <bool VEC>
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  if (VEC) {
    __stcs(reinterpret_cast<float4*>(p), make_float4(v[0], v[1], v[2], v[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[32 * i] = v[i];
  }
}
template <bool VEC>
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
  if (VEC) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    __stcs(reinterpret_cast<uint2*>(p), make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                                   *reinterpret_cast<const uint32_t*>(&b)));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[32 * i] = from_f32<__nv_bfloat16>(v[i]);
  }
}

// A lane's elements of a block of 128: VEC four neighbours, 4 * lane + j, else lane + 32 * j. Both give
// the same results; the second form needs no alignment and takes the blocks that are not whole.
template <bool VEC>
__device__ __forceinline__ uint32_t place(int lane, int j) {
  return VEC ? 4 * lane + j : lane + 32 * j;
}

// A tensor from the first element of a block of threads on: elements are addressed by 32-bit distances
// from pointers that are the same for all threads.
template <class G, class W>
struct View {
  const G* g;
  float* p;
  W* w;
  char *m, *v;
  float *ms, *vs;
  uint32_t place, upper;  // of the random numbers: lower word, upper word times its factor
  bool wraps;             // the upper word changes on the way
  float step, decay, gs;
  __device__ __forceinline__ View(const Desc& d, int64_t base, int bits, uint32_t length, float scale)
      : g(static_cast<const G*>(d.g) + base),
        p(d.p + base),
        w(d.w ? static_cast<W*>(d.w) + base : nullptr),
        m(static_cast<char*>(d.m) + base * (bits / 8)),
        v(static_cast<char*>(d.v) + base * (bits / 8)),
        ms(d.ms + base / BLOCK8),
        vs(d.vs + base / BLOCK8),
        step(d.step),
        decay(d.decay),
        gs(scale) {
    const uint64_t q = d.first + (uint64_t)base;
    place = (uint32_t)q;
    upper = (uint32_t)(q >> 32) * 0x6a09e667u;
    wraps = place > 0xffffffffu - length;
  }
};
template <class T>
__device__ __forceinline__ T* at(T* base, uint32_t i) {
  return reinterpret_cast<T*>(reinterpret_cast<char*>(const_cast<std::remove_const_t<T>*>(base)) +
                              i * (uint32_t)sizeof(T));
}

// One block of 128 elements, by a warp: loads of one, and what is done with them, apart, so that a warp
// has the loads of several blocks in flight. o: the block's place in the view.
template <class G, bool VEC, int BITS>
struct Loaded {
  Raw4<G, VEC> g;
  Raw4<float, VEC> p;
  Raw4<float, VEC> m, v;  // 32 bits
  uint32_t cm, cv;        // 8 bits: four codes each, and their scales
  float ms, vs;
  template <class W>
  __device__ __forceinline__ void load(const View<G, W>& d, uint32_t o, int lane) {
    const uint32_t i = o + place<VEC>(lane, 0);
    g.load(at(d.g, i));
    p.load(at(d.p, i));
    if constexpr (BITS == 32) {
      m.load(at(reinterpret_cast<const float*>(d.m), i));
      v.load(at(reinterpret_cast<const float*>(d.v), i));
    } else {
      const uint8_t *qm = reinterpret_cast<const uint8_t*>(d.m + i),
                    *qv = reinterpret_cast<const uint8_t*>(d.v + i);
      if (VEC) {
        cm = __ldcs(reinterpret_cast<const uint32_t*>(qm));
        cv = __ldcs(reinterpret_cast<const uint32_t*>(qv));
      } else {
        cm = cv = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          cm |= (uint32_t)qm[32 * j] << 8 * j;
          cv |= (uint32_t)qv[32 * j] << 8 * j;
        }
      }
      ms = *at(d.ms, o / BLOCK8);
      vs = *at(d.vs, o / BLOCK8);
    }
  }
};

__device__ __forceinline__ void decode4(uint32_t c, float scale, float (&v)[4]) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> 16 * q & 0xffff), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    v[2 * q] = f.x * scale;
    v[2 * q + 1] = f.y * scale;
  }
}

// p and w of a block, and its new moments.
template <bool VEC, int BITS, class G, class W>
__device__ __forceinline__ void advance(const View<G, W>& d, const Hyper& h, uint32_t o, int lane,
                                        const Loaded<G, VEC, BITS>& x, float (&m)[4], float (&v)[4],
                                        float (&r)[4]) {
  float g[4], p[4];
  x.g.get(g);
  x.p.get(p);
  if constexpr (BITS == 32) {
    x.m.get(m);
    x.v.get(v);
  } else {
    decode4(x.cm, x.ms, m);
    decode4(x.cv, x.vs, r);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = r[j] * r[j];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    adamw_one(__fmul_rn(g[j], d.gs), p[j], m[j], v[j], r[j], d.step, d.decay, h);
  const uint32_t i = o + place<VEC>(lane, 0);
  store4<VEC>(at(d.p, i), p);
  if (d.w) store4<VEC>(at(d.w, i), p);
}

template <bool VEC, class G, class W>
__device__ __forceinline__ void update32(const View<G, W>& d, const Hyper& h, uint32_t o, int lane,
                                         const Loaded<G, VEC, 32>& x) {
  float m[4], v[4], r[4];
  advance<VEC, 32>(d, h, o, lane, x, m, v, r);
  const uint32_t i = o + place<VEC>(lane, 0);
  store4<VEC>(at(reinterpret_cast<float*>(d.m), i), m);
  store4<VEC>(at(reinterpret_cast<float*>(d.v), i), v);
}

template <bool VEC, class G, class W>
__device__ __forceinline__ void store_codes(const View<G, W>& d, uint32_t o, int lane, uint32_t cm,
                                            uint32_t cv) {
  const uint32_t i = o + place<VEC>(lane, 0);
  uint8_t *qm = reinterpret_cast<uint8_t*>(d.m + i), *qv = reinterpret_cast<uint8_t*>(d.v + i);
  if (VEC) {
    __stcs(reinterpret_cast<uint32_t*>(qm), cm);
    __stcs(reinterpret_cast<uint32_t*>(qv), cv);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      qm[32 * j] = (uint8_t)(cm >> 8 * j);
      qv[32 * j] = (uint8_t)(cv >> 8 * j);
    }
  }
}

// The codes of a block with whatever values, and its scales.
template <bool VEC>
__device__ __noinline__ void encode_any(float4 m4, float4 r4, uint64_t q0, const Hyper& h, int lane,
                                        uint32_t& cm, uint32_t& cv, float& ms, float& vs) {
  const float m[4] = {m4.x, m4.y, m4.z, m4.w}, r[4] = {r4.x, r4.y, r4.z, r4.w};
  float top_m = 0.f, top_r = 0.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    top_m = fmaxf(top_m, amax_finite(m[j]));
    top_r = fmaxf(top_r, amax_finite(r[j]));
  }
  top_m = warp_amax(top_m);
  top_r = warp_amax(top_r);
  const float inv_m = inverse(top_m), inv_r = inverse(top_r);
  cm = cv = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t rnd = random_at(q0 + (uint64_t)place<VEC>(lane, j), h);
    cm |= encode(m[j], inv_m, rnd_m(rnd)) << 8 * j;
    cv |= encode_root(r[j], inv_r, rnd_r(rnd)) << 8 * j;
  }
  ms = scale_of(top_m);
  vs = scale_of(top_r);
}

// The larger magnitude; NaN if one is NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}
// The highest bytes of four words.
__device__ __forceinline__ uint32_t top_bytes(const uint32_t (&w)[4]) {
  return __byte_perm(__byte_perm(w[0], w[1], 0x0073), __byte_perm(w[2], w[3], 0x0073), 0x5410);
}

// N = 1 or 2 neighbouring blocks with 8-bit states. What bounds it is the number of instructions, some 85
// an element: codes are made so that they end in the highest byte of a word, where bytes of four elements
// are put together by three permutations.
template <bool VEC, int N, class G, class W>
__device__ __forceinline__ void update8(const View<G, W>& d, const Hyper& h, uint64_t first, uint32_t o,
                                        int lane, const Loaded<G, VEC, 8>* x) {
  float m[N][4], r[N][4];
  uint32_t bits[2 * N];  // the largest magnitudes of m and r, as bits: what is not finite is above the rest
#pragma unroll
  for (int a = 0; a < N; ++a) {
    float v[4], top_m = 0.f, top_r = 0.f;
    advance<VEC, 8>(d, h, o + a * BLOCK8, lane, x[a], m[a], v, r[a]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      top_m = max_nan(top_m, m[a][j]);
      top_r = max_nan(top_r, r[a][j]);
    }
    bits[2 * a] = __float_as_uint(top_m);
    bits[2 * a + 1] = __float_as_uint(top_r);
  }
  uint32_t least = 0xffffffffu, most = 0;
#pragma unroll
  for (int a = 0; a < 2 * N; ++a) {
    bits[a] = __reduce_max_sync(FULL, bits[a]);
    least = min(least, bits[a] - 1);  // (0, as nothing but zeros has it, is no obstacle)
    most = max(most, bits[a]);
  }
  // Values of 0, or from 2^-100 to 2^10, at the blocks' tops: factors of all of them by one division, a lane
  // each, with the ladder's 2^-120 (the one rounding of the two products may differ from two by 2^-20 of a
  // step where it falls on codes below 2^-6). A block of zeros has the factor of 2^-100, which leaves them 0.
  constexpr uint32_t LEAST = 0x0d800000u, MOST = 0x44800000u;
  if (least >= LEAST - 1 && most < MOST && !d.wraps) {
    uint32_t mine = bits[0];
#pragma unroll
    for (int a = 1; a < 2 * N; ++a) mine = lane == a ? bits[a] : mine;
    const float inv = 0x1p-120f * (448.f * __frcp_rn(__uint_as_float(max(mine, LEAST))));
#pragma unroll
    for (int a = 0; a < N; ++a) {
      const float inv_m = __shfl_sync(FULL, inv, 2 * a), inv_r = __shfl_sync(FULL, inv, 2 * a + 1);
      const uint32_t q0 = d.place + o + a * BLOCK8 + place<VEC>(lane, 0);
      uint32_t wm[4], wr[4], sign[4];
      const auto codes = [&](auto first_product) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t rnd = random_from(first_product(VEC ? j : 32 * j), h);
          // (bits + 16 random bits above the 4 lowest) times 16. (nvcc 13.0 loses the high bits of a plain
          // product that is shifted like this; not those of __fmul_rn.)
          wm[j] = __float_as_uint(__fmul_rn(fabsf(m[a][j]), inv_m)) * 16 + __byte_perm(rnd, 0, 0x4104);
          wr[j] = __float_as_uint(__fmul_rn(r[a][j], inv_r)) * 16 + __byte_perm(rnd, 0, 0x4324);
          sign[j] = __float_as_uint(m[a][j]);
        }
      };
      if (d.upper == 0) {
        const uint32_t base = q0 * FIRST_FACTOR + h.seed_lo;
        codes([&](uint32_t j) { return base + j * FIRST_FACTOR; });
      } else {
        codes([&](uint32_t j) { return ((q0 + j) ^ d.upper) * FIRST_FACTOR + h.seed_lo; });
      }
      uint32_t cv = top_bytes(wr);
      if ((cv - 0x01010101u) & ~cv & 0x80808080u) {  // a code of 0, which a positive r does not get
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (!(cv >> 8 * j & 0xff) && r[a][j] > 0.f) cv |= 1u << 8 * j;
      }
      store_codes<VEC>(d, o + a * BLOCK8, lane, top_bytes(wm) | (top_bytes(sign) & 0x80808080u), cv);
    }
    if (lane < 2 * N)
      *at(lane & 1 ? d.vs : d.ms, o / BLOCK8 + lane / 2) = scale_of(__uint_as_float(mine));
    return;
  }
#pragma unroll
  for (int a = 0; a < N; ++a) {
    uint32_t cm, cv;
    float ms, vs;
    encode_any<VEC>(make_float4(m[a][0], m[a][1], m[a][2], m[a][3]),
                    make_float4(r[a][0], r[a][1], r[a][2], r[a][3]), first + o + a * BLOCK8, h, lane, cm,
                    cv, ms, vs);
    store_codes<VEC>(d, o + a * BLOCK8, lane, cm, cv);
    if (lane == 0) {
      *at(d.ms, o / BLOCK8 + a) = ms;
      *at(d.vs, o / BLOCK8 + a) = vs;
    }
  }
}

// The last block of a tensor where it is not whole: element by element.
template <class G, class W, int BITS>
__device__ __noinline__ void update_rest(const Desc& d, const Hyper& h, float gs, int64_t b, int lane) {
  const G* g = static_cast<const G*>(d.g);
  float m[4], r[4];
  float ms = 0.f, vs = 0.f, top_m = 0.f, top_r = 0.f;
  if (BITS == 8) {
    ms = d.ms[b / BLOCK8];
    vs = d.vs[b / BLOCK8];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t i = b + 32 * j + lane;
    m[j] = r[j] = 0.f;
    if (i >= d.n) continue;
    float p = d.p[i], v;
    if (BITS == 8) {
      m[j] = decode(static_cast<uint8_t*>(d.m)[i]) * ms;
      v = decode(static_cast<uint8_t*>(d.v)[i]) * vs;
      v = v * v;
    } else {
      m[j] = static_cast<float*>(d.m)[i];
      v = static_cast<float*>(d.v)[i];
    }
    adamw_one(__fmul_rn(to_f32(g[i]), gs), p, m[j], v, r[j], d.step, d.decay, h);
    d.p[i] = p;
    if (d.w) static_cast<W*>(d.w)[i] = from_f32<W>(p);
    if (BITS == 32) {
      static_cast<float*>(d.m)[i] = m[j];
      static_cast<float*>(d.v)[i] = v;
    }
    top_m = fmaxf(top_m, amax_finite(m[j]));
    top_r = fmaxf(top_r, amax_finite(r[j]));
  }
  if (BITS == 32) return;
  top_m = warp_amax(top_m);
  top_r = warp_amax(top_r);
  const float inv_m = inverse(top_m), inv_r = inverse(top_r);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t i = b + 32 * j + lane;
    if (i >= d.n) continue;
    const uint32_t rnd = random_at(d.first + (uint64_t)i, h);
    static_cast<uint8_t*>(d.m)[i] = (uint8_t)encode(m[j], inv_m, rnd_m(rnd));
    static_cast<uint8_t*>(d.v)[i] = (uint8_t)encode_root(r[j], inv_r, rnd_r(rnd));
  }
  if (lane == 0) {
    d.ms[b / BLOCK8] = scale_of(top_m);
    d.vs[b / BLOCK8] = scale_of(top_r);
  }
}

// A warp's blocks. 32 bits: two loaded at once (64 bytes a lane: more registers buy no more bandwidth). 8
// bits: half the bytes, so the next two are loaded while two are worked on.
template <class G, class W, int BITS, bool VEC>
__device__ __forceinline__ void update_blocks(const Desc& d, const Hyper& h, float gs, int64_t base,
                                              int per, int lane, int warp) {
  using L = Loaded<G, VEC, BITS>;
  const View<G, W> view(d, base, BITS, WARPS * per * BLOCK8, gs);
  const uint64_t first = d.first + (uint64_t)base;
  const uint32_t o = warp * per * BLOCK8;
  const int64_t left = d.n - base - o;
  const int whole = left >= per * BLOCK8 ? per : left > 0 ? (int)(left / BLOCK8) : 0;
  int q = 0;
  if constexpr (BITS == 8) {
    if (whole >= 2) {
      L x[2], y[2];
      x[0].load(view, o, lane);
      x[1].load(view, o + BLOCK8, lane);
#pragma unroll 1
      while (true) {
        const bool next = q + 4 <= whole;
        if (next) {
          y[0].load(view, o + (q + 2) * BLOCK8, lane);
          y[1].load(view, o + (q + 3) * BLOCK8, lane);
        }
        update8<VEC, 2>(view, h, first, o + q * BLOCK8, lane, x);
        q += 2;
        if (!next) break;
        x[0] = y[0];
        x[1] = y[1];
      }
    }
    if (q < whole) {
      L x;
      x.load(view, o + q * BLOCK8, lane);
      update8<VEC, 1>(view, h, first, o + q * BLOCK8, lane, &x);
    }
  } else {
#pragma unroll 1
    for (; q + 2 <= whole; q += 2) {
      L x[2];
      x[0].load(view, o + q * BLOCK8, lane);
      x[1].load(view, o + (q + 1) * BLOCK8, lane);
      update32<VEC>(view, h, o + q * BLOCK8, lane, x[0]);
      update32<VEC>(view, h, o + (q + 1) * BLOCK8, lane, x[1]);
    }
    if (q < whole) {
      L x;
      x.load(view, o + q * BLOCK8, lane);
      update32<VEC>(view, h, o + q * BLOCK8, lane, x);
    }
  }
  if (whole < per && left > whole * BLOCK8)
    update_rest<G, W, BITS>(d, h, gs, base + o + whole * BLOCK8, lane);
}

template <int CAP, class G, class W, int BITS>
__global__ void __launch_bounds__(THREADS) adamw_kernel(const __grid_constant__ Table<CAP> tab,
                                                        const __grid_constant__ Hyper h) {
  dep_launch();
  dep_wait();
  if (h.skip && h.status && (*(volatile const uint32_t*)h.status & USAF_DEV_SKIP_MASK)) return;
  const int ti = tensor_of(tab, blockIdx.x);
  const Desc& d = tab.d[ti];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, per = tab.per;
  const int64_t base = (int64_t)(blockIdx.x - (ti ? tab.end[ti - 1] : 0)) * (WARPS * per * BLOCK8);
  const float gs = h.g_scale ? *h.g_scale : 1.f;
  if (d.vec)
    update_blocks<G, W, BITS, true>(d, h, gs, base, per, lane, warp);
  else
    update_blocks<G, W, BITS, false>(d, h, gs, base, per, lane, warp);
}

// ------------------------------------------------------------------------------------------------
// Norm. Squares and the sums of four neighbours' are fp32; everything above is carried in pairs of fp32
// numbers (Knuth's exact sum of two numbers and its error), because an SM adds two doubles a clock: with
// doubles the blocks' own sums took longer than the reads.
// ------------------------------------------------------------------------------------------------
struct Pair {
  float hi = 0.f, lo = 0.f;
  __device__ __forceinline__ void add(float x) {
    const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
    hi = s;
  }
  __device__ __forceinline__ void add(const Pair& o) {
    add(o.hi);
    lo = __fadd_rn(lo, o.lo);
  }
  __device__ __forceinline__ double value() const { return (double)hi + (double)lo; }
};
__device__ __forceinline__ Pair warp_sum(Pair v, int width) {
  for (int o = width / 2; o; o >>= 1) {
    Pair w;
    w.hi = __shfl_xor_sync(FULL, v.hi, o);
    w.lo = __shfl_xor_sync(FULL, v.lo, o);
    v.add(w);
  }
  return v;
}
// The sum over a block's threads, in the first warp. s: [32]
__device__ __forceinline__ Pair block_sum(Pair v, Pair* s) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, warps = blockDim.x / 32;
  v = warp_sum(v, 32);
  if (lane == 0) s[warp] = v;
  __syncthreads();
  if (warp == 0) v = warp_sum(lane < warps ? s[lane] : Pair(), 32);
  return v;
}
__device__ __forceinline__ float square4(const float (&v)[4]) {
  return (v[0] * v[0] + v[1] * v[1]) + (v[2] * v[2] + v[3] * v[3]);
}
// The squares' sum of the elements [4 q, 4 q + 4) below n: whole ones by one load where `vec`.
template <class G>
__device__ __forceinline__ float square_group(const G* g, int64_t q, int64_t n, bool vec) {
  float v[4];
  if (vec && 4 * q + 4 <= n) {
    Raw4<G, true> x;
    x.load(g + 4 * q);
    x.get(v);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = 4 * q + j < n ? to_f32(g[4 * q + j]) : 0.f;
  }
  return square4(v);
}
__device__ __forceinline__ void finish_norm(const Pair& sum, double max_norm, float* out,
                                            uint32_t* status) {
  const double s = sum.value(), norm = sqrt(s);
  out[0] = (float)norm;
  out[1] = norm > max_norm ? (float)(max_norm / norm) : 1.f;
  if (!isfinite(s)) flag_status(status, USAF_DEV_NONFINITE);
}

template <int CAP, class G>
__global__ void __launch_bounds__(THREADS) norm_part_kernel(const __grid_constant__ Table<CAP> tab,
                                                            float2* __restrict__ part) {
  __shared__ Pair s[32];
  dep_launch();
  dep_wait();
  const int ti = tensor_of(tab, blockIdx.x);
  const Desc& d = tab.d[ti];
  const int64_t chunk = (int64_t)tab.per * 4 * THREADS;
  const int64_t base = (int64_t)(blockIdx.x - (ti ? tab.end[ti - 1] : 0)) * chunk;
  const G* g = static_cast<const G*>(d.g) + base;
  const int64_t n = min(d.n - base, chunk);
  const bool vec = d.vec;
  Pair sum;
  if (n == chunk && vec) {
    constexpr int AHEAD = 4;  // per is a multiple of it
#pragma unroll 2
    for (int i = 0; i < tab.per; i += AHEAD) {
      Raw4<G, true> x[AHEAD];
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) x[a].load(g + 4 * (threadIdx.x + THREADS * (i + a)));
#pragma unroll
      for (int a = 0; a < AHEAD; ++a) {
        float v[4];
        x[a].get(v);
        sum.add(square4(v));
      }
    }
  } else {
    for (int64_t q = threadIdx.x; 4 * q < n; q += THREADS) sum.add(square_group(g, q, n, vec));
  }
  sum = block_sum(sum, s);
  if (threadIdx.x == 0) part[blockIdx.x] = make_float2(sum.hi, sum.lo);
}

__global__ void __launch_bounds__(1024) norm_final_kernel(const float2* __restrict__ part,
                                                          int64_t blocks, double max_norm,
                                                          float* __restrict__ out,
                                                          uint32_t* status) {
  __shared__ Pair s[32];
  dep_launch();
  dep_wait();
  Pair sum;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < blocks; i += blockDim.x) {
    const float2 q = part[i];
    Pair x;
    x.hi = q.x;
    x.lo = q.y;
    sum.add(x);
  }
  sum = block_sum(sum, s);
  if (threadIdx.x == 0) finish_norm(sum, max_norm, out, status);
}

// A few small tensors: all by one block, in one launch, its warps taking 512 elements at a time. (us by one
// block and by two launches, of which the second costs the host some 2 us besides:  8 K elements 3.1, 3.9;
// 16 K in 8 tensors 3.5, 3.9;  in 16 3.9, 3.9;  32 K in 8 4.4, 3.8;  in 32 5.9, 4.1;  64 K in 8 6.3, 3.8)
constexpr int64_t NORM_SMALL = 16384;
constexpr int NORM_SLICE = 512;
template <class G>
__global__ void __launch_bounds__(1024) norm_small_kernel(const __grid_constant__ Table<CAP_SMALL> tab,
                                                          double max_norm, float* __restrict__ out,
                                                          uint32_t* status) {
  __shared__ Pair s[32];
  dep_launch();
  dep_wait();
  const int lane = threadIdx.x % 32;
  const uint32_t slices = tab.count ? tab.end[tab.count - 1] : 0;
  Pair sum;
  for (uint32_t i = threadIdx.x / 32; i < slices; i += 32) {
    const int t = tensor_of(tab, i);
    const Desc& d = tab.d[t];
    const int64_t base = (int64_t)(i - (t ? tab.end[t - 1] : 0)) * NORM_SLICE;
    const G* g = static_cast<const G*>(d.g) + base;
    const int64_t n = min(d.n - base, (int64_t)NORM_SLICE);
    float v[NORM_SLICE / 128];
#pragma unroll
    for (int j = 0; j < NORM_SLICE / 128; ++j) v[j] = square_group(g, lane + 32 * j, n, d.vec);
#pragma unroll
    for (int j = 0; j < NORM_SLICE / 128; ++j) sum.add(v[j]);
  }
  sum = block_sum(sum, s);
  if (threadIdx.x == 0) finish_norm(sum, max_norm, out, status);
}

// launch_dep for a kernel whose first argument is a table: it is not copied on the way.
template <int CAP, class... P, class... A>
usaf_status launch_table(void (*kernel)(Table<CAP>, P...), unsigned blocks, unsigned threads,
                         cudaStream_t st, const Table<CAP>& tab, A... args) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  static_assert(sizeof...(P) == sizeof...(A), "arguments");
  void* ptrs[] = {const_cast<Table<CAP>*>(&tab), (void*)&args...};
  if (cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kernel), ptrs) != cudaSuccess) {
    cudaGetLastError();
    return USAF_ERR_CUDA;
  }
  count_launch();
  return USAF_OK;
}

// Calls f(table, blocks) for tables that together hold every tensor with elements, in order.
template <int CAP, class F, class Fill>
usaf_status in_tables(const usaf_adamw_tensor* t, int64_t count, int per, int64_t chunk, Fill fill,
                      F f) {
  static_assert(sizeof(Table<CAP>) + sizeof(Hyper) + 64 <= 32764, "kernel arguments");
  Table<CAP> tab;
  tab.count = 0;
  tab.per = per;
  int64_t blocks = 0;
  for (int64_t i = 0; i <= count; ++i) {
    // (a single tensor has fewer than 2^42 / 4096 blocks: its list is not short)
    const int64_t need = i < count ? ceil_div(t[i].n, chunk) : 0;
    if (tab.count && (i == count || tab.count == CAP || blocks + need >= (int64_t(1) << 31))) {
      USAF_TRY(f(tab, (unsigned)blocks));
      tab.count = 0;
      blocks = 0;
    }
    if (need == 0) continue;
    blocks += need;
    fill(tab.d[tab.count], t[i]);
    tab.end[tab.count++] = (uint32_t)blocks;
  }
  return USAF_OK;
}

}  // namespace

namespace {
int64_t elements(const usaf_adamw_tensor* t, int64_t count) {
  int64_t n = 0;
  for (int64_t i = 0; i < count; ++i) n += t[i].n;
  return n;
}
}  // namespace

int64_t grad_norm_blocks(const usaf_adamw_tensor* t, int64_t count) {
  const int64_t chunk = (int64_t)norm_per(elements(t, count)) * 4 * THREADS;
  int64_t b = 0;
  for (int64_t i = 0; i < count; ++i) b += ceil_div(t[i].n, chunk);
  return b;
}

void grad_norm_ws_layout(int64_t blocks, Carver& c, NormWs& w) {
  w.part = c.take<float2>(std::max<int64_t>(blocks, 1));
}

usaf_status grad_norm_launch(const usaf_adamw_tensor* t, int64_t count, usaf_dtype gdt,
                             double max_norm, float* out, uint32_t* status, const NormWs& w,
                             int64_t blocks, cudaStream_t st) {
  USAF_TRACE("grad_norm", st);
  const uintptr_t align = gdt == USAF_BF16 ? 7 : 15;
  const int64_t total = elements(t, count);
  const int per = norm_per(total);
  const int64_t chunk = (int64_t)per * 4 * THREADS;
  const auto fill = [&](Desc& d, const usaf_adamw_tensor& q) {
    d.g = q.g;
    d.n = q.n;
    d.vec = !(reinterpret_cast<uintptr_t>(q.g) & align);
  };
  if (count <= CAP_SMALL && total <= NORM_SMALL) {
    Table<CAP_SMALL> tab;
    tab.count = 0;
    uint32_t slices = 0;
    for (int64_t i = 0; i < count; ++i) {
      if (!t[i].n) continue;
      fill(tab.d[tab.count], t[i]);
      tab.end[tab.count++] = slices += (uint32_t)ceil_div(t[i].n, NORM_SLICE);
    }
    return gdt == USAF_BF16 ? launch_table(norm_small_kernel<__nv_bfloat16>, 1, 1024, st, tab, max_norm,
                                           out, status)
                            : launch_table(norm_small_kernel<float>, 1, 1024, st, tab, max_norm, out,
                                           status);
  }
  float2* part = w.part;
  const auto launch = [&](auto& tab, unsigned n) {
    constexpr int CAP = sizeof(tab.end) / sizeof(uint32_t);
    float2* at = part;
    part += n;
    return gdt == USAF_BF16 ? launch_table(norm_part_kernel<CAP, __nv_bfloat16>, n, THREADS, st, tab, at)
                            : launch_table(norm_part_kernel<CAP, float>, n, THREADS, st, tab, at);
  };
  if (count <= CAP_SMALL)
    USAF_TRY((in_tables<CAP_SMALL>(t, count, per, chunk, fill, launch)));
  else
    USAF_TRY((in_tables<CAP_LARGE>(t, count, per, chunk, fill, launch)));
  return launch_dep(norm_final_kernel, dim3(1), blocks > 2048 ? 1024 : 256, 0, st, w.part, blocks,
                    max_norm, out, status);
}

namespace {

template <int CAP, class G, class W>
usaf_status adamw_launch_bits(int bits, const Table<CAP>& tab, const Hyper& h, unsigned n,
                              cudaStream_t st) {
  return bits == 8 ? launch_table(adamw_kernel<CAP, G, W, 8>, n, THREADS, st, tab, h)
                   : launch_table(adamw_kernel<CAP, G, W, 32>, n, THREADS, st, tab, h);
}

}  // namespace

usaf_status adamw_launch(const usaf_adamw_tensor* t, int64_t count, const AdamWArgs& a,
                         cudaStream_t st) {
  USAF_TRACE("adamw", st);
  const double bc1 = 1.0 - std::pow(a.b1, (double)a.step);
  const double bc2 = 1.0 - std::pow(a.b2, (double)a.step);
  const Hyper h{(float)a.b1, (float)a.b2, (float)(1.0 - a.b1), (float)(1.0 - a.b2),
                (float)(1.0 / std::sqrt(bc2)), (float)a.eps, a.g_scale, a.status,
                (uint32_t)a.seed, (uint32_t)(a.seed >> 32), a.skip};
  const auto fill = [&](Desc& d, const usaf_adamw_tensor& q) {
    const double lr = a.lr * q.lr_scale;
    d = Desc{q.g, q.p, q.w, q.m, q.v, q.m_scale, q.v_scale, q.n, (uint64_t)q.first,
             (float)(lr / bc1), (float)(1.0 - lr * q.weight_decay), 0};
    const auto at = [](const void* x) { return reinterpret_cast<uintptr_t>(x); };
    const uintptr_t g16 = a.gdt == USAF_BF16 ? 8 : 16, w16 = a.wdt == USAF_BF16 ? 8 : 16;
    const uintptr_t s16 = a.bits == 8 ? 4 : 16;
    d.vec = !(at(q.g) & (g16 - 1)) && !(at(q.p) & 15) && !(at(q.w) & (w16 - 1)) &&
            !(at(q.m) & (s16 - 1)) && !(at(q.v) & (s16 - 1));
  };
  const auto launch = [&](auto& tab, unsigned n) {
    constexpr int CAP = sizeof(tab.end) / sizeof(uint32_t);
    using B = __nv_bfloat16;
    if (a.gdt == USAF_BF16)
      return a.wdt == USAF_BF16 ? adamw_launch_bits<CAP, B, B>(a.bits, tab, h, n, st)
                                : adamw_launch_bits<CAP, B, float>(a.bits, tab, h, n, st);
    return a.wdt == USAF_BF16 ? adamw_launch_bits<CAP, float, B>(a.bits, tab, h, n, st)
                              : adamw_launch_bits<CAP, float, float>(a.bits, tab, h, n, st);
  };
  const int per = step_per(elements(t, count), a.bits);
  const int64_t chunk = (int64_t)per * WARPS * BLOCK8;
  if (count <= CAP_SMALL) return in_tables<CAP_SMALL>(t, count, per, chunk, fill, launch);
  return in_tables<CAP_LARGE>(t, count, per, chunk, fill, launch);
}

}  // namespace usaf
