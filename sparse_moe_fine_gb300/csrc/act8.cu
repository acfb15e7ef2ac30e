// Activations in 8 bits between a layer's forward and its backward (usaf_act8_save / _restore):
// blocks of 16 values share a power-of-two scale, so that coding and decoding are exact up to the
// one rounding of each code, and every decoded value is a bf16 number.
#include "train.cuh"

namespace usaf {

namespace {

constexpr int BLK = USAF_ACT8_BLOCK;
constexpr int XG_ROWS = 128;  // permuted rows of a gather tile (x 64 features)

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
__device__ __forceinline__ int code_of(float v, float f) {
  if (f == 0.f) return 0;
  const int c = __float2int_rn(v * f);  // v * f is exact: f is a power of two
  return c > 127 ? 127 : (c < -127 ? -127 : c);
}

// One block of n <= 16 consecutive values per thread.
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
    if (i < n) code[i] = (int8_t)code_of(v[i], f);
  *ex = (uint8_t)b;
  return b == 255;
}

template <typename T>
__global__ void __launch_bounds__(256)
    act8_save_kernel(const Act8Args a, const T* __restrict__ x, const T* __restrict__ h,
                     uint32_t* status) {
  const int64_t stride = (int64_t)gridDim.x * 256, i0 = (int64_t)blockIdx.x * 256 + threadIdx.x;
  bool bad = false;
  const int64_t nbx = (a.s.H + BLK - 1) / BLK;
  for (int64_t i = i0; i < a.s.T * nbx; i += stride) {
    const int64_t t = i / nbx, b = i - t * nbx;
    const int64_t o = t * a.s.H + b * BLK;
    bad |= encode_block(x + o, (int)min((int64_t)BLK, a.s.H - b * BLK), a.x_code + o, a.x_exp + i);
  }
  const int64_t nb = a.rt.expert_offset[a.s.E] / BLK, pitch = a.R_cap / BLK;
  for (int64_t i = i0; i < 2 * a.s.I * nb; i += stride) {
    const int64_t j = i / nb, b = i - j * nb;
    const int64_t o = j * a.R_cap + b * BLK;
    bad |= encode_block(h + o, BLK, a.h_code + o, a.h_exp + j * pitch + b);
  }
  flag_status_warp(status, bad, USAF_DEV_NONFINITE);
}

// silu by exp(-|g|), which does not overflow: far negative gates keep their tiny values
__device__ __forceinline__ float silu_tail(float g) {
  const float e = expf(-fabsf(g));
  return g * (g >= 0.f ? 1.f : e) / (1.f + e);
}

template <typename T>
__global__ void __launch_bounds__(256)
    act8_restore_rows_kernel(const Act8Args a, T* __restrict__ x_out, T* __restrict__ h,
                             T* __restrict__ wa) {
  const int64_t stride = (int64_t)gridDim.x * 256, i0 = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (x_out) {
    const int64_t nbx = (a.s.H + BLK - 1) / BLK;
    for (int64_t i = i0; i < a.s.T * a.s.H; i += stride) {
      const int64_t t = i / a.s.H, c = i - t * a.s.H;
      x_out[i] = from_f32<T>((float)a.x_code[i] * value_factor(a.x_exp[t * nbx + c / BLK]));
    }
  }
  const int64_t rows = a.rt.expert_offset[a.s.E], pitch = a.R_cap / BLK;
  for (int64_t i = i0; i < a.s.I * rows; i += stride) {
    const int64_t j = i / rows, r = i - j * rows;
    const int64_t og = j * a.R_cap + r, ou = (a.s.I + j) * a.R_cap + r;
    const float g = (float)a.h_code[og] * value_factor(a.h_exp[j * pitch + r / BLK]);
    const float u = (float)a.h_code[ou] * value_factor(a.h_exp[(a.s.I + j) * pitch + r / BLK]);
    const int slot = a.rt.perm_slot[r];
    const float w = slot >= 0 ? a.rt.topk_w[slot] : 0.f;
    h[og] = from_f32<T>(g);
    h[ou] = from_f32<T>(u);
    wa[og] = from_f32<T>(w * silu_tail(g) * u);
  }
}

// x_perm[f, row] = the decoded x of the row's token, 0 in padding and tail rows
template <typename T>
__global__ void __launch_bounds__(256)
    act8_gather_kernel(const Act8Args a, T* __restrict__ x_perm) {
  __shared__ T tile[64][XG_ROWS + 1];
  const int64_t r0 = (int64_t)blockIdx.x * XG_ROWS;
  const int64_t h0 = (int64_t)blockIdx.y * 64;
  const int64_t end = a.rt.expert_offset[a.s.E], nbx = (a.s.H + BLK - 1) / BLK;
  for (int v = threadIdx.x; v < XG_ROWS * 64; v += 256) {
    const int r = v / 64, f = v % 64;
    const int64_t row = r0 + r, c = h0 + f;
    float val = 0.f;
    if (row < end && c < a.s.H && a.rt.perm_slot[row] >= 0) {
      const int64_t t = a.rt.perm_tok[row];
      val = (float)a.x_code[t * a.s.H + c] * value_factor(a.x_exp[t * nbx + c / BLK]);
    }
    tile[f][r] = from_f32<T>(val);
  }
  __syncthreads();
  for (int v = threadIdx.x; v < XG_ROWS * 64; v += 256) {
    const int f = v / XG_ROWS, r = v % XG_ROWS;
    if (h0 + f < a.s.H) x_perm[(h0 + f) * a.R_cap + r0 + r] = tile[f][r];
  }
}

template <typename T>
usaf_status restore(const Act8Args& a, void* x_out, void* x_perm, void* h, void* wa,
                    cudaStream_t st) {
  {
    USAF_TRACE("act8_restore_rows", st);
    act8_restore_rows_kernel<T><<<grid_dim_for(a.s.I * a.R_cap), 256, 0, st>>>(
        a, static_cast<T*>(x_out), static_cast<T*>(h), static_cast<T*>(wa));
    USAF_CHECK_LAUNCH();
  }
  USAF_TRACE("act8_gather", st);
  const dim3 grid((unsigned)(a.R_cap / XG_ROWS), (unsigned)ceil_div(a.s.H, 64));
  act8_gather_kernel<T><<<grid, 256, 0, st>>>(a, static_cast<T*>(x_perm));
  USAF_CHECK_LAUNCH();
  return USAF_OK;
}

}  // namespace

usaf_status act8_save_launch(const Act8Args& a, const void* x, const void* h, uint32_t* status,
                             cudaStream_t st) {
  USAF_TRACE("act8_save", st);
  const unsigned grid = grid_dim_for((2 * a.s.I * a.R_cap + a.s.T * a.s.H) / BLK);
  if (a.dt == USAF_BF16)
    act8_save_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(
        a, static_cast<const __nv_bfloat16*>(x), static_cast<const __nv_bfloat16*>(h), status);
  else
    act8_save_kernel<float><<<grid, 256, 0, st>>>(a, static_cast<const float*>(x),
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
