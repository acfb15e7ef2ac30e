// The kernel of usaf_gate_topk that chooses experts. gate_sigmoid.cu and gate_softmax.cu compile it, each for
// one kind of score; gate.cu launches what follows.
#pragma once

#include <algorithm>
#include <type_traits>

#include "gate.cuh"

namespace usaf {

namespace {

// ------------------------------------------------------------------------------------------------
// Choice of experts. One warp per token; lane l holds the NL experts l * NL + i, so that a lower lane
// holds lower indices.
//
// Order by fp32 scores, then prove it. Experts are ranked by 32-bit keys: the bits of the score (of the
// logit where there is no bias: the same order), made to compare as unsigned numbers, with the lowest
// BITS replaced by the expert's place in its lane, so that a lane sorts its keys by min and max alone.
// k + 1 rounds of a warp-wide maximum take the best ones off the lanes' sorted lists. What these keys
// cannot tell apart is found afterwards: lane j scores the j-th expert again, and where it is not ahead
// of the next one by more than the keys and scores may be off (but for two taken ones that are equal in
// logit and bias), the order is settled in doubles: all experts within that margin of the last one taken
// are brought in, one per lane, scored in doubles and ranked. Groups whose scores are as near are scored
// in doubles too. With 16,383 tokens of 256 experts in 8 groups some 40 tokens need one of the two. More
// near experts than lanes go to select_exact, which does the whole token in doubles.
//
// What bounds it: instructions (646 a token of 128 experts, 910 of 256 in groups; the integer pipe half
// busy at 2.6 a clock); a row is read once. 16,383 tokens of 256 experts 21 us, 4,096 of 128 7 us.
// ------------------------------------------------------------------------------------------------

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(FULL, v, o));
  return v;
}

// A float as an unsigned number of the same order; -0 is below +0. NOTHING stands for -inf: an expert
// that the token cannot take.
__device__ __forceinline__ uint32_t ordered(float f) {
  const int32_t b = __float_as_int(f);
  return (uint32_t)(b ^ ((b >> 31) | (int32_t)0x80000000));
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}
constexpr uint32_t NOTHING = 0x007fffffu;  // ordered(-inf)

__device__ __forceinline__ void order2(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b);
  b = min(a, b);
  a = hi;
}
// Batcher's odd-even merge sort, descending, by constants alone.
template <int LO, int N, int R, int M>
__device__ __forceinline__ void merge(uint32_t (&a)[M]) {
  if constexpr (2 * R < N) {
    merge<LO, N, 2 * R>(a);
    merge<LO + R, N, 2 * R>(a);
#pragma unroll
    for (int i = LO + R; i + R < LO + N; i += 2 * R) order2(a[i], a[i + R]);
  } else {
    order2(a[LO], a[LO + R]);
  }
}
template <int LO, int N, int M>
__device__ __forceinline__ void sort(uint32_t (&a)[M]) {
  if constexpr (N > 1) {
    sort<LO, N / 2>(a);
    sort<LO + N / 2, N / 2>(a);
    merge<LO, N, 1>(a);
  }
}

constexpr int pow2_of(int n) { return n <= 1 ? 1 : 2 * pow2_of((n + 1) / 2); }
constexpr int bits_of(int n) { return n <= 1 ? 0 : 1 + bits_of((n + 1) / 2); }

// ---------------------------------------------------------------- scores
constexpr float LOG2E = 1.4426950408889634f;
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// In fp32, FAST off by less than 2^-22 (softmax: and by what inv_total is off), else by less than 2^-23.
template <bool SIG, bool FAST>
__device__ __forceinline__ float score_of(float l, float ref, float inv_total) {
  if (SIG) return FAST ? rcp_fast(1.f + exp2_fast(-LOG2E * l)) : 1.f / (1.f + expf(-l));
  return (FAST ? exp2_fast(LOG2E * (l - ref)) : expf(l - ref)) * inv_total;
}

// A double as an unsigned number of the same order, 0 for what a token cannot take.
__device__ __forceinline__ uint64_t ordered64(double d) {
  if (!(d > -INFINITY)) return 0;
  const int64_t b = __double_as_longlong(d + 0.0);
  return (uint64_t)(b ^ ((b >> 63) | (int64_t)0x8000000000000000ull));
}
__device__ __forceinline__ double unordered64(uint64_t u) {
  return __longlong_as_double((int64_t)(u >> 63 ? u ^ 0x8000000000000000ull : ~u));
}

// The token's experts by scores in doubles throughout, for what the fp32 path cannot tell apart: lane j
// gets the j-th expert and whether the token can take it. Lane l has the experts l, l + 32, ... Loops
// are kept as loops and comparisons are made on integers: few tokens come here, each on its own, so the
// time is that of fetching the code and of the few doubles an SM works on at once.
template <int NL>
__device__ __noinline__ void select_exact(const GateParams& p, const float* row, int lane, int& my_e,
                                          bool& my_ok) {
  float mx = -INFINITY;
#pragma unroll 1
  for (int e = lane; e < p.E; e += 32) {
    const float l = row[e];
    if (!isnan(l)) mx = fmaxf(mx, l);
  }
  mx = warp_max(mx);
  const double ref = mx == -INFINITY || p.sigmoid ? 0.0 : (double)mx;
  const double sign = p.sigmoid ? -1.0 : 1.0;
  double ex[NL], total = 0.0;  // exp of the logits (sigmoid: of their negatives)
#pragma unroll 1
  for (int i = 0; i < NL; ++i) {
    const int e = lane + 32 * i;
    const float l = e < p.E ? row[e] : -INFINITY;
    ex[i] = l > -INFINITY ? exp(sign * (double)l - ref) : __longlong_as_double(-1);
    if (l > -INFINITY) total += ex[i];
  }
  const double scale = p.sigmoid ? 1.0 : 1.0 / warp_sum(total);
  uint64_t c[NL];  // choice scores
#pragma unroll 1
  for (int i = 0; i < NL; ++i) {
    const int e = lane + 32 * i;
    double s = p.sigmoid ? 1.0 / (1.0 + ex[i]) : ex[i] * scale;
    if (p.bias && e < p.E) s += (double)p.bias[e];
    c[i] = ordered64(s);  // (0 for NaN: logits it cannot take, NaN biases)
  }
  unsigned kept = FULL;
  if (p.G > 1) {
    double mine = -INFINITY;  // lane g: group g's score
#pragma unroll 1
    for (int g = 0; g < p.G; ++g) {
      uint64_t x = 0, y = 0;  // the two largest of the group
#pragma unroll 1
      for (int i = 0; i < NL; ++i) {
        const int e = lane + 32 * i;
        if (e < g * p.per || e >= (g + 1) * p.per) continue;
        y = max(y, min(x, c[i]));
        x = max(x, c[i]);
      }
#pragma unroll 1
      for (int o = 16; o; o >>= 1) {
        const uint64_t ox = __shfl_xor_sync(FULL, x, o), oy = __shfl_xor_sync(FULL, y, o);
        y = max(min(x, ox), max(y, oy));
        x = max(x, ox);
      }
      if (lane == g && x) mine = unordered64(x) + (p.top == 2 && y ? unordered64(y) : 0.0);
    }
    // a group is kept if fewer than `keep` are better
    int better = 0;
#pragma unroll 1
    for (int g = 0; g < p.G; ++g) {
      const double s = __shfl_sync(FULL, mine, g);
      better += s > mine || (s == mine && g < lane);
    }
    kept = __ballot_sync(FULL, lane < p.G && better < p.keep);
  }
#pragma unroll 1
  for (int i = 0; i < NL; ++i) {
    const int e = lane + 32 * i;
    if (e < p.E) {
      // without a bias the logits order the experts; 1: one that it cannot take, 0: none or taken
      if (!((kept >> (p.G > 1 ? e / p.per : 0)) & 1u) || !c[i]) c[i] = 1;
      else if (!p.bias) c[i] = ordered64((double)row[e]);
    } else {
      c[i] = 0;
    }
  }
#pragma unroll 1
  for (int j = 0; j < p.k; ++j) {
    uint64_t best = 0;
    int be = 0x7fffffff;
#pragma unroll 1
    for (int i = 0; i < NL; ++i)
      if (c[i] > best) {
        best = c[i];
        be = lane + 32 * i;
      }
#pragma unroll 1
    for (int o = 16; o; o >>= 1) {
      const uint64_t ov = __shfl_xor_sync(FULL, best, o);
      const int oe = __shfl_xor_sync(FULL, be, o);
      if (ov > best || (ov == best && oe < be)) {
        best = ov;
        be = oe;
      }
    }
    if ((be & 31) == lane) c[be >> 5] = 0;
    if (lane == j) {
      my_e = be;
      my_ok = best > 1;
    }
  }
}

// Sum over all experts of exp(l - ref), in doubles: the whole warp.
__device__ __noinline__ double total_exact(const GateParams& p, const float* row, float ref,
                                           int lane) {
  double total = 0.0;
#pragma unroll 1
  for (int e = lane; e < p.E; e += 32)
    if (row[e] > -INFINITY) total += exp((double)row[e] - (double)ref);
  return warp_sum(total);
}

// A choice score in doubles (total: total_exact for softmax).
__device__ __forceinline__ double score64(const GateParams& p, float l, float b, float ref,
                                          double total) {
  const double ex = exp(p.sigmoid ? -(double)l : (double)l - (double)ref);
  return (p.sigmoid ? 1.0 / (1.0 + ex) : ex / total) + (double)b;
}

// The groups to keep: those of `sure`, and the best of `open` by scores in doubles.
__device__ __noinline__ unsigned groups_exact(const GateParams& p, const float* row, float ref,
                                              int lane, unsigned sure, unsigned open) {
  const double total = p.sigmoid ? 1.0 : total_exact(p, row, ref, lane);
  double mine = -INFINITY;  // lane g: group g's score
#pragma unroll 1
  for (unsigned left = open; left; left &= left - 1) {
    const int g = __ffs(left) - 1;
    uint64_t x = 0, y = 0;
#pragma unroll 1
    for (int i = lane; i < p.per; i += 32) {
      const int e = g * p.per + i;
      const float l = row[e];
      if (!(l > -INFINITY)) continue;
      const uint64_t c = ordered64(score64(p, l, p.bias ? p.bias[e] : 0.f, ref, total));
      y = max(y, min(x, c));
      x = max(x, c);
    }
#pragma unroll 1
    for (int o = 16; o; o >>= 1) {
      const uint64_t ox = __shfl_xor_sync(FULL, x, o), oy = __shfl_xor_sync(FULL, y, o);
      y = max(min(x, ox), max(y, oy));
      x = max(x, ox);
    }
    if (lane == g && x) mine = unordered64(x) + (p.top == 2 && y ? unordered64(y) : 0.0);
  }
  int better = __popc(sure);
#pragma unroll 1
  for (unsigned left = open; left; left &= left - 1) {
    const int g = __ffs(left) - 1;
    const double s = __shfl_sync(FULL, mine, g);
    better += s > mine || (s == mine && g < lane);
  }
  return sure | __ballot_sync(FULL, ((open >> lane) & 1u) && better < p.keep);
}

// Whether all logits of a row, and all biases, are the same.
__device__ __noinline__ bool uniform_row(const GateParams& p, const float* row, int lane) {
  const float l0 = row[0], b0 = p.bias ? p.bias[0] : 0.f;
  bool other = false;
#pragma unroll 1
  for (int e = lane; e < p.E; e += 32) other |= !(row[e] == l0 && (p.bias ? p.bias[e] : 0.f) == b0);
  return !__any_sync(FULL, other);
}

template <int NL>
struct Lists {
  static constexpr int NP = pow2_of(NL), BITS = bits_of(NL);
  uint32_t a[NP];  // a lane's keys, best first; 0: none left
  // takes the best key of the warp, of equal ones (but for the place) the lowest lane's: key and lane go
  // to *to
  __device__ __forceinline__ void take(unsigned below, int lane, uint2* to) {
    const uint32_t head = a[0] >> BITS;
    const unsigned who = __ballot_sync(FULL, head == __reduce_max_sync(FULL, head));
    const bool win = (who & (below + below + 1)) == below + 1;  // this lane, and none below it
    if (win) *to = make_uint2(a[0], (uint32_t)lane);
#pragma unroll
    for (int i = 0; i < NP; ++i) a[i] = win ? (i + 1 < NP ? a[i + 1 < NP ? i + 1 : 0] : 0u) : a[i];
  }
};

// How groups lie on the lanes.
struct Groups {
  bool whole;  // a group is a power of two of whole lanes
  int lanes;   // then: of a group
  int mine;    // then: this lane's group, else: `lane`
  int first, mask;  // the first lane of the lane's group (else `lane`), and what makes it of a lane
};

// All of one token: writes its indices and weights; returns the lane's expert, which is the rank-th
// taken, or -1. v: the lane's logits, b: biases, -inf for NaN.
template <int NL, bool SIG, bool BIAS>
__device__ __forceinline__ int select_token(const GateParams& p, int64_t t, const float (&v)[NL],
                                            const float (&b)[NL], const Groups& gr, int lane,
                                            uint2* taken, int32_t* topk_idx, float* topk_w,
                                            int& rank) {
  using Ls = Lists<NL>;
  constexpr int NP = Ls::NP, BITS = Ls::BITS;
  const float* row = p.logits + t * p.ld;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < NL; ++i) bad |= isnan(v[i]);
  float ref = 0.f, inv_total = 1.f;
  bool none = false;  // softmax of a row with +inf: no weights
  if (!SIG) {
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < NL; ++i) mx = fmaxf(mx, v[i]);
    mx = unordered(__reduce_max_sync(FULL, ordered(mx)));
    none = mx == INFINITY;
    bad |= none;
    ref = mx == -INFINITY ? 0.f : mx;
    if (BIAS || p.G > 1 || !p.renorm) {
      float total = 0.f;
#pragma unroll
      for (int i = 0; i < NL; ++i) total += v[i] > -INFINITY ? expf(v[i] - ref) : 0.f;
      inv_total = 1.f / warp_sum(total);
    }
  }
  // what orders the experts, as unsigned numbers
  uint32_t f[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const float x = BIAS ? score_of<SIG, true>(v[i], ref, inv_total) + b[i] : v[i] + 0.f;
    f[i] = v[i] > -INFINITY ? ordered(none ? 0.f : x) : NOTHING;
  }
  // What two entries may be apart and be in the wrong order. Scores are off by less than 2^-22 (softmax: and
  // by NL + 8 roundings of the sum), those formed again by less than half of that; without a bias logits
  // are compared, which are exact; keys are off by their lowest bits. Experts that are all scored again
  // need not be further apart than those scores are off. (Logits below the smallest normal number are 2^-149
  // apart whatever their size, so their keys are off by a number that does not fall with them.)
  constexpr float base = !BIAS ? (1 << BITS) * 0x1p-147f : SIG ? 0x1p-20f : 0x1p-19f + (NL + 8) * 0x1p-22f;
  const auto margin = [&](float c) { return base + fabsf(c) * ((1 << BITS) * 0x1p-21f); };
  const auto again = [&](float c) { return !BIAS ? 0.f : SIG ? 0x1p-21f + fabsf(c) * 0x1p-22f : margin(c); };
  if (p.G > 1) {
    const auto value = [&](uint32_t u) {  // the score of an entry, -inf for no expert
      if (u <= NOTHING) return -INFINITY;
      return BIAS ? unordered(u) : score_of<SIG, false>(unordered(u), ref, inv_total);
    };
    const bool whole = gr.whole;
    const int lanes = gr.lanes, group = gr.mine;
    uint32_t x = 0, y = 0;  // the two best of a lane, of a group
    if (whole) {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        y = max(y, min(x, f[i]));
        x = max(x, f[i]);
      }
      for (int o = lanes >> 1; o; o >>= 1) {
        const uint32_t ox = __shfl_xor_sync(FULL, x, o), oy = __shfl_xor_sync(FULL, y, o);
        y = max(min(x, ox), max(y, oy));
        x = max(x, ox);
      }
    } else {
      for (int g = 0; g < p.G; ++g) {
        uint32_t gx = 0, gy = 0;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
          const int e = lane * NL + i;
          if (e >= g * p.per && e < (g + 1) * p.per) {
            gy = max(gy, min(gx, f[i]));
            gx = max(gx, f[i]);
          }
        }
        const uint32_t m1 = __reduce_max_sync(FULL, gx);
        const int w = __ffs(__ballot_sync(FULL, gx == m1)) - 1;
        const uint32_t m2 = __reduce_max_sync(FULL, lane == w ? gy : gx);
        if (lane == g) {
          x = m1;
          y = m2;
        }
      }
    }
    const float vx = value(x), vy = value(y);
    const float mine = p.top == 2 && vy > -INFINITY ? vx + vy : vx;  // the group's score
    // the best group left, `keep` times; equal ones: the lower first
    const bool is = group < p.G;
    const int first_lane = gr.first;
    uint32_t left = is ? ordered(mine) : 0u, last = 0;
    bool in = false;
    for (int i = 0; i < p.keep; ++i) {
      last = __reduce_max_sync(FULL, left);
      const int w = __ffs(__ballot_sync(FULL, left == last)) - 1;
      if (first_lane == (w & gr.mask)) {
        in = true;
        left = 0;
      }
    }
    if (p.keep < p.G) {
      // the last group kept and the first that is not: two sums of two scores. (Without a bias scores are off
      // in proportion, by less than 2^-21 of the largest, and what softmax's sum is off moves all alike. Only
      // below 2^-128, where exp(-l) passes fp32, a sigmoid is 0 instead: four are off by less than 2^-125.)
      const float lo = unordered(last), hi = unordered(max(__reduce_max_sync(FULL, left), NOTHING));
      const float size = vx > -INFINITY ? fabsf(vx) + (vy > -INFINITY ? fabsf(vy) : 0.f) : 0.f;
      const float reach =
          (BIAS ? 2.f * base : 0x1p-125f) +
          __uint_as_float(__reduce_max_sync(FULL, __float_as_uint(size))) * (BIAS ? 0x1p-21f : 0x1p-19f);
      bool unsure = hi > -INFINITY && !none && !(lo - hi > reach);  // the same for all lanes
      // in a row of one logit and one bias throughout all groups are equal, as they are in fp32
      if (unsure) unsure = !uniform_row(p, row, lane);
      if (unsure) {
        // a group so far ahead of the first one out stays in, one so far behind the last one in stays out
        const bool open = is && !(in ? mine - hi > reach : lo - mine > reach);
        unsigned sure = 0, near = 0;
        for (int g = 0; g < p.G; ++g) {
          const int from = whole ? g * lanes : g;
          near |= (unsigned)__shfl_sync(FULL, (int)open, from) << g;
          sure |= (unsigned)__shfl_sync(FULL, (int)(in && !open), from) << g;
        }
        const unsigned now = groups_exact(p, row, ref, lane, sure, near);  // every lane calls it
        in = is && (now >> (group & 31) & 1u);
      }
    }
    if (whole) {
#pragma unroll
      for (int i = 0; i < NL; ++i) f[i] = in ? f[i] : NOTHING;
    } else {
      const unsigned kept = __ballot_sync(FULL, in);
#pragma unroll
      for (int i = 0; i < NL; ++i)
        if (!((kept >> ((lane * NL + i) / p.per & 31)) & 1u)) f[i] = NOTHING;
    }
  }
  // keys: the entry's place in its lane in the lowest bits. (Places behind the last expert hold NOTHING
  // too, and come after every expert.)
  Ls ls;
#pragma unroll
  for (int i = 0; i < NP; ++i)
    ls.a[i] = i < NL ? (f[i < NL ? i : 0] & ~(uint32_t)(NP - 1)) | (NP - 1 - i) : 0u;
  sort<0, NP>(ls.a);

  int my_e = 0;
  rank = lane;
  bool ok = false;
  float my_l = 0.f, my_b = 0.f, my_s = 0.f, my_c = -INFINITY;
  bool exact = p.k >= 32;  // lane k holds the first expert that is not taken
  if (!exact) {
    const int n = p.k < p.E ? p.k + 1 : p.k;
    // lanes from `lane` down to 0, but for itself
    const unsigned below = (1u << lane) - 1;
#pragma unroll 3
    for (int j = 0; j < n; ++j) ls.take(below, lane, taken + j);
    __syncwarp();
    uint2 my = lane < n ? taken[lane] : make_uint2(0u, 0u);  // key, lane
    const auto look = [&](bool on) {  // the expert, its own logit and bias, scored again
      my_e = (int)my.y * NL + (NP - 1 - (int)(my.x & (NP - 1)));
      ok = on && my.x >> BITS > NOTHING >> BITS;
      if (ok) {
        my_l = row[my_e];
        my_b = BIAS ? p.bias[my_e] : 0.f;
        my_s = score_of<SIG, false>(my_l, ref, inv_total);
        my_c = BIAS ? my_s + my_b : my_l;
      }
    };
    look(lane < n);
    const float nc = __shfl_down_sync(FULL, my_c, 1), nl = __shfl_down_sync(FULL, my_l, 1),
                nb = __shfl_down_sync(FULL, my_b, 1);
    const bool inner = lane + 1 < p.k;  // both are taken
    const bool near = lane + 1 < n && ok && nc > -INFINITY && !none &&
                      !(my_c - nc > (inner ? again(my_c) : margin(my_c))) &&
                      !(inner && my_l == nl && my_b == nb);
    if (__any_sync(FULL, near)) {
      // more experts, until one is out of the last taken one's reach, unless all within it equal that one
      const float last = __shfl_sync(FULL, my_c, p.k - 1), last_l = __shfl_sync(FULL, my_l, p.k - 1),
                  last_b = __shfl_sync(FULL, my_b, p.k - 1);
      const auto within = [&](float c) { return c > -INFINITY && !(last - c > margin(last)); };
      int m = n;
      bool open = n > p.k && within(__shfl_sync(FULL, my_c, n - 1));
      if (open) {
        bool other = false;  // (experts of groups that are not kept may count too: then there is more to do)
#pragma unroll 1
        for (int e = lane; e < p.E; e += 32) {
          const float l = row[e], bias = BIAS ? p.bias[e] : 0.f;
          const float c = BIAS ? score_of<SIG, true>(l, ref, inv_total) + bias : l;
          other |= fabsf(c - last) <= 2.f * margin(last) && !(l == last_l && bias == last_b);
        }
        open = __any_sync(FULL, other) || isinf(last);
      }
      if (__any_sync(FULL, near && inner) || open) {
        while (open && m < 32 && m < p.E) {
          ls.take(below, lane, taken + m);
          __syncwarp();
          if (lane == m) my = taken[m];
          ++m;
          look(lane < m);
          open = within(__shfl_sync(FULL, my_c, m - 1));
        }
        if (open && m == 32 && m < p.E) {
          exact = true;
        } else {
          double c = -INFINITY;
          const double total = BIAS && !SIG ? total_exact(p, row, ref, lane) : 1.0;
          if (ok) c = BIAS ? score64(p, my_l, my_b, ref, total) : (double)my_l;
          rank = 0;
#pragma unroll 1
          for (int j = 0; j < m; ++j) {
            const double oc = __shfl_sync(FULL, c, j);
            const int oe = __shfl_sync(FULL, my_e, j);
            rank += oc > c || (oc == c && oe < my_e);
          }
          if (lane >= m) rank = 32;
        }
      }
    }
  }
  if (exact) {
    select_exact<NL>(p, row, lane, my_e, ok);
    rank = lane;
    if (ok) my_l = row[my_e];
    my_s = ok ? score_of<SIG, false>(my_l, ref, inv_total) : 0.f;
  }
  const bool mine = rank < p.k;
  ok = ok && mine;
  // weights
  float a = ok ? my_s : 0.f;
  if (p.renorm) {
    float sum = warp_sum(a);
    if (__any_sync(FULL, ok && !(a > 0x1p-100f))) {
      // a score that fp32 has few bits of, or none, while its ratio to the sum may be any number:
      // relative to the largest taken, with s = exp(min(l, 0)) / (1 + exp(-|l|)) or exp(l) / total
      const float pos = SIG ? fminf(my_l, 0.f) : my_l;
      const float top = warp_max(ok ? pos : -INFINITY);
      a = !ok ? 0.f : SIG ? expf(pos - top) / (1.f + expf(-fabsf(my_l))) : expf(pos - top);
      sum = warp_sum(a);
    }
    a = sum > 0.f ? a / sum : 0.f;
  }
  if (none) a = __int_as_float(0x7fffffff);
  if (mine) {
    topk_idx[t * p.k + rank] = my_e;
    topk_w[t * p.k + rank] = p.scale * a;
  }
  if (__any_sync(FULL, bad) && lane == 0) flag_status(p.status, USAF_DEV_NONFINITE);
  return mine ? my_e : -1;
}

// The NL values of a lane from a row of E: wide loads where the row allows them.
template <int NL>
__device__ __forceinline__ void load_lane(const float* row, int E, int lane, bool vec, float rest,
                                          float (&v)[NL]) {
  const int e0 = lane * NL;
  if (NL % 4 == 0 && vec && e0 + NL <= E) {
#pragma unroll
    for (int i = 0; i < NL; i += 4) {
      const float4 q = *reinterpret_cast<const float4*>(row + e0 + i);
      v[i] = q.x;
      v[i + 1] = q.y;
      v[i + 2] = q.z;
      v[i + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NL; ++i) v[i] = e0 + i < E ? row[e0 + i] : rest;
  }
}

// A block has `tokens` tokens, 8 of a chunk or all 32, its warps take them in turn; it leaves its bytes of the
// chunk's words in masks (gate.cuh), or, where the batch is one chunk, writes the tables itself.
template <int NL, bool SIG, bool BIAS>
__global__ void __launch_bounds__(32 * GATE_MAX_WARPS)
    gate_select_kernel(const GateParams p, const GateTables o, uint32_t* __restrict__ masks,
                       int tokens) {
  extern __shared__ uint2 smem[];
  uint2* taken = smem;                                                // [warps][32]
  uint32_t* mask = reinterpret_cast<uint32_t*>(smem + blockDim.x);    // [E]
  int32_t* s_off = reinterpret_cast<int32_t*>(mask + p.E);            // one chunk: [E + 1]
  int32_t* s_warp = s_off + p.E + 1;                                  // one chunk: [GATE_MAX_WARPS]
  int32_t* s_idx = s_warp + GATE_MAX_WARPS;                           // one chunk: [32 * k]
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t t0 = (int64_t)blockIdx.x * tokens;
  const bool one = gridDim.x == 1;
  const bool vec = ((reinterpret_cast<uintptr_t>(p.logits) | (uintptr_t)(p.ld * 4)) & 15) == 0;
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) mask[e] = 0;
  dep_wait();
  float b[NL];
  if (BIAS) {
    bool bad = false;
    load_lane<NL>(p.bias, p.E, lane, (reinterpret_cast<uintptr_t>(p.bias) & 15) == 0, 0.f, b);
#pragma unroll
    for (int i = 0; i < NL; ++i)
      if (isnan(b[i])) {
        bad = true;
        b[i] = -INFINITY;
      }
    if (__any_sync(FULL, bad) && threadIdx.x == 0) flag_status(p.status, USAF_DEV_NONFINITE);
  }
  Groups gr;
  gr.lanes = p.per / NL;
  gr.whole = gr.lanes * NL == p.per && (gr.lanes & (gr.lanes - 1)) == 0;
  gr.mine = gr.whole ? lane / gr.lanes : lane;
  gr.mask = gr.whole ? ~(gr.lanes - 1) : ~0;
  gr.first = lane & gr.mask;
  __syncthreads();
  for (int tok = warp; tok < tokens && t0 + tok < p.T; tok += blockDim.x / 32) {
    float l[NL];
    load_lane<NL>(p.logits + (t0 + tok) * p.ld, p.E, lane, vec, -INFINITY, l);
    int rank;
    const int e = select_token<NL, SIG, BIAS>(p, t0 + tok, l, b, gr, lane, taken + 32 * warp,
                                              o.topk_idx, o.topk_w, rank);
    __syncwarp();  // taken is read before the next token's are written
    if (e >= 0) {
      atomicOr(&mask[e], 1u << tok);
      if (one) s_idx[tok * p.k + rank] = e;
    }
  }
  // not before: the next kernel's blocks would wait in the room that this one's tokens are worked on in
  // (16,383 tokens: 33 -> 29 us in all)
  dep_launch();
  __syncthreads();
  if (!one) {
    // the block's byte of each word, whose lowest bits are the chunk's first tokens (little-endian)
    const int parts = GATE_CHUNK / tokens, part = (int)(blockIdx.x % parts);
    uint32_t* words = masks + (int64_t)(blockIdx.x / parts) * p.E;
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
      if (parts == 1) words[e] = mask[e];
      else reinterpret_cast<uint8_t*>(words + e)[part] = (uint8_t)mask[e];
    }
    return;
  }
  const auto count = [&](int e) { return __popc(mask[e]); };
  expert_offsets(p.E, count, s_off, s_warp);
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
    o.count[e] = count(e);
    o.offset[e] = s_off[e];
    fill_padding(o, s_off[e] + count(e), s_off[e + 1], 0, 1);
  }
  if (threadIdx.x == 0) o.offset[p.E] = s_off[p.E];
  for (int s = threadIdx.x; s < (int)p.T * p.k; s += blockDim.x) {
    const int e = s_idx[s], tok = s / p.k;
    const int32_t pos = s_off[e] + __popc(mask[e] & ((1u << tok) - 1));
    o.perm_tok[pos] = tok;
    o.perm_slot[pos] = s;
    o.slot_row[s] = pos;
  }
  fill_tail(o, s_off[p.E], o.cap, threadIdx.x, blockDim.x);
}

// The experts a lane holds: as few as will do of these numbers. A number between two powers of two is worth its
// code: it sorts and shifts fewer keys, and groups fall on whole lanes where they would not otherwise (16,383
// tokens, sigmoid with a bias, us; in brackets in 8 groups):
//   E   96: 3 a lane 20.3 (23.1), 4 a lane 20.8 (32.8)     E 136: 5 a lane 22.0 (35.8),  8 a lane 24.1 (42.8)
//   E  160: 5 a lane 22.0 (25.6), 8 a lane 23.9 (43.3)     E 192: 6 a lane 22.9 (27.4),  8 a lane 24.0 (43.7)
//   E  320: 12 a lane 30.5 (56.1), 16 a lane 35.0 (66.9)   E 384: 12 a lane 30.4 (34.3), 16 a lane 35.8 (67.7)
template <bool SIG, bool BIAS>
usaf_status select_width(const GateParams& p, const GateTables& o, uint32_t* masks, unsigned blocks,
                         unsigned threads, size_t smem, int tokens, cudaStream_t st) {
  const auto go = [&](auto nl) {
    return launch_dep(gate_select_kernel<decltype(nl)::value, SIG, BIAS>, dim3(blocks), threads, smem,
                      st, p, o, masks, tokens);
  };
  const int nl = (p.E + 31) / 32;
  if (nl <= 1) return go(std::integral_constant<int, 1>());
  if (nl <= 2) return go(std::integral_constant<int, 2>());
  if (nl <= 3) return go(std::integral_constant<int, 3>());
  if (nl <= 4) return go(std::integral_constant<int, 4>());
  if (nl <= 5) return go(std::integral_constant<int, 5>());
  if (nl <= 6) return go(std::integral_constant<int, 6>());
  if (nl <= 8) return go(std::integral_constant<int, 8>());
  if (nl <= 12) return go(std::integral_constant<int, 12>());
  if (nl <= 16) return go(std::integral_constant<int, 16>());
  return go(std::integral_constant<int, 32>());
}

template <bool SIG>
usaf_status select_scores(const GateParams& p, const GateTables& o, uint32_t* masks, int64_t chunks,
                          cudaStream_t st) {
  // A warp for each token, in blocks of whole chunks, while an SM has no more than 32 tokens; from there on four
  // warps share eight tokens, in blocks small enough that SMs have much the same number of tokens, and for
  // batches that fill the SMs anyway eight warps share a chunk, which clear and write fewer words. Lanes with
  // more than 8 experts are slowed by blocks of 1,024 threads at any size. (us by a warp a token, blocks of
  // eight tokens, chunks of eight warps:)
  //   E 128:  4,096 tokens 12.4, 12.4, 15.6;  4,864 (32 an SM) 12.6, 13.2, 15.7;  5,001 15.2, 13.4, 15.9;
  //           9,728 (64 an SM) 18.5, 16.1, 18.0;  16,383 28.0, 21.9, 22.0;  32,768 (216 an SM) 48.7, 37.6, 36.5
  //   E 256 in 8 groups:  4,864 16.5, 17.2, 20.4;  5,001 19.3, 17.4, 20.7;  16,383 37.0, 28.2, 29.8;
  //           32,768 64.7, 49.2, 49.7;  65,536 127, 90.4, 89.4
  //   E 512:  128 tokens 40.1, 36.4, 41.6;  3,000 22.0, 19.0, 22.6;  16,383 52.1, 34.6, 37.3;
  //           65,536 176, 112.4, 112.4          E 1,024:  4,864 43.7, 44.0, 58.3;  16,383 122, 83.3, 83.5
  // (One chunk alone has the tables to write too. Parts of a chunk without tokens are launched as
  // well: their bits are zero.)
  const int64_t per_sm = ceil_div(p.T, device_sm_count());
  const bool small = chunks > 1 && per_sm <= 128 && (per_sm > 32 || p.E > 256);
  const int tokens = small ? 8 : GATE_CHUNK;
  const unsigned warps = chunks == 1 ? (unsigned)std::max<int64_t>(8, p.T)
                         : small ? 4
                         : per_sm <= 32 ? GATE_MAX_WARPS : 8;
  const unsigned blocks = (unsigned)(chunks * (GATE_CHUNK / tokens)), threads = 32 * warps;
  const size_t smem =
      threads * sizeof(uint2) +
      (chunks > 1 ? p.E : 2 * p.E + 1 + GATE_MAX_WARPS + GATE_CHUNK * p.k) * sizeof(int32_t);
  return p.bias ? select_width<SIG, true>(p, o, masks, blocks, threads, smem, tokens, st)
                : select_width<SIG, false>(p, o, masks, blocks, threads, smem, tokens, st);
}

}  // namespace

}  // namespace usaf
