// Around routed experts: the choice of each token's experts from its router logits, and the weighted sum of
// their outputs.
#include <type_traits>

#include "attn_launch.hpp"
#include "head_common.hpp"
#include "launch.hpp"

namespace ql {
namespace {

// ---------------------------------------------------------------- the choice
//
// p = softmax or sigmoid of the logits, c = p + bias, the best groups, the k largest c: in 64 bits, because
// which expert comes first hangs on the last bits of c (two of 256 scores lie within 1e-7 of each other in
// one token of ten thousand), and the vector units run fp64 at the rate of fp32 here.
//
// One wave a token, EPL neighbouring experts a lane, so that the lowest lane with the largest c holds the
// lowest index: a round takes the lane's largest, the wave's by DPP, and a ballot.  Rounds compare fp32 keys and
// look at 64 bits only where more than one lane has the largest.
//
// Measured: one token of 128 experts 4.2 us; 8192 tokens of 256 experts, sigmoid, 4 of 8 groups, 8 chosen, 17 to 18 us
// against 2 of memory: bound by the vector units, 950 instructions a token, issue 82 % busy (the coefficients of
// the exponential as scalar operands, a sixth fewer instructions: 17.9 against 17.9; each lane's experts in
// order before the rounds, which then only shift them: 18.9).

constexpr double kLowest = -1.7976931348623157e308;  // c of -infinity or NaN
constexpr double kOut = -__builtin_inf();            // not to be chosen (again)

template <int CTRL> __device__ __forceinline__ double dpp64(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp((int)(uint32_t)u, (int)(uint32_t)u, CTRL, 0xf, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp((int)(uint32_t)(u >> 32), (int)(uint32_t)(u >> 32), CTRL, 0xf, 0xf, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lane64(double x, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane), hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// f over the wave, in every lane.
template <typename F> __device__ __forceinline__ double wave64(double x, F f) {
  x = f(x, dpp64<0xB1>(x));
  x = f(x, dpp64<0x4E>(x));
  x = f(x, dpp64<0x141>(x));
  x = f(x, dpp64<0x140>(x));
  // rows of 16 lanes hold their value in every lane
  return f(f(lane64(x, 0), lane64(x, 16)), f(lane64(x, 32), lane64(x, 48)));
}
// The largest over the wave, uniform.
__device__ __forceinline__ int wave_max(int x) {
  auto step = [&](auto ctrl) { x = max(x, __builtin_amdgcn_update_dpp(x, x, decltype(ctrl)::value, 0xf, 0xf, false)); };
  step(std::integral_constant<int, 0xB1>{});
  step(std::integral_constant<int, 0x4E>{});
  step(std::integral_constant<int, 0x141>{});
  step(std::integral_constant<int, 0x140>{});
  return max(max(__builtin_amdgcn_readlane(x, 0), __builtin_amdgcn_readlane(x, 16)),
             max(__builtin_amdgcn_readlane(x, 32), __builtin_amdgcn_readlane(x, 48)));
}
struct Max64 {
  __device__ __forceinline__ double operator()(double a, double b) const { return fmax(a, b); }
};
struct Add64 {
  __device__ __forceinline__ double operator()(double a, double b) const { return a + b; }
};

// e^x for x <= 709.7, within some 2^-52 of its value: 2^k e^r with |r| <= ln 2 / 2, e^r by its series (the
// first term left out is below 2^-57).
__device__ __forceinline__ double exp64(double x) {
  const double k = __builtin_rint(x * 1.4426950408889634074);
  // ln 2 in two parts, the first with 32 bits, so that k times it is exact
  const double r = __builtin_fma(-k, 0x1.473de6af278edp-34, __builtin_fma(-k, 0x1.62e42fefp-1, x));
  double p = 1. / 6227020800.;
  p = __builtin_fma(p, r, 1. / 479001600.);
  p = __builtin_fma(p, r, 1. / 39916800.);
  p = __builtin_fma(p, r, 1. / 3628800.);
  p = __builtin_fma(p, r, 1. / 362880.);
  p = __builtin_fma(p, r, 1. / 40320.);
  p = __builtin_fma(p, r, 1. / 5040.);
  p = __builtin_fma(p, r, 1. / 720.);
  p = __builtin_fma(p, r, 1. / 120.);
  p = __builtin_fma(p, r, 1. / 24.);
  p = __builtin_fma(p, r, 1. / 6.);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.);
  p = __builtin_fma(p, r, 1.);
  return __builtin_ldexp(p, (int)fmax(k, -1100.));
}
// 1 / x for 1 <= x < 2^1020, by Newton's steps.
__device__ __forceinline__ double inverse64(double x) {
  double r = __builtin_amdgcn_rcp(x);
  r = __builtin_fma(__builtin_fma(-x, r, 1.), r, r);
  return __builtin_fma(__builtin_fma(-x, r, 1.), r, r);
}

__device__ __forceinline__ float logit_at(const void* row, int dt, int64_t i) {
  if (dt == DT_F32) return ((const float*)row)[i];
  const uint32_t b = ((const uint16_t*)row)[i];
  return dt == DT_BF16 ? bf16_bits_to_f32(b) : f16_bits_to_f32(b);
}

template <int EPL> __global__ __launch_bounds__(256) void select_kernel(const SelectArgs a, FastDiv group_div, int lpg) {
  __shared__ double sc[4][64 * EPL];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * 4 + wave;
  if (t >= a.t) return;
  int64_t* ids = a.ids + t * a.k;
  float* weights = a.weights + t * a.k;
  if (a.n_rows && t >= a.n_rows[0]) {
    if (lane < a.k) ids[lane] = -1, weights[lane] = 0.f;
    return;
  }
  const uint8_t* row = (const uint8_t*)a.logits + t * a.row_stride * (a.dt == DT_F32 ? 4 : 2);
  float x[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int i = lane * EPL + j;
    x[j] = -__builtin_inff();
    if (i < a.e) {
      const float v = logit_at(row, a.dt, i);
      x[j] = v == v ? v : x[j];
    }
  }
  double p[EPL], c[EPL];
  if (a.sigmoid) {
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      // far below 0 it is e^x itself (next to it, 1 + e^-x and its inverse leave the normal numbers)
      const bool far = x[j] < -700.f;
      const double e = exp64(far ? fmaxf(x[j], -800.f) : -fminf(x[j], 800.f));
      p[j] = far ? e : inverse64(1. + e);
    }
  } else {
    float mx = x[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) mx = fmaxf(mx, x[j]);
    const double m = wave64((double)mx, Max64());
    double z = 0.;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      p[j] = m == kOut ? 0. : (double)x[j] == m ? 1. : exp64(fmax((double)x[j] - m, -800.));
      z += p[j];
    }
    z = wave64(z, Add64());
    const double r = z > 0. ? 1. / z : 0.;
#pragma unroll
    for (int j = 0; j < EPL; ++j) p[j] *= r;
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int i = lane * EPL + j;
    c[j] = p[j];
    if (a.bias && i < a.e) c[j] += (double)a.bias[i];
    c[j] = c[j] >= kLowest ? c[j] : kLowest;
    if (i >= a.e) c[j] = kOut;
  }
  if (a.n_groups > 1) {
    const int m = a.e / a.n_groups;
    // lpg lanes a group: the two largest of its c
    const int gi = lane / lpg, sub = lane % lpg;
    double b1 = kOut, b2 = kOut;
    auto take = [&](double v) {
      b2 = fmax(b2, fmin(b1, v));
      b1 = fmax(b1, v);
    };
    if (m == lpg * EPL) {  // a group's experts are its lanes' own
#pragma unroll
      for (int j = 0; j < EPL; ++j) take(c[j]);
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j) sc[wave][lane * EPL + j] = c[j];
      __builtin_amdgcn_wave_barrier();
      if (gi < a.n_groups)
        for (int i = sub; i < m; i += lpg) take(sc[wave][gi * m + i]);
    }
    for (int o = 1; o < lpg; o <<= 1) {
      const double y1 = __shfl_xor(b1, o), y2 = __shfl_xor(b2, o);
      b2 = fmax(fmax(b2, y2), fmin(b1, y1));
      b1 = fmax(b1, y1);
    }
    double score = b1;
    if (a.group_top == 2 && m > 1) score = b1 + b2;
    score = score >= kLowest ? score : kLowest;
    int ahead = 0;
    for (int g = 0; g < a.n_groups; ++g) {
      const double v = lane64(score, g * lpg);
      ahead += v > score || (v == score && g < gi) ? 1 : 0;
    }
    const uint64_t stay = __ballot(ahead < a.top_groups && gi < a.n_groups);
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int i = lane * EPL + j;
      if (i < a.e && !((stay >> ((int)group_div.div((uint32_t)i) * lpg)) & 1)) c[j] = kOut;
    }
  }
  // a round: the lanes' largest, the wave's among them rounded to fp32 (which keeps their order), and where that
  // leaves more than one lane the wave's in 64 bits
  int my_id = -1;
  double my_p = 0., sum = 0.;
  double best;
  int at;
  auto lane_best = [&] {
    best = c[0], at = 0;
#pragma unroll
    for (int j = 1; j < EPL; ++j)
      if (c[j] > best) best = c[j], at = j;
  };
  lane_best();
  for (int r = 0; r < a.k; ++r) {
    int key = __float_as_int((float)best);
    key ^= (key >> 31) & 0x7fffffff;  // ordered as the values
    uint64_t tied = __ballot(key == wave_max(key));
    if (tied & (tied - 1)) {
      const double top = wave64(best, Max64());
      tied = __ballot(best == top);
    }
    const int from = __builtin_ctzll(tied);
    const int j0 = __builtin_amdgcn_readlane(at, from);
    double pv = p[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) pv = j == j0 ? p[j] : pv;
    const double chosen = lane64(pv, from);
    if (lane == from) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) c[j] = j == j0 ? kOut : c[j];
      lane_best();
    }
    if (lane == r) my_id = from * EPL + j0, my_p = chosen;
    sum += chosen;
  }
  if (lane < a.k) {
    double w = my_p;
    if (a.renormalize) w = sum > 0. ? w / sum : 0.;
    w *= (double)a.scale;
    ids[lane] = my_id;
    weights[lane] = (float)w;
  }
}

// ---------------------------------------------------------------- the combination
//
// out = residual + sum_j w_j y_j: k + 2 rows of memory traffic for k products a value, so memory bounds it.
// A thread holds 16 bytes of a row and has the loads of four positions in flight, ids or not (a load that waits
// for its id: 4096 tokens of 8 x 4096 values 86 us, so 63, 5.3 TB/s; 16 tokens of 4 3.2 us).  Rows that are no
// multiples of 16 bytes go one value a thread: 8 x 4095 values in bf16 83 us, in fp32, whose 4 bytes a lane suffice, 117
// against 124 of 4096.  A token of fewer positions than are in flight loads its last one again, out of the cache: one
// position of 4096 values 17 us, 5.9 TB/s, but of 4095, with 8 in flight, 60.

template <int DT> struct Elem;
template <> struct Elem<DT_F32> {
  using Raw = float;
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float v) { return v; }
};
template <> struct Elem<DT_F16> {
  using Raw = uint16_t;
  static __device__ __forceinline__ float get(uint16_t v) { return f16_bits_to_f32(v); }
  static __device__ __forceinline__ uint16_t put(float v) { return (uint16_t)f32_to_f16_bits(v); }
};
template <> struct Elem<DT_BF16> {
  using Raw = uint16_t;
  static __device__ __forceinline__ float get(uint16_t v) { return bf16_bits_to_f32(v); }
  static __device__ __forceinline__ uint16_t put(float v) { return (uint16_t)f32_to_bf16_bits(v); }
};

// V values a thread (16 bytes, or 1 where rows are not multiples of 16 bytes); JB positions at a time, all of their
// loads in flight, those of positions that are not wanted too.  UNIFORM: a wave lies within one token, whose
// ids and weights are then scalar loads.
template <int DT, int V, bool UNIFORM>
__global__ __launch_bounds__(256) void combine_kernel(const CombineArgs a, FastDiv row_div, int64_t units) {
  using E = Elem<DT>;
  using Raw = typename E::Raw;
  struct __attribute__((aligned(V * sizeof(Raw)))) Vec {
    Raw v[V];
  };
  constexpr int JB = V == 1 ? 8 : 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= units) return;
  const int64_t per = a.n / V;
  int64_t tok = row_div.div((uint32_t)i);
  if (UNIFORM) tok = __builtin_amdgcn_readfirstlane((int)tok);
  const int64_t c = i - tok * per;
  const Vec* y = (const Vec*)a.y + tok * a.k * per + c;
  const int k = (int)a.k;
  float acc[V];
#pragma unroll
  for (int x = 0; x < V; ++x) acc[x] = 0.f;
  if (a.residual) {
    const Vec r = ((const Vec*)a.residual)[i];
#pragma unroll
    for (int x = 0; x < V; ++x) acc[x] = E::get(r.v[x]);
  }
  for (int j0 = 0; j0 < k; j0 += JB) {
    Vec r[JB];
    float w[JB];
    bool on[JB];
#pragma unroll
    for (int j = 0; j < JB; ++j) {
      const int jj = min(j0 + j, k - 1);
      r[j] = y[jj * per];
      w[j] = a.weights[tok * k + jj];
      on[j] = j0 + j < k;
      if (a.ids) {
        const int64_t id = a.ids[tok * k + jj];
        on[j] = on[j] && id >= 0 && id < a.e;
      }
    }
#pragma unroll
    for (int j = 0; j < JB; ++j)
      if (on[j]) {
#pragma unroll
        for (int x = 0; x < V; ++x) acc[x] = __builtin_fmaf(w[j], E::get(r[j].v[x]), acc[x]);
      }
  }
  Vec o;
#pragma unroll
  for (int x = 0; x < V; ++x) o.v[x] = E::put(acc[x]);
  ((Vec*)a.out)[i] = o;
}

template <int DT> hipError_t combine(const CombineArgs& a, hipStream_t s) {
  constexpr int V = DT == DT_F32 ? 4 : 8;
  auto whole = [](const void* p) { return (uintptr_t)p % 16 == 0; };
  const bool wide = a.n % V == 0 && whole(a.y) && whole(a.out) && whole(a.residual);
  const int64_t per = wide ? a.n / V : a.n, units = a.t * per;
  const unsigned grid = (unsigned)((units + 255) / 256);
  const FastDiv div = fast_div((uint32_t)per);
  if (!wide)
    combine_kernel<DT, 1, false><<<grid, 256, 0, s>>>(a, div, units);
  else if (per % 64 == 0)
    combine_kernel<DT, V, true><<<grid, 256, 0, s>>>(a, div, units);
  else
    combine_kernel<DT, V, false><<<grid, 256, 0, s>>>(a, div, units);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_select_experts(const SelectArgs& a, hipStream_t s) {
  const unsigned grid = (unsigned)((a.t + 3) / 4);
  const FastDiv div = fast_div((uint32_t)(a.e / a.n_groups));
  int lpg = 64;  // lanes of a group
  while (lpg * a.n_groups > 64) lpg /= 2;
  if (a.e <= 64)
    select_kernel<1><<<grid, 256, 0, s>>>(a, div, lpg);
  else if (a.e <= 128)
    select_kernel<2><<<grid, 256, 0, s>>>(a, div, lpg);
  else if (a.e <= 256)
    select_kernel<4><<<grid, 256, 0, s>>>(a, div, lpg);
  else if (a.e <= 512)
    select_kernel<8><<<grid, 256, 0, s>>>(a, div, lpg);
  else
    select_kernel<16><<<grid, 256, 0, s>>>(a, div, lpg);
  return hipGetLastError();
}

hipError_t launch_combine_experts(const CombineArgs& a, hipStream_t s) {
  return a.dt == DT_F32 ? combine<DT_F32>(a, s) : a.dt == DT_F16 ? combine<DT_F16>(a, s) : combine<DT_BF16>(a, s);
}

}  // namespace ql
