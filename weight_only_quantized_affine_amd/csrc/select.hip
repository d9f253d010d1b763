// Around routed experts: the choice of each token's experts from its router logits, and the weighted sum of
// their outputs.
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
// lowest index: a round takes the lane's largest, the wave's by DPP, and a ballot.

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
struct Max64 {
  __device__ __forceinline__ double operator()(double a, double b) const { return fmax(a, b); }
};
struct Add64 {
  __device__ __forceinline__ double operator()(double a, double b) const { return a + b; }
};

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
    for (int j = 0; j < EPL; ++j) p[j] = 1. / (1. + exp(-(double)x[j]));
  } else {
    float mx = x[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) mx = fmaxf(mx, x[j]);
    const double m = wave64((double)mx, Max64());
    double z = 0.;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      p[j] = m == kOut ? 0. : (double)x[j] == m ? 1. : exp((double)x[j] - m);
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
#pragma unroll
    for (int j = 0; j < EPL; ++j) sc[wave][lane * EPL + j] = c[j];
    __builtin_amdgcn_wave_barrier();
    // lpg lanes a group: the two largest of its c
    const int gi = lane / lpg, sub = lane % lpg;
    double b1 = kOut, b2 = kOut;
    if (gi < a.n_groups) {
      for (int i = sub; i < m; i += lpg) {
        const double v = sc[wave][gi * m + i];
        b2 = fmax(b2, fmin(b1, v));
        b1 = fmax(b1, v);
      }
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
  int my_id = -1;
  double my_p = 0., sum = 0.;
  for (int r = 0; r < a.k; ++r) {
    double best = c[0];
#pragma unroll
    for (int j = 1; j < EPL; ++j) best = fmax(best, c[j]);
    const double top = wave64(best, Max64());
    const int from = __builtin_ctzll(__ballot(best == top));
    int at = 0;
    double pv = p[0];
#pragma unroll
    for (int j = EPL - 1; j >= 0; --j)
      if (c[j] == top) at = j, pv = p[j];
    const int j0 = __builtin_amdgcn_readlane(at, from);
    const double chosen = lane64(pv, from);
    if (lane == from) {
#pragma unroll
      for (int j = 0; j < EPL; ++j) c[j] = j == j0 ? kOut : c[j];
    }
    if (lane == r) my_id = from * EPL + j0, my_p = chosen;
    sum += chosen;
  }
  if (lane < a.k) {
    double w = my_p * (double)a.scale;
    if (a.renormalize) w = sum > 0. ? w / sum : 0.;
    ids[lane] = my_id;
    weights[lane] = (float)w;
  }
}

// ---------------------------------------------------------------- the combination
//
// out = residual + sum_j w_j y_j: k + 2 rows of memory traffic for k products a value, so memory bounds it.
// A thread holds 16 bytes of a row and has the loads of all its token's positions in flight.

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

// V values a thread (16 bytes, or 1 where rows are not multiples of 16 bytes); JB positions at a time.
template <int DT, int V> __global__ __launch_bounds__(256) void combine_kernel(const CombineArgs a, FastDiv row_div, int64_t units) {
  using E = Elem<DT>;
  using Raw = typename E::Raw;
  struct __attribute__((aligned(V * sizeof(Raw)))) Vec {
    Raw v[V];
  };
  constexpr int JB = 8;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= units) return;
  const int64_t per = a.n / V;
  const int64_t tok = row_div.div((uint32_t)i), c = i - tok * per;
  float acc[V];
#pragma unroll
  for (int x = 0; x < V; ++x) acc[x] = 0.f;
  if (a.residual) {
    const Vec r = ((const Vec*)a.residual)[i];
#pragma unroll
    for (int x = 0; x < V; ++x) acc[x] = E::get(r.v[x]);
  }
  const Vec* y = (const Vec*)a.y + tok * a.k * per + c;
  for (int64_t j0 = 0; j0 < a.k; j0 += JB) {
    Vec r[JB];
    float w[JB];
    bool on[JB];
#pragma unroll
    for (int j = 0; j < JB; ++j) {
      on[j] = j0 + j < a.k;
      if (on[j] && a.ids) {
        const int64_t id = a.ids[tok * a.k + j0 + j];
        on[j] = id >= 0 && id < a.e;
      }
      w[j] = 0.f;
      if (on[j]) w[j] = a.weights[tok * a.k + j0 + j], r[j] = y[(j0 + j) * per];
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
  if (a.n % V == 0 && whole(a.y) && whole(a.out) && whole(a.residual)) {
    const int64_t units = a.t * (a.n / V);
    combine_kernel<DT, V><<<(unsigned)((units + 255) / 256), 256, 0, s>>>(a, fast_div((uint32_t)(a.n / V)), units);
  } else {
    const int64_t units = a.t * a.n;
    combine_kernel<DT, 1><<<(unsigned)((units + 255) / 256), 256, 0, s>>>(a, fast_div((uint32_t)a.n), units);
  }
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
