// Per-head RMS norm and position rotation of q and k, and the append of k and v to a paged cache.
//
// Row (token, head) of d values: r = 1 / sqrt(mean x^2 + eps), y = x r w, then for each of the
// rot/2 pairs (a, b) the rotation (a c - b s, b c + a s) with the token's (c, s) from the table;
// fp32 throughout, rounded once when stored.  Pairs are (i, i + rot/2), or (2i, 2i + 1) when
// interleaved.
//
// Bound by memory at many tokens (each row is read and written once) and by the launch at few.  A
// group of lanes with 8 values each holds a row (16 lanes at d = 128) and takes ROWS heads of one
// token: their loads are in flight together and the token's table values are read once for all of
// them.  The mean is a reduction by DPP within 16 lanes, and a value's partner lies in a lane
// rot/16 further in its group.
//
// Measured (bf16, 40 heads of 128): 8192 tokens 34 us, 172 MB, 5.1 TB/s (a large copy reaches 5.1
// here); append of 4096 tokens 19 us; one token 2.9 us.
//
// Append to a cache in 4 bits: the rows of k (in 64 bits up to their rounding, since a code hangs on the last
// bits) and of v are quantized where they are, 8 values and one word of codes a lane, a group's
// smallest and largest value by DPP within its 4, 8 or 16 lanes.  Rows of k and v are taken token after token of
// one head, so that neighbouring groups of lanes write neighbouring rows of a head-major page (head after
// head: 4096 tokens 41 us, so 25).  Measured (bf16, 32 + 8 + 8 heads of 128, groups of 64): 64 tokens of 16 + 8 + 8
// heads 4.4 us, 4096 tokens 25 us, 3.5 TB/s (17 of it memory, the rest the rows' work on the vector units);
// reading 4096 tokens back 7.8 us.
#include "head_common.hpp"

namespace ql {
namespace {

// x + x of the lane that DPP control CTRL names (within 16 lanes).
template <int CTRL> __device__ __forceinline__ float add_dpp(float x) {
  const int y = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, false);
  return x + __builtin_bit_cast(float, y);
}
// Sum over aligned groups of L lanes, in every lane.
template <int L> __device__ __forceinline__ float group_sum(float x) {
  if (L >= 2) x = add_dpp<0xB1>(x);   // lane ^ 1
  if (L >= 4) x = add_dpp<0x4E>(x);   // lane ^ 2
  if (L >= 8) x = add_dpp<0x141>(x);  // mirrored 8 lanes: the other four
  if (L >= 16) x = add_dpp<0x140>(x);  // mirrored 16 lanes: the other eight
  if (L >= 32) x += __shfl_xor(x, 16);
  if (L >= 64) x += __shfl_xor(x, 32);
  return x;
}

template <typename T> __device__ __forceinline__ void unpack8(u32x4_t w, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = param_to_f32<T>(w[i] & 0xffffu);
    f[2 * i + 1] = param_to_f32<T>(w[i] >> 16);
  }
}
// 8 norm weights at chunk c in their dtype.
__device__ __forceinline__ void weights8(const void* w, int wdt, int c, float* f) {
  if (wdt == DT_F32) {
    const f32x4_t a = ((const f32x4_t*)w)[2 * c], b = ((const f32x4_t*)w)[2 * c + 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = a[i], f[4 + i] = b[i];
  } else if (wdt == DT_BF16) {
    unpack8<BF16>(((const u32x4_t*)w)[c], f);
  } else {
    unpack8<F16>(((const u32x4_t*)w)[c], f);
  }
}

// The same for sums in 64 bits.
template <int CTRL> __device__ __forceinline__ double add_dpp(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xf, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xf, 0xf, false);
  return x + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// The value 8 lanes further in 16.
__device__ __forceinline__ double turn8(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, 0x128, 0xf, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), 0x128, 0xf, 0xf, false);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <int L> __device__ __forceinline__ double group_sum(double x) {
  if (L >= 2) x = add_dpp<0xB1>(x);
  if (L >= 4) x = add_dpp<0x4E>(x);
  if (L >= 8) x = add_dpp<0x141>(x);
  if (L >= 16) x = add_dpp<0x140>(x);
  if (L >= 32) x += __shfl_xor(x, 16);
  if (L >= 64) x += __shfl_xor(x, 32);
  return x;
}

// 1 / sqrt(x) within 2^-50 of its value: the approximate one (2^-26 and better) after one step of third order.
__device__ __forceinline__ double rsqrt64(double x) {
  const double r = __builtin_amdgcn_rsq(x);
  const double e = __builtin_fma(-x * r, r, 1.);
  return __builtin_fma(r * e, __builtin_fma(0.375, e, 0.5), r);
}

// Monotone integer key of an fp32 value (-0 < +0), and back.
__device__ __forceinline__ int32_t order_key(float f) {
  const int32_t i = __float_as_int(f);
  return i ^ ((i >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float from_order_key(int32_t i) { return __int_as_float(i ^ ((i >> 31) & 0x7fffffff)); }
template <int CTRL> __device__ __forceinline__ void span_dpp(int32_t& lo, int32_t& hi) {
  lo = min(lo, __builtin_amdgcn_update_dpp(0, lo, CTRL, 0xf, 0xf, false));
  hi = max(hi, __builtin_amdgcn_update_dpp(0, hi, CTRL, 0xf, 0xf, false));
}
// The codes of a lane's 8 values and the word of their group (of `lanes` lanes): scale (max - min) / 15 and
// bias min rounded to fp16, codes the nearest levels of those, as qlinear_quantize; magnitudes past 2^15
// and NaN (the largest or smallest key) give scale 0 and bias NaN.
__device__ __forceinline__ uint32_t quantize8(const float* f, int lanes, uint32_t& group) {
  int32_t lo = order_key(f[0]), hi = lo;
#pragma unroll
  for (int j = 1; j < 8; ++j) lo = min(lo, order_key(f[j])), hi = max(hi, order_key(f[j]));
  span_dpp<0xB1>(lo, hi);
  span_dpp<0x4E>(lo, hi);
  if (lanes >= 8) span_dpp<0x141>(lo, hi);
  if (lanes >= 16) span_dpp<0x140>(lo, hi);
  const float mn = from_order_key(lo), mx = from_order_key(hi);
  const bool held = __builtin_fabsf(mn) <= 32768.f && __builtin_fabsf(mx) <= 32768.f;
  const uint32_t sb = f32_to_f16_bits(__fdiv_rn(mx - mn, 15.f)), bb = f32_to_f16_bits(mn);
  const float s = f16_bits_to_f32(sb), b = f16_bits_to_f32(bb);
  group = held ? sb | (bb << 16) : 0x7e000000u;
  if (!held || s == 0.f) return 0;
  // rint of the rounded quotient: an approximate one and its residual tell it, but next to a half
  const float inv = __builtin_amdgcn_rcpf(s), edge = s * (0.5f - 0x1p-18f);
  float d[8], r[8];
  bool near_half = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    d[j] = f[j] - b;
    r[j] = __builtin_rintf(d[j] * inv);
    near_half |= !(__builtin_fabsf(__builtin_fmaf(-r[j], s, d[j])) < edge);
  }
  if (near_half) {
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = __builtin_rintf(__fdiv_rn(d[j], s));
  }
  uint32_t word = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) word |= (uint32_t)__builtin_amdgcn_fmed3f(r[j], 0.f, 15.f) << (4 * j);
  return word;
}

// The cosines and sines of a position's row for the 8 values of chunk c; second: of the pairs' second values
// (not interleaved: sn holds the sign).
__device__ __forceinline__ void cos_sin8(const float* at, int rot, bool interleaved, int c, bool second, float* cs, float* sn) {
  const f32x4_t* row = (const f32x4_t*)at;
  const int n = rot / 8;  // 4-value words of the cosines
  if (interleaved) {
    const f32x4_t u = row[c], v = row[n + c];
#pragma unroll
    for (int i = 0; i < 4; ++i) cs[2 * i] = cs[2 * i + 1] = u[i], sn[2 * i] = sn[2 * i + 1] = v[i];
  } else {
    const int b = 2 * (second ? c - rot / 16 : c);
    const f32x4_t u0 = row[b], u1 = row[b + 1], v0 = row[n + b], v1 = row[n + b + 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cs[i] = u0[i], cs[4 + i] = u1[i];
      sn[i] = second ? v0[i] : -v0[i], sn[4 + i] = second ? v1[i] : -v1[i];
    }
  }
}

// Rows of unit (block `block`): ROWS heads of one token.
template <typename T, int L, int ROWS>
__device__ __forceinline__ void norm_rope_rows(const NormRopeArgs& a, int block, FastDiv per_token, int groups,
                                               int64_t units) {
  const int lane = threadIdx.x & 63;
  const int c = lane % L;  // the lane's 8 values of a row
  const int64_t unit = (int64_t)block * (256 / L) + threadIdx.x / L;
  if (unit >= units) return;  // whole groups of lanes
  const int64_t tok = (int64_t)per_token.div((uint32_t)unit);
  const int h0 = (int)(unit - tok * groups) * ROWS;
  const int heads = a.hq + a.hk + a.hv;
  const bool on = 8 * c < a.d;

  int64_t page = -1;
  int at = 0;
  if (a.slots) {
    const int64_t slot = a.slots[tok];
    if (slot >= 0 && slot < a.n_slots) {
      page = a.page_div.div((uint32_t)slot);
      at = (int)(slot - page * a.page_size);
    }
  }
  // loads of every row first
  u32x4_t x[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int h = h0 + i;
    x[i] = u32x4_t{0, 0, 0, 0};
    if (h < heads && on) {
      const uint8_t* p = h < a.hq            ? a.q + tok * a.q_ts + h * a.q_hs
                         : h < a.hq + a.hk ? a.k + tok * a.k_ts + (h - a.hq) * a.k_hs
                                             : a.v + tok * a.v_ts + (h - a.hq - a.hk) * a.v_hs;
      x[i] = *(const u32x4_t*)(p + 16 * c);
    }
  }
  // the token's cosines and sines for this lane's values
  float cs[8] = {}, sn[8] = {};
  bool known = true;
  const bool turned = 8 * c < a.rot;
  const int half = a.rot / 16;  // lanes between the two values of a pair
  const bool second = !a.interleaved && c >= half;
  if (a.rot > 0) {
    const int64_t pos = a.positions[tok];
    known = pos >= 0 && pos < a.max_pos;
    if (turned) {
      const f32x4_t* row = (const f32x4_t*)(a.cos_sin + (known ? pos : 0) * a.rot);
      const int n = a.rot / 8;  // 4-value words of the cosines
      if (a.interleaved) {
        const f32x4_t u = row[c], v = row[n + c];
#pragma unroll
        for (int i = 0; i < 4; ++i) cs[2 * i] = cs[2 * i + 1] = u[i], sn[2 * i] = sn[2 * i + 1] = v[i];
      } else {
        const int b = 2 * (second ? c - half : c);
        const f32x4_t u0 = row[b], u1 = row[b + 1], v0 = row[n + b], v1 = row[n + b + 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          cs[i] = u0[i], cs[4 + i] = u1[i];
          sn[i] = second ? v0[i] : -v0[i], sn[4 + i] = second ? v1[i] : -v1[i];
        }
      }
    }
  }
  float w[8];
  const void* loaded = nullptr;
  const float inv_d = 1.0f / (float)a.d;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int h = h0 + i;
    const bool is_q = h < a.hq, is_v = h >= a.hq + a.hk;
    const void* wp = is_q ? a.q_weight : is_v ? nullptr : a.k_weight;
    float f[8];
    unpack8<T>(x[i], f);
    if (wp) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = __builtin_fmaf(f[j], f[j], ss);
      ss = group_sum<L>(ss);
      const float r = __builtin_amdgcn_rsqf(__builtin_fmaf(ss, inv_d, a.eps));
      if (wp != loaded) {  // most heads share the weights of the one before
        if (on) weights8(wp, a.wdt, c, w);
        loaded = wp;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = f[j] * r * w[j];
    }
    if (a.rot > 0) {
      float y[8];
      if (a.interleaved) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          y[j] = f[j] * cs[j] - f[j + 1] * sn[j];
          y[j + 1] = f[j + 1] * cs[j] + f[j] * sn[j];
        }
      } else {
        float o[8];
        if (L == 16 && half == 8) {  // the other half of the row: a rotation of 16 lanes by 8
#pragma unroll
          for (int j = 0; j < 8; ++j)
            o[j] = __builtin_bit_cast(
                float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, f[j]), 0x128, 0xf, 0xf, false));
        } else {
          const int from = (lane & ~(L - 1)) | ((second ? c - half : c + half) & (L - 1));
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = __shfl(f[j], from);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = f[j] * cs[j] + o[j] * sn[j];  // sn holds the sign
      }
      if (turned) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = y[j];
      }
    }
    if (h >= heads || !on) continue;
    u32x4_t o = x[i];
    if (!is_v) {
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = known ? pack2(T{}, f[2 * j], f[2 * j + 1]) : 0u;
    }
    uint8_t* p;
    if (is_q) {
      p = a.q_out + tok * a.qo_ts + h * a.qo_hs;
    } else {
      const int hh = is_v ? h - a.hq - a.hk : h - a.hq;
      p = is_v ? a.v_out + hh * a.vo_hs : a.k_out + hh * a.ko_hs;
      if (a.slots) {
        if (page < 0) continue;  // a token without a slot is not stored
        p += page * a.page_stride + at * (is_v ? a.vo_ts : a.ko_ts);
      } else {
        p += tok * a.ko_ts;
      }
    }
    if (ROWS > 1)
      __builtin_nontemporal_store(o, (u32x4_t*)(p + 16 * c));
    else
      *(u32x4_t*)(p + 16 * c) = o;
  }
}

template <typename T, int L, int ROWS>
__global__ __launch_bounds__(256) void norm_rope_kernel(const NormRopeArgs a, FastDiv per_token, int groups,
                                                        int64_t units) {
  norm_rope_rows<T, L, ROWS>(a, blockIdx.x, per_token, groups, units);
}

// One row of k or v: normed, rotated (k) and quantized, 8 values and a word of codes a lane.
template <typename T, int L>
__device__ __forceinline__ void quantized_row(const Append4Args& a, int64_t tok, int h, bool is_v) {
  const int lane = threadIdx.x & 63;
  const int c = lane % L;
  const bool on = 8 * c < a.d;
  const int64_t slot = a.slots[tok];
  const uint8_t* p = is_v ? a.v + tok * a.v_ts + h * a.v_hs : a.k + tok * a.k_ts + h * a.k_hs;
  u32x4_t x = {0, 0, 0, 0};
  if (on) x = *(const u32x4_t*)(p + 16 * c);
  float f[8];
  unpack8<T>(x, f);
  if (!is_v) {
    const int half = a.rot / 16;  // lanes between the two values of a pair
    const bool turned = 8 * c < a.rot, second = !a.interleaved && c >= half;
    bool known = true;
    float cs[8] = {}, sn[8] = {};
    if (a.rot > 0) {
      const int64_t pos = a.positions[tok];
      known = pos >= 0 && pos < a.max_pos;
      if (turned) cos_sin8(a.cos_sin + (known ? pos : 0) * a.rot, a.rot, a.interleaved, c, second, cs, sn);
    }
    double y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = f[j];
    if (a.k_weight) {
      float w[8] = {};
      if (on) weights8(a.k_weight, a.wdt, c, w);
      double ss = 0.;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = __builtin_fma((double)f[j], (double)f[j], ss);  // exact squares: bf16's leave fp32
      const double r = rsqrt64(__builtin_fma(group_sum<L>(ss), a.inv_d, (double)a.eps));
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = y[j] * r * w[j];
    }
    if (a.rot > 0) {
      double z[8];
      if (a.interleaved) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          z[j] = y[j] * cs[j] - y[j + 1] * sn[j];
          z[j + 1] = y[j + 1] * cs[j] + y[j] * sn[j];
        }
      } else {
        const int from = (lane & ~(L - 1)) | ((second ? c - half : c + half) & (L - 1));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const double o = L == 16 && half == 8 ? turn8(y[j]) : __shfl(y[j], from);
          z[j] = y[j] * cs[j] + o * sn[j];  // sn holds the sign
        }
      }
      if (turned) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = z[j];
      }
    }
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const uint32_t two = known ? pack2(T{}, (float)y[j], (float)y[j + 1]) : 0u;
      f[j] = param_to_f32<T>(two & 0xffffu), f[j + 1] = param_to_f32<T>(two >> 16);
    }
  }
  uint32_t group;
  const uint32_t word = quantize8(f, a.group / 8, group);
  if (!on || slot < 0 || slot >= a.n_slots) return;  // a token without a slot is not stored
  const int64_t page = a.page_div.div((uint32_t)slot), at = slot - page * a.page_size;
  uint8_t* cp = (is_v ? a.v_out : a.k_out) + page * a.page_stride + at * a.ko_ts + h * a.ko_hs;
  ((uint32_t*)cp)[c] = word;
  const int per = a.group / 8;
  uint32_t* gp = (is_v ? a.v_groups : a.k_groups) + page * a.group_ps + at * a.group_ts + h * a.group_hs;
  if ((c & (per - 1)) == 0) gp[c / per] = group;
}

// The rows of q as above in the first q_blocks blocks; then those of k and v, a head's tokens side by side, so
// that a wave's rows are neighbours in a page (4096 tokens, 32 heads on 8: 25 us; with a token's rows
// side by side 31, and 41 where a wave held q next to k and v).
template <typename T, int L, int ROWS>
__global__ __launch_bounds__(256) void append4_kernel(const Append4Args a, FastDiv per_token, int groups, int64_t q_units,
                                                      int q_blocks, FastDiv per_head) {
  if ((int)blockIdx.x < q_blocks) {
    norm_rope_rows<T, L, ROWS>(a, blockIdx.x, per_token, groups, q_units);
  } else {
    const int64_t unit = (int64_t)(blockIdx.x - q_blocks) * (256 / L) + threadIdx.x / L;
    if (unit >= a.t * 2 * a.cache_heads) return;  // whole groups of lanes
    const int h = (int)per_head.div((uint32_t)unit);
    const bool is_v = h >= a.cache_heads;
    quantized_row<T, L>(a, unit - (int64_t)h * a.t, is_v ? h - a.cache_heads : h, is_v);
  }
}

template <typename T, int L, int ROWS> hipError_t run_rows(const NormRopeArgs& a, hipStream_t s) {
  const int groups = (a.hq + a.hk + a.hv + ROWS - 1) / ROWS;
  const int64_t units = a.t * groups;
  const unsigned grid = (unsigned)((units + 256 / L - 1) / (256 / L));
  norm_rope_kernel<T, L, ROWS><<<grid, 256, 0, s>>>(a, fast_div((uint32_t)groups), groups, units);
  return hipGetLastError();
}
template <typename T, int L> hipError_t run(const NormRopeArgs& a, hipStream_t s) {
  // Waves when each lane holds one row: below 16 a compute unit the launch's latency counts and one
  // row a lane is shortest (1, 2, 4 rows: 1 token x 40 rows of 128 2.9, 3.3, 4.2 us; 256 tokens 3.6,
  // 3.9, 4.8); from 64 on the rows in flight count (512 tokens 4.9, 4.5, 5.3; 1024 8.5, 6.2, 6.8;
  // 2048 12.5, 10.8, 10.0; 4096 21.3, 17.6, 17.0).  Outputs of that size pass the caches on the way
  // to memory (non-temporal stores, 8192 tokens: 41 -> 35 us; what reads them next is not slower).
  const int64_t waves = a.t * (a.hq + a.hk + a.hv) * L / 64;
  return waves < 4096 ? run_rows<T, L, 1>(a, s) : waves < 16384 ? run_rows<T, L, 2>(a, s) : run_rows<T, L, 4>(a, s);
}
// Rows a lane of q as above, by the rows of q alone.
template <typename T, int L, int ROWS> hipError_t append_rows(const Append4Args& a, hipStream_t s) {
  const int groups = (a.hq + ROWS - 1) / ROWS;
  const int64_t units = a.t * groups, rows = a.t * 2 * a.cache_heads;
  const int per = 256 / L, q_blocks = (int)((units + per - 1) / per);
  const unsigned grid = (unsigned)(q_blocks + (rows + per - 1) / per);
  append4_kernel<T, L, ROWS><<<grid, 256, 0, s>>>(a, fast_div((uint32_t)(groups > 0 ? groups : 1)), groups, units, q_blocks,
                                                  fast_div((uint32_t)a.t));
  return hipGetLastError();
}
template <typename T, int L> hipError_t run(const Append4Args& a, hipStream_t s) {
  const int64_t waves = a.t * a.hq * L / 64;
  return waves < 4096 ? append_rows<T, L, 1>(a, s) : waves < 16384 ? append_rows<T, L, 2>(a, s) : append_rows<T, L, 4>(a, s);
}
template <typename T, typename Args> hipError_t run_l(const Args& a, hipStream_t s) {
  const int n = a.d / 8;
  if (n <= 8) return run<T, 8>(a, s);
  if (n <= 16) return run<T, 16>(a, s);
  if (n <= 32) return run<T, 32>(a, s);
  return run<T, 64>(a, s);
}

}  // namespace

hipError_t launch_norm_rope(const NormRopeArgs& a, int dt, hipStream_t s) {
  return dt == DT_BF16 ? run_l<BF16>(a, s) : run_l<F16>(a, s);
}
hipError_t launch_append4(const Append4Args& a, int dt, hipStream_t s) {
  return dt == DT_BF16 ? run_l<BF16>(a, s) : run_l<F16>(a, s);
}

namespace {

// One lane for 8 values of a row of k or v.
template <typename T> __global__ __launch_bounds__(256) void read4_kernel(const Read4Args a, FastDiv per_row, FastDiv per_token, int64_t n) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const int64_t unit = per_row.div((uint32_t)i);  // (token, k or v, head)
  const int c = (int)(i - unit * (a.d / 8));
  const int64_t tok = per_token.div((uint32_t)unit);
  const int h2k = (int)(unit - tok * 2 * a.hk);
  const bool is_v = h2k >= a.hk;
  const int h = is_v ? h2k - a.hk : h2k;
  const int64_t slot = a.slots[tok];
  u32x4_t o = {0, 0, 0, 0};
  if (slot >= 0 && slot < a.n_slots) {
    const int64_t page = a.page_div.div((uint32_t)slot), at = slot - page * a.page_size;
    const uint8_t* cp = (is_v ? a.v : a.k) + page * a.page_stride + at * a.token_stride + h * a.head_stride;
    const uint32_t* gp = (is_v ? a.vg : a.kg) + page * a.group_ps + at * a.group_ts + h * a.group_hs;
    const uint32_t w = ((const uint32_t*)cp)[c], g = gp[c / (a.group / 8)];
    const float s = f16_bits_to_f32(g & 0xffffu), b = f16_bits_to_f32(g >> 16);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = pack2(T{}, __builtin_fmaf((float)((w >> (8 * j)) & 15), s, b), __builtin_fmaf((float)((w >> (8 * j + 4)) & 15), s, b));
  }
  uint8_t* p = is_v ? a.v_out + tok * a.vo_ts + h * a.vo_hs : a.k_out + tok * a.ko_ts + h * a.ko_hs;
  *(u32x4_t*)(p + 16 * c) = o;
}

}  // namespace

hipError_t launch_read4(const Read4Args& a, int dt, hipStream_t s) {
  const int64_t n = a.t * 2 * a.hk * (a.d / 8);
  const unsigned grid = (unsigned)((n + 255) / 256);
  const FastDiv row = fast_div((uint32_t)(a.d / 8)), tok = fast_div((uint32_t)(2 * a.hk));
  if (dt == DT_BF16)
    read4_kernel<BF16><<<grid, 256, 0, s>>>(a, row, tok, n);
  else
    read4_kernel<F16><<<grid, 256, 0, s>>>(a, row, tok, n);
  return hipGetLastError();
}

}  // namespace ql
