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

template <typename T, int L, int ROWS>
__global__ __launch_bounds__(256) void norm_rope_kernel(const NormRopeArgs a, FastDiv per_token, int groups,
                                                        int64_t units) {
  const int lane = threadIdx.x & 63;
  const int c = lane % L;  // the lane's 8 values of a row
  const int64_t unit = (int64_t)blockIdx.x * (256 / L) + threadIdx.x / L;
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
template <typename T> hipError_t run_l(const NormRopeArgs& a, hipStream_t s) {
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

}  // namespace ql
