// Paged attention, few rows: sequences whose new tokens times query heads per kv head are at most
// 16 or 32 rows (single tokens, drafted tokens).
//
// The cache is read once and bounds the call: 2 D multiply-adds per row and cached value pair
// leave the matrix cores mostly idle at 32 rows.  So the split serves the memory: all (sequence,
// kv head) items are laid end to end in tiles of 128 positions, and each workgroup takes an equal
// run of tiles whatever the sequences' lengths; an item cut between workgroups leaves its pieces
// in the workspace for the joining kernel.  In a workgroup each of the 4 waves streams its own 32
// positions of a tile with its own copies into LDS and its own waits (no barrier in the loop): K
// of the next tile is in flight while the scores are turned into P and V is multiplied, V while
// the scores are computed.  The waves' sums join in LDS at the end of an item.
//
// Measured (bf16, 32 heads on 8 of 128): one sequence of 131071 positions, 537 MB in 94 us, 5.7 TB/s
// (a plain read of 1 GB reaches 5.9 here); 64 ragged sequences, 762 MB in 133 us, 5.7 TB/s; one
// sequence of 1025 positions with 16 heads on 8, 12 us, the latency of two launches and of the chain
// lengths, page ids, keys.
#include "attn_few.hpp"

namespace ql {
namespace {

// P V of one tile of 32 positions x 16 columns into o (D/16 tiles of 16 values).
template <typename T, int D>
__device__ __forceinline__ void few_pv(const uint8_t* sv, int lane, u32x4_t p, f32x4_t* o) {
  const int g = lane >> 4, l = lane & 15;
  const int row = 4 * g + (l >> 2);
#pragma unroll
  for (int dt = 0; dt < D / 16; ++dt) {
    const int c = 2 * dt + ((l & 3) >> 1);
    const uint8_t* at = sv + row * (D * 2) + 8 * (l & 1);
    const s16x4_t v0 = read_tr(at + (c ^ swz_v<D>(row)) * 16);
    const s16x4_t v1 = read_tr(at + 16 * D * 2 + (c ^ swz_v<D>(row + 16)) * 16);
    const u32x2_t w0 = __builtin_bit_cast(u32x2_t, v0), w1 = __builtin_bit_cast(u32x2_t, v1);
    o[dt] = mfma16(T{}, u32x4_t{w0[0], w0[1], w1[0], w1[1]}, p, o[dt]);
  }
}

template <typename T, int D> __device__ __forceinline__ bool few_v_nonfinite(const uint8_t* sv, int lane) {
  asm volatile("" : "+v"(lane));
  uint32_t acc = 0;
#pragma unroll
  for (int i = 0; i < 32 * D * 2 / 1024; ++i) {
    const u32x4_t w = *(const u32x4_t*)(sv + i * 1024 + lane * 16);
    for (int j = 0; j < 4; ++j) acc |= nonfinite2<T>(w[j]);
  }
  return __any((acc & 0x80008000u) != 0);
}

// Adds the non-finite values of the wave's V tile to the columns whose P is not zero, and leaves
// zeros in their place.
template <typename T, int D, int NC>
__device__ __forceinline__ void few_nonfinite(uint8_t* sv, int lane, const u32x4_t* p, f32x4_t (*o)[D / 16]) {
  asm volatile("" : "+v"(lane));  // the addresses stay in this rare path
  const int g = lane >> 4, col = lane & 15;
#pragma unroll 1
  for (int j = 0; j < 32; ++j) {
    // P of key j: word (j & 3) / 2 of its 16 keys, in the lanes of (j & 15) / 4
    bool on[NC];
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const uint32_t a = j < 16 ? p[n][0] : p[n][2], b = j < 16 ? p[n][1] : p[n][3];
      const uint32_t w = __shfl((j & 2) ? b : a, 16 * ((j & 15) >> 2) + col);
      on[n] = ((j & 1) ? w >> 16 : w) & 0x7fffu;
    }
#pragma unroll
    for (int dt = 0; dt < D / 16; ++dt) {
      const int c = 2 * dt + (g >> 1);
      const u32x2_t w = *(const u32x2_t*)(sv + j * (D * 2) + (c ^ swz_v<D>(j)) * 16 + 8 * (g & 1));
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float a, b;
          only_nonfinite<T>(w[y], on[n], a, b);
          o[n][dt][2 * y] += a;
          o[n][dt][2 * y + 1] += b;
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 32 * D * 2 / 1024; ++i) {
    u32x4_t* at = (u32x4_t*)(sv + i * 1024 + lane * 16);
    u32x4_t w = *at;
    for (int j = 0; j < 4; ++j) w[j] = finite2<T>(w[j]);
    *at = w;
  }
}

template <typename T, int D, int NC>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void attn_few_kernel(const AttnArgs a) {
  constexpr int ROW = D * 2;          // bytes of a cache row
  constexpr int TILE = 32 * ROW;      // bytes of a wave's K (or V) tile
  constexpr int NI = TILE / 1024;     // copies per tile
  constexpr int NS = D / 32;          // k-steps of the scores
  constexpr int ND = D / 16;          // output tiles
  __shared__ __attribute__((aligned(1024))) uint8_t sm[4 * 2 * TILE];
  __shared__ float sml[4][16 * NC][2];
  __shared__ int ssh[8];
  __shared__ int sfound[4];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, col = lane & 15;

  FewRun run;
  // Two units for an item's start and end where the runs are long (64 ragged sequences: 146 -> 138 us), none
  // where they are short (8 sequences, window 1024: 17.4 against 19.1 us).
  if (!few_run<128, 2, 20>(a, ssh, sfound, run)) return;
  const int u1 = run.u1, item_units = run.item_units;
  int s = run.s, base = run.base;

  uint8_t* sk = sm + wave * 2 * TILE;
  uint8_t* sv = sk + TILE;
  TileCopy<D, 16, 2, 128, true> tc;
  tc.init(a, 0, lane);
  bool recorded = false;
  for (int u = run.u0; u < u1;) {
    const AttnSeq q = attn_seq(a, s);
    int lo, hi, first;
    attn_span(a, q, 0, q.nq - 1, lo, hi);
    const bool ours = q.nq >= 1 && attn_is_few(a, q.nq);
    const int nt = attn_tiles<128>(lo, hi, first), per = nt + item_units;
    if (!ours || u >= base + per * a.hk) {  // on to the next sequence
      if (ours) base += per * a.hk;
      ++s;
      continue;
    }
    const int head = (u - base) / per;
    const int item0 = base + head * per + item_units;  // the item's tiles are the units [item0, item0 + nt)
    const int ta = max(0, u - item0), tb = min(nt, u1 - item0);
    u = item0 + nt;
    if (tb <= ta) continue;  // the run ends before the item's first tile
    const int rows = q.nq * a.g;

    // The wave's queries: column c of tile n is row 16 n + c.
    u32x4_t qf[NC][NS];
    int qpos[NC];
    const uint8_t* kb = a.k + (int64_t)head * a.head_stride;
    const uint8_t* vb = a.v + (int64_t)head * a.head_stride;
    const int32_t* table = a.table + (int64_t)s * a.table_stride;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const int r = 16 * n + col;
      const int i = (int)a.g_div.div((uint32_t)r);
      const bool in = r < rows;
      qpos[n] = q.kv - q.nq + (in ? i : q.nq - 1);
      const uint8_t* qp = a.q + ((int64_t)(q.q0 + (in ? i : 0)) * a.q_ts + (int64_t)(head * a.g + (in ? r - i * a.g : 0)) * a.q_hs);
#pragma unroll
      for (int st = 0; st < NS; ++st) {
        const u32x4_t z = {0, 0, 0, 0};
        qf[n][st] = in ? *(const u32x4_t*)(qp + (4 * st + g) * 16) : z;
      }
    }
    const int pos_lo = q.kv - q.nq, pos_hi = q.kv - 1;  // first and last query's position

    f32x4_t o[NC][ND];
    float m[NC], l[NC];
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      m[n] = kNegInf;
      l[n] = 0.f;
#pragma unroll
      for (int d = 0; d < ND; ++d) o[n][d] = f32x4_t{0, 0, 0, 0};
    }

    const int k00 = (first + ta) * 128 + wave * 32;
    tc.lookup(a, table, k00, lo, hi, lane, true);
    tc.resolve(a, lo, hi, lane);
    tc.template copy<false>(tc.now, kb, sk, 0, lane);
    tc.template copy<true>(tc.now, vb, sv, 0, lane);
    uint32_t seen = tc.seen;
    if (ta + 1 < tb) tc.lookup(a, table, k00 + 128, lo, hi, lane, false);

    for (int t = ta; t < tb; ++t) {
      const int k0 = (first + t) * 128 + wave * 32;
      const bool more = t + 1 < tb;
      attn_wait_vm<NI>();  // K of this tile
      f32x4_t sc[NC][2];
#pragma unroll
      for (int kt = 0; kt < 2; ++kt) {
        const int row = 16 * kt + col;
        u32x4_t kf[NS];
#pragma unroll
        for (int st = 0; st < NS; ++st)
          kf[st] = *(const u32x4_t*)(sk + row * ROW + ((4 * st + g) ^ swz_k<D>(row)) * 16);
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          sc[n][kt] = f32x4_t{0, 0, 0, 0};
#pragma unroll
          for (int st = 0; st < NS; ++st) sc[n][kt] = mfma16(T{}, kf[st], qf[n][st], sc[n][kt]);
        }
      }
      const uint32_t seen_now = seen;
      if (more) {
        tc.resolve(a, lo, hi, lane);
        seen = tc.seen;
        attn_wait_lds();
        tc.template copy<false>(tc.now, kb, sk, 0, lane);
      }
      // masks: rows that are not loaded, keys past a column's query, keys before its window
      const bool cut = k0 + 31 > pos_lo || (a.window > 0 && k0 <= pos_hi - a.window);
      if (cut || seen_now != 0xffffffffu) {
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          const int last = qpos[n] - k0, before = a.window > 0 ? last - a.window : -1;
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            const int j = 16 * (r >> 2) + 4 * g + (r & 3);
            const bool see = ((int)((seen_now >> j) & 1) & (int)(j <= last) & (int)(j > before)) != 0;
            sc[n][r >> 2][r & 3] = see ? sc[n][r >> 2][r & 3] : kNegInf;
          }
        }
      }
      u32x4_t p[NC];
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        float mx = fmaxf(sc[n][0][0], sc[n][1][0]);
#pragma unroll
        for (int r = 1; r < 4; ++r) mx = max3(mx, sc[n][0][r], sc[n][1][r]);
        mx = join32(join16(mx, MaxF()), MaxF()) * a.sl;
        if (__any(mx > m[n] + kLazy)) {
          const float mn = fmaxf(m[n], mx);
          const float f = m[n] == kNegInf ? 0.f : exp2_fast(m[n] - mn);
          m[n] = mn;
          l[n] *= f;
#pragma unroll
          for (int d = 0; d < ND; ++d)
            for (int r = 0; r < 4; ++r) o[n][d][r] *= f;
        }
        const float mr = m[n] == kNegInf ? 0.f : m[n];
        float e[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) e[r] = exp2_fast(__builtin_fmaf(sc[n][r >> 2][r & 3], a.sl, -mr));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          p[n][r] = pack2(T{}, e[2 * r], e[2 * r + 1]);
          l[n] = add2(T{}, p[n][r], l[n]);
        }
      }
      if (more)
        attn_wait_vm<NI>();  // V of this tile; the next K may be in flight
      else
        attn_wait_vm<0>();
      // a key that only some columns see may hold an infinity or a NaN
      if (cut && q.nq > 1 && few_v_nonfinite<T, D>(sv, lane)) few_nonfinite<T, D, NC>(sv, lane, p, o);
#pragma unroll
      for (int n = 0; n < NC; ++n) few_pv<T, D>(sv, lane, p[n], o[n]);
      if (more) {
        attn_wait_lds();
        tc.template copy<true>(tc.now, vb, sv, 0, lane);
        if (t + 2 < tb) tc.lookup(a, table, k0 + 256, lo, hi, lane, false);
      }
    }

    const bool whole = ta == 0 && tb == nt;
    few_finish<D, NC>(a, tid, sm, 2 * TILE, sml, o, m, l, run.w, q, head, rows, ta == 0, whole,
                      [](void* p, float x, float y, float z, float w) { store4(T{}, p, x, y, z, w); });
    if (ta == 0) few_record(a, run, s, head, q.q0, rows, item0 + nt, whole, recorded);
  }
  if (!recorded && !a.few_by_item && tid == 0) run.rec->pieces = 0;
}

}  // namespace

template <typename T, int D, int NC> static hipError_t few(const AttnArgs& a, hipStream_t s) {
  attn_few_kernel<T, D, NC><<<a.nw_few, 256, 0, s>>>(a);
  return hipGetLastError();
}
template <typename T> static hipError_t few_d(const AttnArgs& a, int d, int nc, hipStream_t s) {
  if (d == 64) return nc == 1 ? few<T, 64, 1>(a, s) : few<T, 64, 2>(a, s);
  if (d == 128) return nc == 1 ? few<T, 128, 1>(a, s) : few<T, 128, 2>(a, s);
  return few<T, 256, 1>(a, s);
}
hipError_t launch_attn_few(const AttnArgs& args, int dt, int d, int nc, hipStream_t s) {
  AttnArgs a = args;
  attn_record_kind(a);
  return dt == DT_BF16 ? few_d<BF16>(a, d, nc, s) : few_d<F16>(a, d, nc, s);
}

}  // namespace ql
