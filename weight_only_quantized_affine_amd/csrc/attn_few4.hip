// Paged attention over a cache in 4 bits, few rows: as attn_few.hip (whose division of the work and end of
// an item it shares), with 64 positions a wave and 256 a workgroup's tile.
//
// The codes are decoded in registers, between LDS and the matrix cores.  K: a lane of the 16x16x32 product
// holds one key and, of its row, words of eight codes under one scale, so a word becomes an operand by
// 13 instructions (one shift, four masks under exponent bits, four exact differences, four fused products
// with scale and bias).  V: the 4-bit transposing LDS read hands a lane the codes of 16 keys for one
// of the d values, in any order of the keys that the reading lanes' addresses give: the order in which the
// lane holds the scores of those keys, so that the weights are the other operand as they are.  The
// scales and biases of a lane's 16 keys are put into pairs once per group of values.
#include "attn_common4.hpp"
#include "attn_few.hpp"

namespace ql {
namespace {

typedef __attribute__((ext_vector_type(2))) int i32x2_t;
typedef __attribute__((address_space(3))) i32x2_t at_lds_i32x2;
__device__ __forceinline__ u32x2_t read_tr4(const uint8_t* p) {
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr4_b64_v2i32((at_lds_i32x2*)p));
}

// Position of 16-byte chunk c of row r (of D / 32 chunks).  K is read 16 rows at one chunk (D = 256: rows are
// half the LDS's 256 bytes of banks); V by 16 lanes at one chunk of the rows i + 16 k, i and k = 0 .. 3.
template <int D> __device__ __forceinline__ int swz4_k(int r) { return D == 256 ? (r & 7) : 0; }
template <int D> __device__ __forceinline__ int swz4_v(int r) {
  if (D == 256) return ((r >> 1) & 1) | (((r >> 4) & 3) << 1);
  return D == 128 ? ((r >> 4) & 3) : ((r >> 4) & 1);
}

// The 64 cache rows of a wave's tile (positions base .. base + 63, a multiple of 64), K and V alike, and
// the words of their groups; tiles are STEP positions apart.  Lane l looks up row l.
template <int D, int GROUP, int STEP> struct Copy4 {
  static constexpr int CH = D / 32;          // 16-byte chunks of a row
  static constexpr int RPI = 64 / CH;        // rows of an instruction (1 KB)
  static constexpr int NI = 64 / RPI;        // instructions of a tile
  static constexpr int GP = D / GROUP;       // groups of a row
  static constexpr int COPIES = NI + GP;     // all instructions of K, and of V
  static constexpr int BLOCK = 16;           // tiles whose page ids are read at once
  int ids, block;   // a.page16: pages of the runs of BLOCK tiles (lane t + 16 u: tile t, run u), position of the first
  int id, base;     // else: page of the lane's row
  bool whole;       // uniform: every row is to be seen and pages hold runs of 16
  int64_t at[4];    // uniform, where whole: the runs' places
  int64_t row;      // the lane's row among the codes, -1 for a row that is not to be seen
  int64_t prow;     // and among the words
  uint64_t seen;    // bit r: row r is to be seen

  __device__ __forceinline__ void lookup(const AttnArgs4& a, const int32_t* table, int first, int lo, int hi, int lane,
                                         bool begins) {
    base = first;
    if (a.page16) {
      if (begins || first - block >= BLOCK * STEP) {
        block = first;
        const int p = first + (lane & 15) * STEP + (lane >> 4) * 16;
        ids = -1;
        if (p + 16 > lo && p < hi) ids = table[a.page_div.div((uint32_t)p)];
        asm volatile("" : "+v"(ids));  // the wait for the load is here
      }
    } else {
      const int p = first + lane;
      id = -1;
      if (p >= lo && p < hi) id = table[a.page_div.div((uint32_t)p)];
    }
  }
  __device__ __forceinline__ void resolve(const AttnArgs4& a, int lo, int hi, int lane) {
    const int p = base + lane;
    const int tile = a.page16 ? (base - block) / STEP : 0;
    if (a.page16) id = __shfl(ids, (lane & 48) + tile);
    const int in = p - (int)a.page_div.div((uint32_t)p) * a.page_size;
    const bool see = p >= lo && p < hi && (uint32_t)id < (uint32_t)a.n_pages;
    seen = __ballot(see);
    prow = see ? (int64_t)id * a.p_page_stride + (int64_t)in * a.p_token_stride : -1;
    whole = a.page16 && seen == ~0ull;
    if (whole) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int pu = base + 16 * u, iu = __builtin_amdgcn_readlane(ids, tile + 16 * u);
        at[u] = (int64_t)iu * a.page_stride + (int64_t)(pu - (int)a.page_div.div((uint32_t)pu) * a.page_size) * a.token_stride;
      }
    } else {
      row = see ? (int64_t)id * a.page_stride + (int64_t)in * a.token_stride : -1;
    }
  }
  // Starts the copies of the codes to dst (rows back to back) and of the words to wdst (64 of each group).
  template <bool IS_V>
  __device__ __forceinline__ void copy(const AttnArgs4& a, const uint8_t* head, const uint8_t* words, uint8_t* dst,
                                       uint8_t* wdst, int lane) const {
    const int c = lane % CH, r0 = lane / CH;
    if (whole) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int r = i * RPI + r0;  // its run: i * RPI / 16, where an instruction lies in one
        const int cc = c ^ (IS_V ? swz4_v<D>(r) : swz4_k<D>(r));
        if constexpr (RPI <= 16) {
          const uint32_t off = (uint32_t)(r & 15) * (uint32_t)a.token_stride + cc * 16;
          copy16_from<true, false>(uniform64((int64_t)(uintptr_t)head + at[i * RPI / 16]), off, 0, dst + i * 1024);
        } else {
          const int64_t b = (lane < 32 ? at[2 * i] : at[2 * i + 1]) + (int64_t)((r & 15) * (int)a.token_stride + cc * 16);
          copy16<true>(head + b, dst + i * 1024);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int r = i * RPI + r0;
        const int cc = c ^ (IS_V ? swz4_v<D>(r) : swz4_k<D>(r));
        const int lo = __shfl((int)row, r), hi = __shfl((int)(row >> 32), r);
        const int64_t o = ((int64_t)hi << 32) | (uint32_t)lo;
        copy16<true>((hi < 0 ? (const uint8_t*)kZeroRow : head + o) + cc * 16, dst + i * 1024);
      }
    }
    const uint8_t* pw = prow < 0 ? (const uint8_t*)kZeroRow : words + prow;
#pragma unroll
    for (int i = 0; i < GP; ++i) copy4(pw + 4 * i, wdst + i * 256);
  }
};

// Adds the values of the keys in `odd` (whose groups fp16 may not hold) to the columns whose weight is
// not zero, and clears their words, so that the products take zeros there.
template <int D, int GROUP, int NC>
__device__ __forceinline__ void few4_odd(const uint8_t* sv, uint8_t* swv, uint64_t odd, int lane,
                                         const u32x4_t (*p)[2], f32x4_t (*o)[D / 16]) {
  asm volatile("" : "+v"(lane));  // the addresses stay in this rare path
  const int g = lane >> 4, col = lane & 15;
#pragma unroll 1
  while (odd) {
    const int j = __builtin_ctzll(odd);
    odd &= odd - 1;
    // the weight of key j = 16 k + 4 q + i: lanes of q, half k & 1 of word i of product k >> 1
    float w[NC];
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      uint32_t x = 0;
#pragma unroll
      for (int y = 0; y < 8; ++y) x = y == 4 * (j >> 5) + (j & 3) ? p[n][y >> 2][y & 3] : x;
      x = __shfl(x, 16 * ((j >> 2) & 3) + col);
      w[n] = param_to_f32<F16>((j >> 4) & 1 ? x >> 16 : x & 0xffffu);
    }
#pragma unroll 1
    for (int dt = 0; dt < D / 16; ++dt) {
      const f16x2_t gr = h2(*(const uint32_t*)(swv + (16 * dt / GROUP) * 256 + 4 * j));
      const uint32_t c = *(const uint16_t*)(sv + j * (D / 2) + (((dt >> 1) ^ swz4_v<D>(j)) * 16) + 8 * (dt & 1) + 2 * g);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const _Float16 v = __builtin_fmaf16((_Float16)(float)((c >> (4 * r)) & 15), gr[0], gr[1]);
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          const float add = w[n] != 0.f ? w[n] * (float)v : 0.f;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) o[n][d][r] += d == dt ? add : 0.f;
        }
      }
    }
    if (lane < D / GROUP) *(uint32_t*)(swv + lane * 256 + 4 * j) = 0;
  }
}

template <int D, int GROUP, int NC>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void attn_few4_kernel(const AttnArgs4 a) {
  using Copy = Copy4<D, GROUP, 256>;
  constexpr int ROW = D / 2;            // bytes of a row's codes
  constexpr int TILE = 64 * ROW;        // of a wave's tile
  constexpr int GP = Copy::GP, WORDS = GP * 256;
  constexpr int WAVE = 2 * (TILE + WORDS);
  constexpr int NS = D / 32;            // k-steps of the scores
  constexpr int ND = D / 16;            // output tiles
  constexpr int NP = D == 256 ? 2 : 1;  // groups that a lane's part of a key's row may lie in
  static_assert(WAVE >= 16 * D * 4, "the joining of the waves takes the tiles' place");
  __shared__ __attribute__((aligned(1024))) uint8_t sm[4 * WAVE];
  __shared__ float sml[4][16 * NC][2];
  __shared__ int ssh[8];
  __shared__ int sfound[4];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, col = lane & 15;

  FewRun run;
  if (!few_run<256>(a, ssh, sfound, run)) return;
  const int u1 = run.u1, item_units = run.item_units;
  int s = run.s, base = run.base;

  uint8_t* sk = sm + wave * WAVE;
  uint8_t* sv = sk + TILE;
  uint8_t* swk = sv + TILE;
  uint8_t* swv = swk + WORDS;
  Copy tc;
  bool recorded = false;
  for (int u = run.u0; u < u1;) {
    const AttnSeq q = attn_seq(a, s);
    int lo, hi, first;
    attn_span(a, q, 0, q.nq - 1, lo, hi);
    const bool ours = q.nq >= 1 && attn_is_few(a, q.nq);
    const int nt = attn_tiles<256>(lo, hi, first), per = nt + item_units;
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

    const uint8_t* kb = a.k + (int64_t)head * a.head_stride;
    const uint8_t* vb = a.v + (int64_t)head * a.head_stride;
    const uint8_t* kw = a.kp + (int64_t)head * a.p_head_stride;
    const uint8_t* vw = a.vp + (int64_t)head * a.p_head_stride;
    const int32_t* table = a.table + (int64_t)s * a.table_stride;
    const int k00 = (first + ta) * 256 + wave * 64;
    tc.lookup(a, table, k00, lo, hi, lane, true);
    tc.resolve(a, lo, hi, lane);
    tc.template copy<false>(a, kb, kw, sk, swk, lane);
    tc.template copy<true>(a, vb, vw, sv, swv, lane);
    uint64_t seen = tc.seen;

    // The wave's queries: column c of tile n is row 16 n + c; a lane holds the values that meet its part
    // of the keys' rows, word by word.
    u32x4_t qf[NC][NS];
    int qpos[NC];
    float sl[NC];  // scale * log2(e) * 2^t
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const int r = 16 * n + col;
      const int i = (int)a.g_div.div((uint32_t)r);
      const bool in = r < rows;
      qpos[n] = q.kv - q.nq + (in ? i : q.nq - 1);
      const uint8_t* qp = a.q + ((int64_t)(q.q0 + (in ? i : 0)) * a.q_ts + (int64_t)(head * a.g + (in ? r - i * a.g : 0)) * a.q_hs);
      float amax = 0.f;
#pragma unroll
      for (int st = 0; st < NS; ++st) {
        const u32x4_t z = {0, 0, 0, 0};
        const int word = D == 64 ? 2 * g + st : 16 * (st / 4) + 4 * g + st % 4;
        qf[n][st] = in ? *(const u32x4_t*)(qp + word * 16) : z;
        amax = amax8(qf[n][st], amax);
      }
      const int t = a.io == DT_BF16 ? q_exponent(join32(join16(amax, MaxF()), MaxF())) : 0;
      const float factor = __builtin_ldexpf(1.f, -t);
      sl[n] = __builtin_ldexpf(a.sl, t);
#pragma unroll
      for (int st = 0; st < NS; ++st) qf[n][st] = q_pairs(qf[n][st], a.io, factor);
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
    if (ta + 1 < tb) tc.lookup(a, table, k00 + 256, lo, hi, lane, false);

    for (int t = ta; t < tb; ++t) {
      const int k0 = (first + t) * 256 + wave * 64;
      const bool more = t + 1 < tb;
      attn_wait_vm<Copy::COPIES>();  // K of this tile
      uint32_t kf[4][NS];
      uint32_t kg[4][NP];
#pragma unroll
      for (int kt = 0; kt < 4; ++kt) {
        const int row = 16 * kt + col;
        if constexpr (D == 64) {
          const u32x2_t w = *(const u32x2_t*)(sk + row * ROW + g * 8);
          kf[kt][0] = w[0], kf[kt][1] = w[1];
          kg[kt][0] = *(const uint32_t*)(swk + (16 * g / GROUP) * 256 + row * 4);
        } else {
#pragma unroll
          for (int c = 0; c < NP; ++c) {
            const u32x4_t w = *(const u32x4_t*)(sk + row * ROW + ((4 * c + g) ^ swz4_k<D>(row)) * 16);
            for (int x = 0; x < 4; ++x) kf[kt][4 * c + x] = w[x];
            kg[kt][c] = *(const uint32_t*)(swk + ((128 * c + 32 * g) / GROUP) * 256 + row * 4);
          }
        }
      }
      const uint64_t seen_now = seen;
      if (more) {
        tc.resolve(a, lo, hi, lane);
        seen = tc.seen;
        attn_wait_lds();
        tc.template copy<false>(a, kb, kw, sk, swk, lane);
      }
      f32x4_t sc[NC][4];
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) sc[n][kt] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int kt = 0; kt < 4; ++kt)
#pragma unroll
        for (int st = 0; st < NS; ++st) {
          const u32x4_t kv = values4(kf[kt][st], kg[kt][st / 4]);
#pragma unroll
          for (int n = 0; n < NC; ++n) sc[n][kt] = mfma16(F16{}, kv, qf[n][st], sc[n][kt]);
        }
      // masks: rows that are not loaded, keys past a column's query, keys before its window
      const bool cut = k0 + 63 > pos_lo || (a.window > 0 && k0 <= pos_hi - a.window);
      if (cut || seen_now != ~0ull) {
        const uint32_t s0 = (uint32_t)seen_now >> (4 * g), s1 = (uint32_t)(seen_now >> 32) >> (4 * g);
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          const int last = qpos[n] - k0 - 4 * g, before = a.window > 0 ? last - a.window : -65;
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const int j = 16 * (r >> 2) + (r & 3);
            const bool see = ((int)(((r < 8 ? s0 : s1) >> (j & 31)) & 1) & (int)(j <= last) & (int)(j > before)) != 0;
            sc[n][r >> 2][r & 3] = see ? sc[n][r >> 2][r & 3] : kNegInf;
          }
        }
      }
      u32x4_t p[NC][2];
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        float mx = fmaxf(fmaxf(sc[n][0][0], sc[n][1][0]), fmaxf(sc[n][2][0], sc[n][3][0]));
#pragma unroll
        for (int r = 1; r < 4; ++r) mx = max3(max3(mx, sc[n][0][r], sc[n][1][r]), sc[n][2][r], sc[n][3][r]);
        mx = join32(join16(mx, MaxF()), MaxF()) * sl[n];
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
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            p[n][h][r] = pack2(F16{}, exp2_fast(__builtin_fmaf(sc[n][2 * h][r], sl[n], -mr)),
                               exp2_fast(__builtin_fmaf(sc[n][2 * h + 1][r], sl[n], -mr)));
            l[n] = add2(F16{}, p[n][h][r], l[n]);
          }
      }
      if (more)
        attn_wait_vm<Copy::COPIES>();  // V of this tile; the next K may be in flight
      else
        attn_wait_vm<0>();
      // a key that only some columns see may stand for an infinity or a NaN
      if (cut && q.nq > 1) {
        bool mine = false;
#pragma unroll
        for (int i = 0; i < GP; ++i) mine |= odd_group(*(const uint32_t*)(swv + i * 256 + lane * 4));
        const uint64_t odd = __ballot(mine);
        if (odd) few4_odd<D, GROUP, NC>(sv, swv, odd, lane, p, o);
      }
      const int vrow = 16 * (col >> 2) + 4 * g + (col & 3);
#pragma unroll
      for (int gr = 0; gr < GP; ++gr) {
        // scales and biases of the lane's keys 16 k + 4 g + i, as pairs k = (0, 1) and (2, 3)
        f16x2_t vs[2][4], vbias[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const u32x4_t x = *(const u32x4_t*)(swv + gr * 256 + (32 * h + 4 * g) * 4);
          const u32x4_t y = *(const u32x4_t*)(swv + gr * 256 + (32 * h + 16 + 4 * g) * 4);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            vs[h][i] = h2(perm(y[i], x[i], 0x05040100u));
            vbias[h][i] = h2(perm(y[i], x[i], 0x07060302u));
          }
        }
#pragma unroll
        for (int dd = 0; dd < GROUP / 16; ++dd) {
          const int d = gr * (GROUP / 16) + dd;
          const u32x2_t w = read_tr4(sv + vrow * ROW + (((d >> 1) ^ swz4_v<D>(vrow)) * 16) + 8 * (d & 1));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const u32x4_t v = values4(w[h], vs[h], vbias[h]);
#pragma unroll
            for (int n = 0; n < NC; ++n) o[n][d] = mfma16(F16{}, v, p[n][h], o[n][d]);
          }
        }
      }
      if (more) {
        attn_wait_lds();
        tc.template copy<true>(a, vb, vw, sv, swv, lane);
        if (t + 2 < tb) tc.lookup(a, table, k0 + 512, lo, hi, lane, false);
      }
    }

    const bool whole = ta == 0 && tb == nt;
    few_finish<D, NC>(a, sm, WAVE, sml, o, m, l, run.w, q, head, rows, ta == 0, whole,
                      [io = a.io](void* p, float x, float y, float z, float w) {
                        if (io == DT_BF16)
                          store4(BF16{}, p, x, y, z, w);
                        else
                          store4(F16{}, p, x, y, z, w);
                      });
    if (ta == 0) few_record(a, run, s, head, q.q0, rows, item0 + nt, whole, recorded);
  }
  if (!recorded && !a.few_by_item && tid == 0) run.rec->pieces = 0;
}

template <int D, int GROUP, int NC> hipError_t few4(const AttnArgs4& a, hipStream_t s) {
  attn_few4_kernel<D, GROUP, NC><<<a.nw_few, 256, 0, s>>>(a);
  return hipGetLastError();
}
template <int D, int GROUP> hipError_t few4_n(const AttnArgs4& a, int nc, hipStream_t s) {
  if constexpr (D < 256) {
    if (nc == 2) return few4<D, GROUP, 2>(a, s);
  }
  return few4<D, GROUP, 1>(a, s);
}
template <int D> hipError_t few4_g(const AttnArgs4& a, int nc, hipStream_t s) {
  if constexpr (D > 64) {
    if (a.group_log2 == 7) return few4_n<D, 128>(a, nc, s);
  }
  return a.group_log2 == 6 ? few4_n<D, 64>(a, nc, s) : few4_n<D, 32>(a, nc, s);
}

}  // namespace

hipError_t launch_attn_few4(const AttnArgs4& args, int d, int nc, hipStream_t s) {
  AttnArgs4 a = args;
  attn_record_kind(a);
  return d == 64 ? few4_g<64>(a, nc, s) : d == 128 ? few4_g<128>(a, nc, s) : few4_g<256>(a, nc, s);
}

}  // namespace ql
