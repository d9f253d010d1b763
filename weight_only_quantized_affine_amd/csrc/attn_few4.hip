// Paged attention over a cache in 4 bits, few rows: as attn_few.hip (whose division of the work and end of
// an item it shares), with 64 positions a wave and 256 a workgroup's tile.
//
// No value is decoded.  A code masked into the low bits of a half is the fp16 subnormal c 2^-24, or 16 c 2^-24
// four bits further up, so a word of eight codes becomes an operand of the 16x16x32 product by one shift and
// four masks, and scales and biases enter as they are:
//   scores   q.k = sum over groups of s (q.c) + b sum(q), one accumulator a group, sum(q) as two fp16 numbers;
//   output   sum_j w_j v_j = sum_j (w_j s_j) (c_j - 8) + sum_j w_j (b_j + 8 s_j), the products w s and the weights
//            of the second sum rounded to fp16 (as large as a rounding of w in w v, since a group's middle is
//            taken out), the sum of the w s taken out 8 times.
// A product of the matrix cores aligns its terms by their operands' exponents, a subnormal one's taken as 2^-14, and
// drops what lies below 2^-24 of the largest: over codes that is 2^-14 of the largest w s (or |q| s) among its 32,
// not of the sum.  Over many keys it is little next to the weights' rounding (fp16 outputs of 16000 tokens are off by
// 0.0003 where one rounding of the exact ones is 0.0002).
// The factors 16 are taken out of q and of the weights.  So that w s stays within fp16 and keeps its small
// values, a group's products are held times 2^(7 - E), E the exponent of its largest scale that the row has met:
// they are below 2^15, and keys that a row does not see change no bit of it.
// V: the 4-bit transposing LDS read hands a lane the codes of 16 keys for one of the d values, in any order
// of the keys that the reading lanes' addresses give: the order in which the lane holds the scores.
// (Decoding every code to fp16 by 13 instructions a word: 131071 tokens 54 us, 64 ragged sequences 105.)
//
// Bound by the vector units next to memory: a tile of 64 positions takes some 540 vector instructions a wave, the
// ragged batch 730 with its items' starts and ends.  Two workgroups a compute unit share its registers (three,
// with fewer each: 131071 tokens 53 us against 46).  V of two tiles lies in LDS and K of one, whose codes are in
// registers before the next K is copied; sums of weight times bias and of the codes' middles are extra rows of
// the products where registers allow (kSumInRow; both steps together: 64 ragged sequences 71 -> 61 us).
//
// Measured (bf16, 32 heads on 8 of 128, groups of 64): 64 ragged sequences of 100 to 16000 tokens, pages of 16,
// 59 to 63 us, 3.4 TB/s with the joining; one of 131071 tokens, pages of 64, 47 us; 64 sequences of 5 drafted
// tokens 107.  64 values a head 79, 256 values 87, groups of 32 89, of 128 59; token-major pages 103, pages of 24
// 73.  (The 16-bit cache: 139 and 97 us.)
#include "attn_common4.hpp"
#include "attn_few.hpp"

namespace ql {
namespace {

typedef __attribute__((ext_vector_type(2))) int i32x2_t;
typedef __attribute__((address_space(3))) i32x2_t at_lds_i32x2;
__device__ __forceinline__ u32x2_t read_tr4(const uint8_t* p) {
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr4_b64_v2i32((at_lds_i32x2*)p));
}

// Position of 16-byte chunk c of row r (of D / 32 chunks): the reads of K take 16 rows at one place, those of V
// the rows i + 16 k, i and k = 0 .. 3; either set's positions are distinct modulo the LDS's 256 bytes of banks.
template <int D> __device__ __forceinline__ int swz4_k(int r) {
  return D == 256 ? ((r >> 1) & 7) : D == 128 ? ((r >> 2) & 3) : ((r >> 3) & 1);
}
template <int D> __device__ __forceinline__ int swz4_v(int r) {
  if (D == 256) return ((r >> 1) & 1) | (((r >> 4) & 3) << 1);
  return D == 128 ? ((r >> 4) & 3) : ((r >> 4) & 1);
}

// The 64 cache rows of a wave's tile (positions base .. base + 63), K and V alike, and the words of their
// groups; tiles are STEP positions apart.
//
// Where pages are multiples of 16 slots (a.page16) the places of the 4 runs of the next 16 tiles are worked
// out at once, a run a lane, and a tile whose rows are all to be seen is copied from scalar bases and lane
// offsets that never change.  Else row l is looked up by lane l and handed to the lanes that copy it.
template <int D, int GROUP, int STEP> struct Copy4 {
  static constexpr int CH = D / 32;          // 16-byte chunks of a row
  static constexpr int RPI = 64 / CH;        // rows of an instruction (1 KB)
  static constexpr int NI = 64 / RPI;        // instructions of a tile
  static constexpr int GP = D / GROUP;       // groups of a row
  static constexpr int WI = GP > 4 ? 8 : 4;  // instructions of a tile's words: 16 rows of up to 4 groups each
  static constexpr int COPIES = NI + WI;     // all instructions of K, and of V
  int64_t run, wrun;  // a.page16: a run's place among the codes and the words (lane t + 16 u: tile t, run u)
  uint64_t known;     // bit of each such lane: its page is in the cache
  int block;          // position of the first of the 16 tiles
  int id, base;       // else: page of the lane's row; first position
  bool whole;         // uniform: every row is to be seen and pages hold runs of 16
  int tile;           // uniform, where whole: the tile among the 16
  int64_t row, wrow;  // else: the lane's row, -1 for a row that is not to be seen
  uint64_t seen;      // bit r: row r is to be seen

  __device__ __forceinline__ int64_t place(const AttnArgs4& a, int id, int p) const {
    return (int64_t)id * a.page_stride + (int64_t)(p - (int)a.page_div.div((uint32_t)p) * a.page_size) * a.token_stride;
  }
  __device__ __forceinline__ int64_t word_place(const AttnArgs4& a, int id, int p) const {
    return (int64_t)id * a.p_page_stride + (int64_t)(p - (int)a.page_div.div((uint32_t)p) * a.page_size) * a.p_token_stride;
  }
  __device__ __forceinline__ void lookup(const AttnArgs4& a, const int32_t* table, int first, int lo, int hi, int lane,
                                         bool begins) {
    base = first;
    if (a.page16) {
      if (begins || first - block >= 16 * STEP) {
        block = first;
        const int p = first + (lane & 15) * STEP + (lane >> 4) * 16;
        int i = -1;
        if (p + 16 > lo && p < hi) i = table[a.page_div.div((uint32_t)p)];
        known = __ballot((uint32_t)i < (uint32_t)a.n_pages);  // the wait for the load is here
        run = place(a, i, p);
        wrun = word_place(a, i, p);
      }
    } else {
      const int p = first + lane;
      id = -1;
      if (p >= lo && p < hi) id = table[a.page_div.div((uint32_t)p)];
    }
  }
  __device__ __forceinline__ int64_t lane64(int64_t x, int l) const {
    const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)x, l), hi = __builtin_amdgcn_readlane((int)(uint32_t)(x >> 32), l);
    return (int64_t)((uint64_t)hi << 32 | lo);
  }
  __device__ __forceinline__ void resolve(const AttnArgs4& a, int lo, int hi, int lane) {
    whole = false;
    if (a.page16) {
      constexpr uint64_t kRuns = 0x0001000100010001ull;
      tile = (base - block) / STEP;
      whole = ((known >> tile) & kRuns) == kRuns && base >= lo && base + 64 <= hi;
      seen = ~0ull;
    }
    if (!whole) {
      const int p = base + lane;
      bool see = p >= lo && p < hi;
      if (a.page16) {
        const int from = (lane & 48) + tile;
        row = (int64_t)((uint64_t)(uint32_t)__shfl((int)(run >> 32), from) << 32 | (uint32_t)__shfl((int)(uint32_t)run, from));
        wrow = (int64_t)((uint64_t)(uint32_t)__shfl((int)(wrun >> 32), from) << 32 | (uint32_t)__shfl((int)(uint32_t)wrun, from));
        see = see && ((known >> from) & 1);
        row += (int64_t)(lane & 15) * a.token_stride;
        wrow += (int64_t)(lane & 15) * a.p_token_stride;
      } else {
        see = see && (uint32_t)id < (uint32_t)a.n_pages;
        row = place(a, id, p);
        wrow = word_place(a, id, p);
      }
      seen = __ballot(see);
      if (!see) row = wrow = -1;
    }
  }
  // Starts the copies of the codes to dst (rows back to back) and of the words to wdst ([run][group][16 rows]).
  template <bool IS_V>
  __device__ __forceinline__ void copy(const AttnArgs4& a, const uint8_t* head, const uint8_t* words, uint8_t* dst,
                                       uint8_t* wdst, int lane) const {
    asm volatile("" : "+v"(lane));  // the lane's places are worked out here, not kept in registers
    const int c = lane % CH, r0 = lane / CH;
    auto chunk = [&](int r) { return (c ^ (IS_V ? swz4_v<D>(r) : swz4_k<D>(r))) * 16; };
    if (whole) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int r = i * RPI + r0;
        if constexpr (RPI <= 16) {
          const uint32_t off = (uint32_t)(r & 15) * (uint32_t)a.token_stride + chunk(r);
          copy16_from<true, false>((int64_t)(uintptr_t)head + lane64(run, tile + i * RPI / 16 * 16), off, 0, dst + i * 1024);
        } else {
          const int64_t b0 = lane64(run, tile + 32 * i), b1 = lane64(run, tile + 32 * i + 16);
          copy16<true>(head + (lane < 32 ? b0 : b1) + ((r & 15) * (int)a.token_stride + chunk(r)), dst + i * 1024);
        }
      }
      const uint32_t woff = (uint32_t)(lane & 15) * (uint32_t)a.p_token_stride + (lane >> 4) * 4;
      int64_t b[4];  // read from other lanes while all lanes are active
#pragma unroll
      for (int u = 0; u < 4; ++u) b[u] = (int64_t)(uintptr_t)words + lane64(wrun, tile + 16 * u);
      if (GP >= 4 || lane < 16 * GP) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          copy4_from(b[u], woff, wdst + u * GP * 64);
          if (GP > 4) copy4_from(b[u], woff + 16, wdst + u * GP * 64 + 256);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        const int r = i * RPI + r0;
        const int lo = __shfl((int)row, r), hi = __shfl((int)(row >> 32), r);
        const int64_t o = ((int64_t)hi << 32) | (uint32_t)lo;
        copy16<true>((hi < 0 ? (const uint8_t*)kZeroRow : head + o) + chunk(r), dst + i * 1024);
      }
      const uint8_t* p[4];  // read from other lanes while all lanes are active
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int r = 16 * u + (lane & 15);
        const int lo = __shfl((int)wrow, r), hi = __shfl((int)(wrow >> 32), r);
        const int64_t o = ((int64_t)hi << 32) | (uint32_t)lo;
        p[u] = (hi < 0 ? (const uint8_t*)kZeroRow : words + o) + (lane >> 4) * 4;
      }
      if (GP >= 4 || lane < 16 * GP) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          copy4(p[u], wdst + u * GP * 64);
          if (GP > 4) copy4(p[u] + 16, wdst + u * GP * 64 + 256);
        }
      }
    }
  }
};

// The codes of a word as fp16 subnormals, pairs (i, i + 4): c 2^-24 for even i, 16 c 2^-24 for odd i.
__device__ __forceinline__ u32x4_t codes_as_fp16(uint32_t w) {
  const uint32_t v = w >> 8;
  return u32x4_t{w & 0x000f000fu, w & 0x00f000f0u, v & 0x000f000fu, v & 0x00f000f0u};
}

// Whether a group's scale or bias is infinite or NaN.
__device__ __forceinline__ bool odd_word(uint32_t w) { return (w & 0x7c00u) == 0x7c00u || (w & 0x7c000000u) == 0x7c000000u; }

// Adds the values of the groups that hold an infinity or a NaN, of the keys in `odd`, to the columns whose
// weight is not zero, and clears their words, so that the products take zeros there.  w: the weights as they are
// held, e[n][kt][i] of key 16 kt + 4 g + i.
template <int D, int GROUP, int NC>
__device__ __forceinline__ void few4_odd(const uint8_t* sv, uint8_t* swv, uint64_t odd, int lane, const float (*e)[4][4],
                                         const int (*up)[D / GROUP], f32x4_t (*o)[D / 16]) {
  asm volatile("" : "+v"(lane));  // the addresses stay in this rare path
  constexpr int GP = D / GROUP;
  const int g = lane >> 4, col = lane & 15;
#pragma unroll 1
  while (odd) {
    const int j = __builtin_ctzll(odd);
    odd &= odd - 1;
    float w[NC];
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      float x = 0.f;
#pragma unroll
      for (int y = 0; y < 16; ++y) x = y == 4 * (j >> 4) + (j & 3) ? e[n][y >> 2][y & 3] : x;
      w[n] = __shfl(x, 16 * ((j >> 2) & 3) + col);
    }
    uint8_t* words = swv + (j >> 4) * GP * 64 + (j & 15) * 4;
#pragma unroll 1
    for (int dt = 0; dt < D / 16; ++dt) {
      const uint32_t word = *(const uint32_t*)(words + (16 * dt / GROUP) * 64);
      if (!odd_word(word)) continue;
      const f16x2_t gr = h2(word);
      const uint32_t c = *(const uint16_t*)(sv + j * (D / 2) + (((dt >> 1) ^ swz4_v<D>(j)) * 16) + 8 * (dt & 1) + 2 * g);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float v = __builtin_fmaf((float)((c >> (4 * r)) & 15), (float)gr[0], (float)gr[1]);
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          int u = up[n][0];
#pragma unroll
          for (int x = 1; x < D / GROUP; ++x) u = 16 * dt / GROUP == x ? up[n][x] : u;
          const float add = w[n] != 0.f ? __builtin_ldexpf(w[n] * v, 7 - u - 24) : 0.f;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) o[n][d][r] += d == dt ? add : 0.f;
        }
      }
    }
    if (lane < GP && odd_word(*(uint32_t*)(words + lane * 64))) *(uint32_t*)(words + lane * 64) = 0;
  }
}

template <int D, int GROUP, int NC>
__global__ __launch_bounds__(256, D == 256 ? 1 : 2) void attn_few4_kernel(const AttnArgs4 a) {
  using Copy = Copy4<D, GROUP, 256>;
  constexpr int ROW = D / 2;            // bytes of a row's codes
  constexpr int TILE = 64 * ROW;        // of a wave's tile
  constexpr int GP = Copy::GP, WORDS = GP * 256;
  constexpr int WAVE = 3 * TILE + 4 * WORDS;  // K, V of two tiles, words of two tiles each
  constexpr int WPL = GROUP / 32;       // words of a group that a lane holds of a key's row
  constexpr int ND = D / 16;            // output tiles
  // The queries' operands lie in LDS where the registers are full: a spilled register's reload waits for the
  // copies in flight.
  constexpr bool kSumInRow = GP * NC <= 2;
  constexpr bool kQInLds = D == 256 || (D == 128 && (NC == 2 || GROUP == 32));
  static_assert(WAVE >= 16 * D * 4, "the joining of the waves takes the tiles' place");
  __shared__ __attribute__((aligned(1024))) uint8_t sm[4 * WAVE];
  __shared__ u32x4_t sq[kQInLds ? NC * GP * WPL * 64 : 1];
  __shared__ float sml[4][16 * NC][2];
  __shared__ int ssh[8];
  __shared__ int sfound[4];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  FewRun run;
  // An item's start and end take about as long as two tiles: with 0, 2, 3 or 4 units for them 64 ragged
  // sequences (8 heads, 128 values, 16-slot pages) take 91, 61, 64, 67 us.
  if (!few_run<256, 2, 4>(a, ssh, sfound, run)) return;
  const int u1 = run.u1, item_units = run.item_units;
  int s = run.s, base = run.base;

  uint8_t* sk = sm + wave * WAVE;
  uint8_t* svs = sk + TILE;
  uint8_t* swvs = svs + 2 * TILE;
  uint8_t* swks = swvs + 2 * WORDS;
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
    int lane = tid & 63;  // places are worked out in each item, not kept in registers
    asm volatile("" : "+v"(lane));

    const uint8_t* kb = a.k + (int64_t)head * a.head_stride;
    const uint8_t* vb = a.v + (int64_t)head * a.head_stride;
    const uint8_t* kw = a.kp + (int64_t)head * a.p_head_stride;
    const uint8_t* vw = a.vp + (int64_t)head * a.p_head_stride;
    const int32_t* table = a.table + (int64_t)s * a.table_stride;
    const int k00 = (first + ta) * 256 + wave * 64;
    tc.lookup(a, table, k00, lo, hi, lane, true);
    tc.resolve(a, lo, hi, lane);
    tc.template copy<false>(a, kb, kw, sk, swks, lane);
    tc.template copy<true>(a, vb, vw, svs, swvs, lane);
    uint64_t seen = tc.seen;

    const int g = lane >> 4, col = lane & 15;
    // The wave's queries: column c of tile n is row 16 n + c; a lane holds the values that meet its part
    // of the keys' rows, word by word; and, for the keys' biases, the sums of each group's values as two fp16
    // numbers a group (four groups a lane; every lane group takes part, with its share of the sum), held 2^16 times
    // larger than the codes' products: both together keep 22 bits, or 2^-29 of the row's largest value (at the
    // products' size the second one would be subnormal and keep 2^-13 of that; taking the 2^16 out costs 62.2 -> 63.2
    // us of 64 ragged sequences).
    u32x4_t qf[NC][GP * WPL];
    u32x4_t qb[NC];
    int qpos[NC];
    float sl[NC];  // scale * log2(e) * 2^(t + 24)
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      const int r = 16 * n + col;
      const int i = (int)a.g_div.div((uint32_t)r);
      const bool in = r < rows;
      qpos[n] = q.kv - q.nq + (in ? i : q.nq - 1);
      const uint8_t* qp = a.q + ((int64_t)(q.q0 + (in ? i : 0)) * a.q_ts + (int64_t)(head * a.g + (in ? r - i * a.g : 0)) * a.q_hs);
      float amax = 0.f;
#pragma unroll
      for (int x = 0; x < GP * WPL; ++x) {
        const u32x4_t z = {0, 0, 0, 0};
        const int word = (x / WPL) * (GROUP / 8) + g * WPL + x % WPL;
        qf[n][x] = in ? *(const u32x4_t*)(qp + word * 16) : z;
        amax = amax8(qf[n][x], a.io, amax);
      }
      const int t = q_exponent(join32(join16(amax, MaxF()), MaxF()));
      sl[n] = q_scale(a.sl, t + 24);
      float qs[GP];
#pragma unroll
      for (int x = 0; x < GP * WPL; ++x) {
        u32x4_t w = q_pairs(qf[n][x], a.io, t);
        float sum = x % WPL == 0 ? 0.f : qs[x / WPL];
#pragma unroll
        for (int y = 0; y < 4; ++y) sum = add2(F16{}, w[y], sum);
        qs[x / WPL] = sum;
        const f16x2_t sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
        w[1] = w2(h2(w[1]) * sixteenth), w[3] = w2(h2(w[3]) * sixteenth);
        if constexpr (kQInLds)
          sq[(n * GP * WPL + x) * 64 + lane] = w;  // each wave the same
        else
          qf[n][x] = w;
      }
#pragma unroll
      for (int x = 0; x < GP; ++x) qs[x] = join32(join16(qs[x], SumF()), SumF()) * (GP == 8 ? 0x1p-9f : 0x1p-10f);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        float v = x < GP ? qs[x % GP] : 0.f;
        if (GP == 8 && (g & 1)) v = qs[(x + 4) % GP];
        const float hi = f16_bits_to_f32(f32_to_f16_bits(v));
        qb[n][x] = pack2(F16{}, hi, v - hi);
      }
    }
    const int pos_lo = q.kv - q.nq, pos_hi = q.kv - 1;  // first and last query's position

    f32x4_t o[NC][ND], bs[NC][GP], ps[NC][GP];
    float m[NC], l[NC];
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      m[n] = kNegInf;
      l[n] = 0.f;
#pragma unroll
      for (int d = 0; d < ND; ++d) o[n][d] = f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int x = 0; x < GP; ++x) bs[n][x] = ps[n][x] = f32x4_t{0, 0, 0, 0};
    }
    int up[NC][GP];
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int x = 0; x < GP; ++x) up[n][x] = -14;
    uint32_t top[GP];  // uniform: every column's exponents cover scales (fp16 bits) below it
#pragma unroll
    for (int x = 0; x < GP; ++x) top[x] = 0x400u;
    if (ta + 1 < tb) tc.lookup(a, table, k00 + 256, lo, hi, lane, false);

    for (int t = ta; t < tb; ++t) {
      int ln = lane;  // LDS places are worked out in each tile, not kept in registers
      asm volatile("" : "+v"(ln));
      const int g = ln >> 4, col = ln & 15;
      const int k0 = (first + t) * 256 + wave * 64;
      const bool more = t + 1 < tb;
      const int now = (t - ta) & 1, next = now ^ 1;
      uint8_t* sv = svs + now * TILE;
      uint8_t* swv = swvs + now * WORDS;
      attn_wait_vm<Copy::COPIES>();  // K of this tile
      uint32_t kf[4][GP * WPL];
#pragma unroll
      for (int kt = 0; kt < 4; ++kt) {
        const int row = 16 * kt + col;
#pragma unroll
        for (int x = 0; x < GP; ++x) {
          const int byte = x * (GROUP / 2) + g * WPL * 4;
          const uint8_t* at = sk + row * ROW + ((byte >> 4) ^ swz4_k<D>(row)) * 16 + (byte & 15);
          if constexpr (WPL == 4) {
            const u32x4_t w = *(const u32x4_t*)at;
            for (int y = 0; y < 4; ++y) kf[kt][4 * x + y] = w[y];
          } else if constexpr (WPL == 2) {
            const u32x2_t w = *(const u32x2_t*)at;
            kf[kt][2 * x] = w[0], kf[kt][2 * x + 1] = w[1];
          } else {
            kf[kt][x] = *(const uint32_t*)at;
          }
        }
      }
      const uint64_t seen_now = seen;
      const uint8_t* kwords = swks + now * WORDS;
      if (more) {
        tc.resolve(a, lo, hi, ln);
        seen = tc.seen;
        attn_wait_lds();
        tc.template copy<false>(a, kb, kw, sk, swks + next * WORDS, ln);
        tc.template copy<true>(a, vb, vw, svs + next * TILE, swvs + next * WORDS, ln);
        if (t + 2 < tb) tc.lookup(a, table, k0 + 512, lo, hi, ln, false);
      }
      auto query = [&](int n, int x) {
        if constexpr (kQInLds)
          return sq[(n * GP * WPL + x) * 64 + ln];
        else
          return qf[n][x];
      };
      f32x4_t sc[NC][4];
#pragma unroll
      for (int kt = 0; kt < 4; ++kt) {
        u32x4_t w[GP];
#pragma unroll
        for (int x = 0; x < GP; ++x) w[x] = *(const u32x4_t*)(kwords + (kt * GP + x) * 64 + g * 16);
        u32x4_t kb2 = {0, 0, 0, 0};  // the biases of the lane's key, twice each
#pragma unroll
        for (int x = 0; x < (GP < 4 ? GP : 4); ++x) {
          const uint32_t b = *(const uint32_t*)(kwords + (kt * GP + x + (GP == 8 ? 4 * (g & 1) : 0)) * 64 + col * 4);
          kb2[x] = perm(b, b, 0x07060706u);
        }
        f32x4_t acc[NC][GP];
#pragma unroll
        for (int n = 0; n < NC; ++n) sc[n][kt] = mfma16(F16{}, kb2, qb[n], f32x4_t{0, 0, 0, 0});
#pragma unroll
        for (int x = 0; x < GP; ++x)
#pragma unroll
          for (int y = 0; y < WPL; ++y) {
            const u32x4_t c = codes_as_fp16(kf[kt][x * WPL + y]);
#pragma unroll
            for (int n = 0; n < NC; ++n)
              acc[n][x] = mfma16(F16{}, c, query(n, x * WPL + y), y == 0 ? f32x4_t{0, 0, 0, 0} : acc[n][x]);
          }
#pragma unroll
        for (int x = 0; x < GP; ++x)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float ks = (float)h2(w[x][r])[0];
#pragma unroll
            for (int n = 0; n < NC; ++n)
              sc[n][kt][r] = __builtin_fmaf(ks, acc[n][x][r], x == 0 ? sc[n][kt][r] * 0x1p-16f : sc[n][kt][r]);
          }
        __builtin_amdgcn_sched_barrier(0);  // one key tile at a time: its words and sums fit in the registers
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
      if (more)
        attn_wait_vm<2 * Copy::COPIES>();  // V of this tile; the next K and V may be in flight
      else
        attn_wait_vm<0>();
      // the exponents of the groups' largest scales so far: a group's products are held times 2^(7 - up)
      int up_now[NC][GP];
      if (cut && q.nq > 1) {  // of the keys that the column sees
#pragma unroll
        for (int x = 0; x < GP; ++x) {
          uint32_t big[NC];
#pragma unroll
          for (int n = 0; n < NC; ++n) big[n] = 0x400u;
#pragma unroll
          for (int kt = 0; kt < 4; ++kt) {
            const u32x4_t w = *(const u32x4_t*)(swv + (kt * GP + x) * 64 + g * 16);
#pragma unroll
            for (int r = 0; r < 4; ++r)
#pragma unroll
              for (int n = 0; n < NC; ++n)
                if (sc[n][kt][r] != kNegInf && !odd_word(w[r])) big[n] = max(big[n], w[r] & 0x7fffu);
          }
#pragma unroll
          for (int n = 0; n < NC; ++n) {
            const float all = join32(join16(__uint_as_float(big[n]), MaxF()), MaxF());  // ordered as their bits
            up_now[n][x] = max(up[n][x], (int)(__float_as_uint(all) >> 10) - 14);
          }
        }
      } else {
        uint32_t w[GP];
        bool more_up = false;
#pragma unroll
        for (int x = 0; x < GP; ++x) {
          w[x] = *(const uint32_t*)(swv + (g * GP + x) * 64 + col * 4) & 0x7fffu;
          more_up |= w[x] >= top[x];
#pragma unroll
          for (int n = 0; n < NC; ++n) up_now[n][x] = up[n][x];
        }
        if (__any(more_up)) {
#pragma unroll
          for (int x = 0; x < GP; ++x) {
            const int all = (int)(wave_max(w[x] >= 0x7c00u ? 0u : w[x]) >> 10);
            top[x] = max(top[x], (uint32_t)(all + 1) << 10);
#pragma unroll
            for (int n = 0; n < NC; ++n) up_now[n][x] = max(up[n][x], all - 14);
          }
        }
      }
      float e[NC][4][4];
      u32x4_t ew[NC][2];  // the same in fp16, pairs of keys 16 k + 4 g + i with k = (0, 1) and (2, 3)
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        float mx = fmaxf(fmaxf(sc[n][0][0], sc[n][1][0]), fmaxf(sc[n][2][0], sc[n][3][0]));
#pragma unroll
        for (int r = 1; r < 4; ++r) mx = max3(max3(mx, sc[n][0][r], sc[n][1][r]), sc[n][2][r], sc[n][3][r]);
        mx = join32(join16(mx, MaxF()), MaxF()) * sl[n];
        bool raise = mx > m[n] + kLazy;
#pragma unroll
        for (int x = 0; x < GP; ++x) raise |= up_now[n][x] > up[n][x];
        if (__any(raise)) {
          const float mn = mx > m[n] + kLazy ? mx : m[n];
          const float f = m[n] == kNegInf ? 0.f : exp2_fast(m[n] - mn);
          m[n] = mn;
          l[n] *= f;
#pragma unroll
          for (int x = 0; x < GP; ++x) {
            const float fx = __builtin_ldexpf(f, up[n][x] - up_now[n][x]);
            up[n][x] = up_now[n][x];
            for (int r = 0; r < (kSumInRow ? 4 : 2); ++r) bs[n][x][r] *= f;
            for (int r = 0; r < (kSumInRow ? 4 : 1); ++r) ps[n][x][r] *= fx;
#pragma unroll
            for (int d = x * (GROUP / 16); d < (x + 1) * (GROUP / 16); ++d)
              for (int r = 0; r < 4; ++r) o[n][d][r] *= fx;
          }
        }
        const float mr = m[n] == kNegInf ? 0.f : m[n];
#pragma unroll
        for (int kt = 0; kt < 4; ++kt)
#pragma unroll
          for (int r = 0; r < 4; ++r) e[n][kt][r] = exp2_fast(__builtin_fmaf(sc[n][kt][r], sl[n], -mr));
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            ew[n][h][r] = pack2(F16{}, e[n][2 * h][r], e[n][2 * h + 1][r]);
            l[n] = add2(F16{}, ew[n][h][r], l[n]);
          }
      }
      // a key that only some columns see may stand for an infinity or a NaN
      if (cut && q.nq > 1) {
        bool mine = false;
#pragma unroll
        for (int x = 0; x < GP; ++x) {
          mine |= odd_word(*(const uint32_t*)(swv + (g * GP + x) * 64 + col * 4));
        }
        const uint64_t keys = __ballot(mine);
        if (keys) few4_odd<D, GROUP, NC>(sv, swv, keys, ln, e, up, o);
      }
      const int vrow = 16 * (col >> 2) + 4 * g + (col & 3);
#pragma unroll
      for (int x = 0; x < GP; ++x) {
        // the weights times the keys' scales, in the same pairs
        u32x4_t p[NC][2];
        u32x4_t w[4];
#pragma unroll
        for (int kt = 0; kt < 4; ++kt) w[kt] = *(const u32x4_t*)(swv + (kt * GP + x) * 64 + g * 16);
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          const float even = __builtin_ldexpf(1.f, 7 - up[n][x]), odd = 0.0625f * even;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              // one instruction each: a fused product whose operand and result are halves
              f16x2_t y;
              y[0] = (_Float16)__builtin_fmaf(e[n][2 * h][r] * (r & 1 ? odd : even), (float)h2(w[2 * h][r])[0], 0.f);
              y[1] = (_Float16)__builtin_fmaf(e[n][2 * h + 1][r] * (r & 1 ? odd : even), (float)h2(w[2 * h + 1][r])[0], 0.f);
              p[n][h][r] = w2(y);
            }
        }
        // the sums of weight times scale (even rows) and times bias (odd rows), and of those products by a row of
        // ones, which are normal numbers: ones held as the codes are, 2^-24, drop the low bits of a sum that counts
        // 8 times (16000 tokens, fp16: off by 0.0010 of the output, so 0.0003); where that takes too many registers
        // on the vector units
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (kSumInRow) {
            u32x4_t sb;
            const uint32_t half = ln & 1 ? 0x07060302u : 0x05040100u;
#pragma unroll
            for (int r = 0; r < 4; ++r) sb[r] = perm(w[2 * h + 1][r], w[2 * h][r], half);
#pragma unroll
            for (int n = 0; n < NC; ++n) {
              bs[n][x] = mfma16(F16{}, sb, ew[n][h], bs[n][x]);
              ps[n][x] = mfma16(F16{}, u32x4_t{0x3c003c00u, 0x4c004c00u, 0x3c003c00u, 0x4c004c00u}, p[n][h], ps[n][x]);
            }
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const uint32_t s = perm(w[2 * h + 1][r], w[2 * h][r], 0x05040100u), b = perm(w[2 * h + 1][r], w[2 * h][r], 0x07060302u);
#pragma unroll
              for (int n = 0; n < NC; ++n) {
                bs[n][x][0] = dot2(F16{}, ew[n][h][r], s, bs[n][x][0]);
                bs[n][x][1] = dot2(F16{}, ew[n][h][r], b, bs[n][x][1]);
                ps[n][x][0] = dot2(F16{}, p[n][h][r], r & 1 ? 0x4c004c00u : 0x3c003c00u, ps[n][x][0]);  // 16 or 1
              }
            }
          }
        }
#pragma unroll
        for (int dd = 0; dd < GROUP / 16; ++dd) {
          const int d = x * (GROUP / 16) + dd;
          const u32x2_t c = read_tr4(sv + vrow * ROW + (((d >> 1) ^ swz4_v<D>(vrow)) * 16) + 8 * (d & 1));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const u32x4_t v = codes_as_fp16(c[h]);
#pragma unroll
            for (int n = 0; n < NC; ++n) o[n][d] = mfma16(F16{}, v, p[n][h], o[n][d]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }

    // to the units of the sums: the factors of the weights and of the codes, and the groups' middles
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int x = 0; x < GP; ++x) {
        const float held = __builtin_ldexpf(1.f, up[n][x] + 24 - 7);
        float sum = ps[n][x][0], ss = bs[n][x][0], sb = bs[n][x][1];
        if (!kSumInRow) {
          sum = join32(join16(sum, SumF()), SumF());
          ss = join32(join16(ss, SumF()), SumF());
          sb = join32(join16(sb, SumF()), SumF());
        }
        const float b = sb + 8.f * (ss - sum * (held * 0x1p-24f));
#pragma unroll
        for (int d = x * (GROUP / 16); d < (x + 1) * (GROUP / 16); ++d)
          for (int r = 0; r < 4; ++r) o[n][d][r] = __builtin_fmaf(o[n][d][r], held, b);
      }
    const bool whole = ta == 0 && tb == nt;
    int end_tid = tid;  // its places are worked out here, not kept in registers over the tiles
    asm volatile("" : "+v"(end_tid));
    few_finish<D, NC>(a, end_tid, sm, WAVE, sml, o, m, l, run.w, q, head, rows, ta == 0, whole,
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
