// Paged attention, many rows: tiles of 256 query rows (128 at 256 values a head) of one sequence and
// kv head (the query heads that share it are folded into the rows: row r is token r / g, head r % g
// of the group).
//
// The matrix cores bound it: 4 D flops per row and key against D / 64 bytes of cache (a tile of keys
// is read once for 256 rows).  8 waves hold 32 rows each, two on every SIMD.  Every wave turns a
// tile's scores into weights on the vector units, then multiplies: O += V^T P^T of this tile and
// S^T = K Q^T of the next, one stream of 32x32x16 products whose LDS fragments are read ahead.  One
// barrier a tile, met by the first four waves after their products and by the others after their
// weights, keeps the two groups half a tile apart, so that one multiplies while the other is on the
// vector units.  (Left to themselves the two waves of a SIMD fall into step and wait for the same
// unit: matrix cores 42 % busy, vector units 37 %, never together, 646 us against 495 for 1000
// tokens at 32767, 32 heads on 8 of 128.  A barrier at every half tile: 520.  Now 51 %, what is left
// is each wave's own chain of weights and products; two waves a SIMD fill the registers.)  The
// first four waves copy the K and V tiles into LDS, a period ahead of their first reader
// (attn_order.hpp has the order of it all).
//
// At 256 values a head the registers hold one wave a SIMD, 4 waves, all in step: weights and products
// take turns, matrix cores 34 % busy.  At 64 values the vector units bound it: a tile takes as many
// exponentials as at 128 for half the products (matrix cores 34 % busy, vector issue 55 %).
//
// Measured (bf16, 32 heads on 8 of 128): 4096 tokens 143 us, 960 TFLOP/s; 1000 tokens at 32767
// 495 us, 1070 TFLOP/s; a large bf16 library product reaches 1219 here.  The same with 64 heads on 16
// of 64: 206 us, 670 and 639 us, 830; with 16 heads on 4 of 256: 172 us, 800 and 648 us, 820.
//
// Work split.  With enough items (sequence, kv head, row tile) to fill the chip, one workgroup each,
// the longest first, kv heads fastest so that a head's tiles run on one XCD and share its L2.  Else
// all items are laid end to end in units of one row tile x 64 keys and cut into equal runs, one
// per compute unit; cut items leave pieces for the joining kernel.
#include <algorithm>
#include <type_traits>

#include "attn_common.hpp"
#include "attn_order.hpp"

namespace ql {
namespace {

constexpr int BN = kAttnTileKeys;
// LDS fragments read ahead of the products that take them: a product lasts 32 cycles, a read about
// four of them.  The order is pinned, since the compiler puts each read right before its product.
constexpr int kAhead = 4;
// An item's start and end, and its pieces' way through memory, cost as much as several of its key
// tiles (10 against 2 us): in the division of the work each item has units for them before its first
// tile (0, 4, 8, 12 units: 12 mixed sequences 147, 144, 141, 144 us; 8 x 500 tokens 73, 68, 58, 57).
constexpr int kItemUnits = 8;

// Stages of K and of V: the two wave groups read neighbouring tiles while a third is copied; one
// group reads one.
constexpr int tile_stages(int d) { return d == 256 ? 2 : 3; }
// LDS for the finite copies of two V tiles, one for each wave group (at 256 values a head none is
// left).
constexpr int tile_clean_bytes(int d) { return d == 256 ? 0 : 2 * BN * d * 2; }

// V^T fragment of 32 values (tile dt) x 16 keys (step ks): two transposing reads of 4 keys each.
template <int D> __device__ __forceinline__ u32x4_t v_frag(const uint8_t* sv, int lane, int dt, int ks) {
  const int h = lane >> 5, l = lane & 15;
  const int row = 16 * ks + 4 * h + (l >> 2);
  const int c = 4 * dt + 2 * ((lane >> 4) & 1) + ((l & 3) >> 1);
  const uint8_t* at = sv + row * (D * 2) + 8 * (l & 1);
  const s16x4_t v0 = read_tr(at + (c ^ swz_v<D>(row)) * 16);
  const s16x4_t v1 = read_tr(at + 8 * D * 2 + (c ^ swz_v<D>(row + 8)) * 16);
  const u32x2_t w0 = __builtin_bit_cast(u32x2_t, v0), w1 = __builtin_bit_cast(u32x2_t, v1);
  return u32x4_t{w0[0], w0[1], w1[0], w1[1]};
}

// Adds the non-finite values of a V tile to the wave's columns whose P is not zero.
template <typename T, int D>
__device__ __forceinline__ void tile_nonfinite(const uint8_t* sv, int lane, const u32x4_t* p, f32x16_t* o) {
  asm volatile("" : "+v"(lane));  // the addresses stay in this rare path
  const int h = lane >> 5, col = lane & 31;
#pragma unroll 1
  for (int j = 0; j < BN; ++j) {
    // P of key j: of its 16 keys (step j / 16), key 8 x + 4 h + y is value 4 x + y of half h, in
    // word 2 x + y / 2
    uint32_t w = 0;
#pragma unroll
    for (int x = 0; x < BN / 4; ++x) w = x == 4 * (j >> 4) + 2 * ((j >> 3) & 1) + ((j >> 1) & 1) ? p[x >> 2][x & 3] : w;
    w = __shfl(w, 32 * ((j >> 2) & 1) + col);
    const bool on = ((j & 1) ? w >> 16 : w) & 0x7fffu;
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const u32x2_t v = *(const u32x2_t*)(sv + j * (D * 2) + ((4 * d + y) ^ swz_v<D>(j)) * 16 + 8 * h);
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          float x0, x1;
          only_nonfinite<T>(v[z], on, x0, x1);
          o[d][4 * y + 2 * z] += x0;
          o[d][4 * y + 2 * z + 1] += x1;
        }
      }
  }
}

// Units of row tile j of a sequence: its span's tiles of BN keys.
template <int BM> __device__ __forceinline__ int tile_cost(const AttnArgs& a, const AttnSeq& q, int j, int& lo, int& hi, int& first) {
  const int i0 = (int)a.g_div.div((uint32_t)(j * BM));
  const int i1 = min(q.nq - 1, (int)a.g_div.div((uint32_t)(j * BM + BM - 1)));
  attn_span(a, q, i0, i1, lo, hi);
  return attn_tiles<BN>(lo, hi, first);
}
template <int BM> __device__ __forceinline__ int row_tiles(const AttnArgs& a, int s) {
  if (s >= a.n_seqs) return 0;
  const AttnSeq q = attn_seq(a, s);
  return q.nq < 1 || attn_is_few(a, q.nq) ? 0 : (q.nq * a.g + BM - 1) / BM;
}

template <typename T, int D, bool RUNS>
__global__ __launch_bounds__(64 * attn_tile_waves(D), attn_tile_waves(D) / 4) void attn_tile_kernel(const AttnArgs a) {
  constexpr int WAVES = attn_tile_waves(D), BM = 32 * WAVES;
  constexpr int ROW = D * 2;
  constexpr int KB = BN * ROW;  // bytes of a K (or V) stage
  constexpr int NK = BN / 32;   // score tiles of 32 keys
  constexpr int NS = D / 16;    // k-steps of the scores
  constexpr int ND = D / 32;    // output tiles of 32 values
  constexpr int NV = BN / 16;   // k-steps of the output
  constexpr int R = BN / 4;     // keys of a tile that each of the first four waves copies
  constexpr bool kClean = tile_clean_bytes(D) > 0;
  constexpr int ST = tile_stages(D);  // stages of K, and of V
  // K stages, V stages, finite copies of V, then (RUNS) the plan
  extern __shared__ __attribute__((aligned(1024))) uint8_t sm[];
  __shared__ int ssh[WAVES];
  __shared__ int sfound[4];
  __shared__ __attribute__((aligned(8))) uint16_t sseen[4][4];  // bit j: key j is loaded
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = lane >> 5, col = lane & 31;

  int u0, u1, W, nw, w;
  // RUNS: first unit (of one head) of each row tile, then the sequences' first tiles
  int* plan = (int*)(sm + 2 * ST * KB + tile_clean_bytes(D));
  int nt_all = 0;
  int* seq_first = nullptr;
  AttnRecord* rec = nullptr;
  if constexpr (RUNS) {
    // first tile of each sequence, then first unit of each tile
    seq_first = plan + a.plan_tiles + 1;
    for (int s0 = 0; s0 < a.n_seqs; s0 += 64 * WAVES) {
      int total;
      const int e = block_scan<WAVES>(row_tiles<BM>(a, s0 + tid), ssh, total);
      if (s0 + tid < a.n_seqs) seq_first[s0 + tid] = nt_all + e;
      nt_all += total;
    }
    nt_all = min(nt_all, a.plan_tiles);  // overlapping sequences could ask for more than t rows hold
    __syncthreads();
    int units = 0;
    for (int t0 = 0; t0 < nt_all; t0 += 64 * WAVES) {
      const int ti = t0 + tid;
      int c = 0;
      if (ti < nt_all) {
        int b = 0, e = a.n_seqs;  // the last sequence with seq_first <= ti
        while (e - b > 1) {
          const int m = (b + e) / 2;
          if (seq_first[m] <= ti) b = m; else e = m;
        }
        int lo, hi, first;
        c = kItemUnits + tile_cost<BM>(a, attn_seq(a, b), ti - seq_first[b], lo, hi, first);
      }
      int total;
      const int e = block_scan<WAVES>(c, ssh, total);
      if (ti < nt_all) plan[ti] = units + e;
      units += total;
    }
    if (tid == 0) plan[nt_all] = units;
    __syncthreads();
    W = units * a.hk;
    nw = min(a.nw_tile, W);
    // workgroups of one XCD (every 8th) take neighbouring runs
    const int per = a.nw_tile / 8;
    w = (blockIdx.x & 7) * per + (blockIdx.x >> 3);
    rec = a.rec + a.nw_few + w;
    if (a.tile_by_item) {  // the first workgroup clears the records of items that there are not
      if (blockIdx.x == 0)
        for (int i = nt_all * a.hk + tid; i < a.plan_tiles * a.hk; i += 64 * WAVES) a.rec[a.nw_few + i].pieces = 0;
    } else if (w >= nw && tid == 0) {
      rec->pieces = 0;
    }
    if (w >= nw) return;
    u0 = attn_cut(w, nw, W);
    u1 = attn_cut(w + 1, nw, W);
  } else {
    w = 0, nw = 1, W = 0;
    u0 = blockIdx.x;
    u1 = u0 + 1;
  }

  const int late = wave / 4;  // the second four waves run half a tile behind
  const bool copier = wave < 4;
  const int row0 = R * (wave & 3);  // first key of a tile that a copying wave copies
  TileCopy<D, R, 1, BN, false> tc;
  tc.init(a, row0, lane);
  bool recorded = false;
  for (int u = u0; u < u1;) {
    int s, j, head, ta, tb, nt, item0 = 0, lo, hi, first;
    AttnSeq q;
    if constexpr (RUNS) {
      const int units = plan[nt_all];
      head = u / units;
      const int uh = u - head * units;
      int b = 0, e = nt_all;
      while (e - b > 1) {
        const int m = (b + e) / 2;
        if (plan[m] <= uh) b = m; else e = m;
      }
      const int ti = b;
      nt = plan[ti + 1] - plan[ti] - kItemUnits;
      item0 = head * units + plan[ti] + kItemUnits;  // the item's tiles are the units [item0, item0 + nt)
      ta = max(0, u - item0);
      tb = min(nt, u1 - item0);
      u = item0 + nt;
      if (tb <= ta) continue;  // the run ends before the item's first tile
      if (a.tile_by_item) {
        rec = a.rec + a.nw_few + ti * a.hk + head;
        if (ta == 0 && tb == nt && tid == 0) rec->pieces = 0;
      }
      b = 0, e = a.n_seqs;
      while (e - b > 1) {
        const int m = (b + e) / 2;
        if (seq_first[m] <= ti) b = m; else e = m;
      }
      s = __builtin_amdgcn_readfirstlane(b);
      j = __builtin_amdgcn_readfirstlane(ti - seq_first[b]);
      head = __builtin_amdgcn_readfirstlane(head);
      q = attn_seq(a, s);
      tile_cost<BM>(a, q, j, lo, hi, first);
    } else {
      head = u % a.hk;
      const int target = u / a.hk;
      int before = 0;
      if (tid == 0) sfound[0] = -1;
      for (int s0 = 0; s0 < a.n_seqs; s0 += 64 * WAVES) {
        int total;
        const int c = row_tiles<BM>(a, s0 + tid);
        const int e = before + block_scan<WAVES>(c, ssh, total);
        if (e <= target && target < e + c) sfound[0] = s0 + tid, sfound[1] = c - 1 - (target - e);  // longest first
        before += total;
        if (before > target) break;
      }
      __syncthreads();
      s = sfound[0], j = sfound[1];
      if (s < 0) return;  // more workgroups than row tiles
      q = attn_seq(a, s);
      nt = tile_cost<BM>(a, q, j, lo, hi, first);
      ta = 0, tb = nt;
      u = u1;
    }
    const int rows = min(BM, q.nq * a.g - j * BM);

    // The wave's 32 rows, one per column.
    const int r = j * BM + 32 * wave + col;
    const bool in = r < q.nq * a.g;
    const int i = in ? (int)a.g_div.div((uint32_t)r) : q.nq - 1;
    const int hq = head * a.g + (in ? r - i * a.g : 0);
    const int qpos = q.kv - q.nq + i;
    u32x4_t qf[NS];
    {
      const uint8_t* qp = a.q + ((int64_t)(q.q0 + i) * a.q_ts + (int64_t)hq * a.q_hs);
#pragma unroll
      for (int st = 0; st < NS; ++st) {
        const u32x4_t z = {0, 0, 0, 0};
        qf[st] = in ? *(const u32x4_t*)(qp + (2 * st + h) * 16) : z;
      }
    }
    // first and last position among the wave's rows
    const int pos_lo = q.kv - q.nq + min(q.nq - 1, (int)a.g_div.div((uint32_t)(j * BM + 32 * wave)));
    const int pos_hi = q.kv - q.nq + min(q.nq - 1, (int)a.g_div.div((uint32_t)(j * BM + 32 * wave + 31)));

    // and among the workgroup's
    const int wg_lo = q.kv - q.nq + (int)a.g_div.div((uint32_t)(j * BM));
    const int wg_hi = q.kv - q.nq + min(q.nq - 1, (int)a.g_div.div((uint32_t)(j * BM + BM - 1)));
    const bool idle = 32 * wave >= rows;

    f32x16_t o[ND];
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int x = 0; x < 16; ++x) o[d][x] = 0.f;
    float m = kNegInf, l = 0.f;
    f32x16_t sc[NK];
    u32x4_t p[NV];

    const uint8_t* kb = a.k + (int64_t)head * a.head_stride;
    const uint8_t* vb = a.v + (int64_t)head * a.head_stride;
    const int32_t* table = a.table + (int64_t)s * a.table_stride;
    const int n = tb - ta, kfirst = (first + ta) * BN;
    auto stage_k = [&](int t) { return sm + attn_stage<ST>(t) * KB; };
    auto stage_v = [&](int t) { return sm + (ST + attn_stage<ST>(t)) * KB; };
    auto copy_k = [&](int t) {
      tc.resolve(a, lo, hi, lane);
      if (lane == 0) sseen[attn_seen_at(t)][wave & 3] = (uint16_t)tc.seen;
      tc.template copy<false>(tc.now, kb, stage_k(t) + row0 * ROW, row0, lane);
      if (t + 1 < n) tc.lookup(a, table, kfirst + (t + 1) * BN + row0, lo, hi, lane, false);
    };
    auto is_cut = [&](int t) {  // whether some row does not see all of it
      const int k0 = kfirst + t * BN;
      return k0 + BN - 1 > pos_lo || (a.window > 0 && k0 <= pos_hi - a.window);
    };

    // Without room for a finite copy the workgroup cleans the tile in place, all waves (which are in
    // step there) between barriers: a quarter is searched and cleaned by each.
    auto wg_cut = [&](int t) {
      const int k0 = kfirst + t * BN;
      return k0 + BN - 1 > wg_lo || (a.window > 0 && k0 <= wg_hi - a.window);
    };
    auto found_odd = [&](int t) {
      uint32_t acc = 0;
#pragma unroll 4
      for (int x = 0; x < KB / (1024 * WAVES); ++x) {
        const u32x4_t v = *(const u32x4_t*)(stage_v(t) + x * (1024 * WAVES) + tid * 16);
        for (int y = 0; y < 4; ++y) acc |= nonfinite2<T>(v[y]);
      }
      return __syncthreads_or((acc & 0x80008000u) != 0) != 0;
    };
    auto clean_in_place = [&](int t) {
      attn_barrier();
#pragma unroll 4
      for (int x = 0; x < KB / (1024 * WAVES); ++x) {
        u32x4_t* at = (u32x4_t*)(stage_v(t) + x * (1024 * WAVES) + tid * 16);
        u32x4_t v = *at;
        for (int y = 0; y < 4; ++y) v[y] = finite2<T>(v[y]);
        *at = v;
      }
      attn_barrier();
    };

    // Products A .. B of the list: first the NV ND of output(t), o += V^T P^T, then the NK NS of
    // scores(t + 1), with the LDS fragments read kAhead products before their own.
    constexpr int NO = NV * ND, NP = NO + NK * NS;
    auto products = [&](int t, auto A, auto B) {
      const uint8_t* sv = stage_v(t);
      if (!kClean && A < NO && wg_cut(t) && found_odd(t)) {
        tile_nonfinite<T, D>(sv, lane, p, o);
        clean_in_place(t);
      }
      if (kClean && A < NO && is_cut(t)) {  // a key that only some rows see may hold an infinity or a NaN
        uint32_t acc = 0;
#pragma unroll 4
        for (int x = 0; x < KB / 1024; ++x) {
          const u32x4_t v = *(const u32x4_t*)(sv + x * 1024 + lane * 16);
          for (int y = 0; y < 4; ++y) acc |= nonfinite2<T>(v[y]);
        }
        const bool odd = __any((acc & 0x80008000u) != 0);
        if (odd) {
          tile_nonfinite<T, D>(sv, lane, p, o);
          // every wave that meets such a tile writes the same finite copy of it before its own reads
          uint8_t* clean = sm + (2 * ST + attn_clean_at(t)) * KB;
#pragma unroll 4
          for (int x = 0; x < KB / 1024; ++x) {
            u32x4_t v = *(const u32x4_t*)(sv + x * 1024 + lane * 16);
            for (int y = 0; y < 4; ++y) v[y] = finite2<T>(v[y]);
            *(u32x4_t*)(clean + x * 1024 + lane * 16) = v;
          }
          sv = clean;
        }
      }
      const uint8_t* kr = stage_k(t + 1) + col * ROW;
      auto load = [&](int i) {
        if (i >= NO) {  // step j / NK of keys 32 (j % NK) ..
          const int j = i - NO;
          return *(const u32x4_t*)(kr + (j % NK) * (32 * ROW) + ((2 * (j / NK) + h) ^ swz_k<D>(col)) * 16);
        }
        return v_frag<D>(sv, lane, i % ND, i / ND);
      };
      if (B > NO) {
#pragma unroll
        for (int kt = 0; kt < NK; ++kt)
#pragma unroll
          for (int x = 0; x < 16; ++x) sc[kt][x] = 0.f;
      }
      u32x4_t f[NP];
#pragma unroll
      for (int i = A; i < A + kAhead; ++i) f[i] = load(i);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = A; i < B; ++i) {
        if (i < NO)
          o[i % ND] = mfma32(T{}, f[i], p[i / ND], o[i % ND]);
        else
          sc[(i - NO) % NK] = mfma32(T{}, f[i], qf[(i - NO) / NK], sc[(i - NO) % NK]);
        if (i + kAhead < B) f[i + kAhead] = load(i + kAhead);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    constexpr std::integral_constant<int, 0> kFirst{};
    constexpr std::integral_constant<int, NO> kScores{};
    constexpr std::integral_constant<int, NP> kLast{};

    auto weights = [&](int t) {
      const int k0 = kfirst + t * BN;
      if (is_cut(t)) {
        asm volatile("");  // kept a branch: few tiles are cut
        const int last = qpos - k0 - 4 * h, before = a.window > 0 ? last - a.window : -BN - 1;
#pragma unroll
        for (int x = 0; x < 16 * NK; ++x) {
          const int jj = 32 * (x >> 4) + 8 * ((x >> 2) & 3) + (x & 3);
          sc[x >> 4][x & 15] = ((int)(jj <= last) & (int)(jj > before)) ? sc[x >> 4][x & 15] : kNegInf;
        }
      }
      const uint64_t seen = *(const uint64_t*)sseen[attn_seen_at(t)];
      if (seen != ~(uint64_t)0) {
        asm volatile("");
        const uint32_t s0 = (uint32_t)seen >> (4 * h), s1 = (uint32_t)(seen >> 32) >> (4 * h);
#pragma unroll
        for (int x = 0; x < 32; ++x)
          sc[x >> 4][x & 15] = ((x < 16 ? s0 : s1) >> (8 * ((x >> 2) & 3) + (x & 3)) & 1) ? sc[x >> 4][x & 15] : kNegInf;
      }
      static_assert(NK == 2, "two score tiles");
      float mx = fmaxf(sc[0][0], sc[NK - 1][0]);
#pragma unroll
      for (int x = 1; x < 16; ++x) mx = max3(mx, sc[0][x], sc[NK - 1][x]);
      mx = join32(mx, MaxF()) * a.sl;
      if (__any(mx > m + kLazy)) {
        const float mn = fmaxf(m, mx);
        const float f = m == kNegInf ? 0.f : exp2_fast(m - mn);
        m = mn;
        l *= f;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int x = 0; x < 16; ++x) o[d][x] *= f;
      }
      const float mr = m == kNegInf ? 0.f : m;
#pragma unroll
      for (int ks = 0; ks < NV; ++ks) {
        float e[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) e[x] = exp2_fast(__builtin_fmaf(sc[ks >> 1][8 * (ks & 1) + x], a.sl, -mr));
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          p[ks][x] = pack2(T{}, e[2 * x], e[2 * x + 1]);
          l = add2(T{}, p[ks][x], l);
        }
      }
    };
    attn_tile_order<ST>(n, copier, late, idle, [&](auto what, int t) {
      constexpr AttnStep S = decltype(what)::value;
      if constexpr (S == AttnStep::kBarrier) attn_barrier();
      if constexpr (S == AttnStep::kPages) tc.lookup(a, table, kfirst + row0, lo, hi, lane, true);
      if constexpr (S == AttnStep::kCopyK) copy_k(t);
      if constexpr (S == AttnStep::kCopyV) tc.template copy<true>(tc.now, vb, stage_v(t) + row0 * ROW, row0, lane);
      if constexpr (S == AttnStep::kWait) attn_wait_vm<0>();
      if constexpr (S == AttnStep::kScores) products(t - 1, kScores, kLast);
      if constexpr (S == AttnStep::kWeights) weights(t);
      if constexpr (S == AttnStep::kProducts) products(t, kFirst, kLast);
      if constexpr (S == AttnStep::kIdle) {
        if (!kClean && wg_cut(t) && found_odd(t)) clean_in_place(t);
      }
    });
    l = join32(l, SumF());

    // The lane holds its row's values 32 d + 8 y + 4 h .. + 3.
    if (!RUNS || (ta == 0 && tb == nt)) {
      if (in) {
        const float inv = attn_scale(a.sinks, hq, m, l);
        uint8_t* op = a.out + ((int64_t)(q.q0 + i) * a.out_ts + (int64_t)hq * a.out_hs) + 8 * h;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int y = 0; y < 4; ++y)
            store4(T{}, op + 64 * d + 16 * y, o[d][4 * y] * inv, o[d][4 * y + 1] * inv, o[d][4 * y + 2] * inv,
                   o[d][4 * y + 3] * inv);
      }
    } else {
      float* part = a.part_tile + (int64_t)(ta == 0 ? 2 * w + 1 : 2 * w) * (BM * (D + 2));
      const int row = 32 * wave + col;
      if (row < rows) {
        if (h == 0) part[row] = m, part[BM + row] = l;
        float* po = part + 2 * BM + row * D + 4 * h;
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int y = 0; y < 4; ++y)
            *(f32x4_t*)(po + 32 * d + 8 * y) = f32x4_t{o[d][4 * y], o[d][4 * y + 1], o[d][4 * y + 2], o[d][4 * y + 3]};
      }
      if (ta == 0) {
        recorded = true;
        if (tid == 0) {
          AttnRecord rr = {};
          rr.w = w;
          rr.pieces = attn_last(item0 + nt, nw, W) - w + 1;
          rr.q0 = q.q0;
          rr.row0 = j * BM;
          rr.rows = rows;
          rr.head = head;
          *rec = rr;
        }
      }
    }
  }
  if constexpr (RUNS) {
    if (!recorded && !a.tile_by_item && tid == 0) rec->pieces = 0;
  }
}

// Joins the pieces of the items that were cut.  The threads of a row hold 4 values each; a block has
// room for SLOTS rows, or for fewer whose pieces are shared out to `lanes` of them: each lane keeps
// a running maximum and sum over its pieces, four loads in flight, and the lanes join in LDS.  The
// host sets lanes from the pieces an item has on average (one sequence of 131071, 4 rows of 64
// pieces: 33 us with one lane; 12 mixed sequences, 256-row items of 3 pieces: 25 us with two).
constexpr int kJoinThreads = 256;
template <int D> constexpr int join_slots() { return kJoinThreads / (D / 4); }
template <typename T, int D>
__global__ __launch_bounds__(kJoinThreads) void attn_join_kernel(const AttnArgs a, int few_blocks, int few_per,
                                                                 int few_lanes, int tile_per, int tile_lanes) {
  constexpr int TPR = D / 4, SLOTS = join_slots<D>(), BM = 32 * attn_tile_waves(D);
  __shared__ f32x4_t sx[kJoinThreads];
  __shared__ float sl[SLOTS], sm[SLOTS];
  const bool is_few = (int)blockIdx.x < few_blocks;
  const int b = is_few ? blockIdx.x : blockIdx.x - few_blocks;
  const int per = is_few ? few_per : tile_per, lanes = is_few ? few_lanes : tile_lanes;
  const AttnRecord r = a.rec[(is_few ? 0 : a.nw_few) + b / per];
  const int row0 = b % per * (SLOTS / lanes);
  if (r.pieces == 0 || row0 >= r.rows) return;
  const int w = r.w;
  const int cap = is_few ? a.cap_few : BM;
  const int slot_floats = is_few ? a.part_floats : BM * (D + 2);
  const float* part = is_few ? a.part : a.part_tile;
  const int c = threadIdx.x % TPR, slot = threadIdx.x / TPR;
  const int lane = slot & (lanes - 1), row = row0 + slot / lanes, row_end = r.rows;
  auto piece = [&](int p) { return part + (int64_t)(p == 0 ? 2 * w + 1 : 2 * (w + p)) * slot_floats; };
  {
    float m = kNegInf, l = 0.f;
    f32x4_t x = {0, 0, 0, 0};
    if (row < row_end) {
      for (int p0 = lane; p0 < r.pieces; p0 += 4 * lanes) {
        float mp[4], lp[4];
        f32x4_t v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int p = p0 + i * lanes;
          mp[i] = kNegInf;
          lp[i] = 0.f;
          v[i] = f32x4_t{0, 0, 0, 0};
          if (p < r.pieces) {
            const float* sp = piece(p);
            mp[i] = sp[row];
            lp[i] = sp[cap + row];
            v[i] = *(const f32x4_t*)(sp + 2 * cap + row * D + 4 * c);
          }
        }
        const float mn = max3(max3(mp[0], mp[1], mp[2]), mp[3], m);
        const float f = m == kNegInf ? (l == 0.f ? 0.f : 1.f) : exp2_fast(m - mn);
        l = f == 0.f ? 0.f : l * f;
        for (int y = 0; y < 4; ++y) x[y] = f == 0.f ? 0.f : x[y] * f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float fp = join_factor(mp[i], lp[i], mn);
          if (fp != 0.f) {
            l += lp[i] * fp;
            x += v[i] * fp;
          }
        }
        m = mn;
      }
    }
    if (lanes > 1) {
      __syncthreads();
      sx[threadIdx.x] = x;
      if (c == 0) sl[slot] = l, sm[slot] = m;
      __syncthreads();
      if (lane == 0) {
        float mt = m;
        for (int i = 1; i < lanes; ++i) mt = fmaxf(mt, sm[slot + i]);
        l = 0.f;
        x = f32x4_t{0, 0, 0, 0};
        for (int i = 0; i < lanes; ++i) {
          const float li = sl[slot + i], f = join_factor(sm[slot + i], li, mt);
          if (f != 0.f) {
            l += li * f;
            x += sx[threadIdx.x + i * TPR] * f;
          }
        }
        m = mt;
      }
    }
    if (lane == 0 && row < row_end) {
      const int rr = r.row0 + row;
      const int tok = (int)a.g_div.div((uint32_t)rr);
      const int hq = r.head * a.g + rr - tok * a.g;
      const float inv = attn_scale(a.sinks, hq, m, l);
      uint8_t* op = a.out + ((int64_t)(r.q0 + tok) * a.out_ts + (int64_t)hq * a.out_hs) + c * 8;
      store4(T{}, op, x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
    }
  }
}

template <typename T, int D> hipError_t tile(const AttnArgs& a, hipStream_t s) {
  const size_t lds = (size_t)2 * tile_stages(D) * BN * D * 2 + tile_clean_bytes(D);
  constexpr int threads = 64 * attn_tile_waves(D);
  if (a.nw_tile > 0) {
    const size_t plan = ((size_t)a.plan_tiles + 1 + a.n_seqs) * 4;
    attn_tile_kernel<T, D, true><<<a.nw_tile, threads, lds + plan, s>>>(a);
  } else {
    attn_tile_kernel<T, D, false><<<a.items_tile, threads, lds, s>>>(a);
  }
  return hipGetLastError();
}
template <typename T, int D> hipError_t join(const AttnArgs& a, hipStream_t s) {
  constexpr int SLOTS = join_slots<D>(), BM = 32 * attn_tile_waves(D);
  // pieces of an item, on average, at four a lane
  auto lanes_for = [](int64_t workgroups, int64_t items) {
    int n = 1;
    while (n < SLOTS && 4 * n * items < workgroups) n *= 2;
    return n;
  };
  int few = 0, few_per = 1, few_lanes = 1, many = 0, tile_per = 1, tile_lanes = 1;
  if (a.join_few) {
    few_lanes = lanes_for(a.nw_few, (int64_t)a.n_seqs * a.hk);
    const int rows = (int)std::min<int64_t>(a.cap_few, (int64_t)a.max_q * a.g);
    few_per = (rows * few_lanes + SLOTS - 1) / SLOTS;
    few = (a.few_by_item ? a.n_seqs * a.hk : a.nw_few) * few_per;
  }
  if (a.nw_tile > 0 && a.join_tile) {
    tile_lanes = lanes_for(a.nw_tile, (int64_t)a.plan_tiles * a.hk);
    const int rows = (int)std::min<int64_t>(BM, (int64_t)a.max_q * a.g);
    tile_per = (rows * tile_lanes + SLOTS - 1) / SLOTS;
    many = (a.tile_by_item ? a.plan_tiles * a.hk : a.nw_tile) * tile_per;
  }
  if (few + many == 0) return hipSuccess;
  attn_join_kernel<T, D><<<few + many, kJoinThreads, 0, s>>>(a, few, few_per, few_lanes, tile_per, tile_lanes);
  return hipGetLastError();
}

}  // namespace

AttnPlan attn_plan(int64_t t, int64_t n_seqs, int64_t hq, int64_t hk, int d, int64_t max_q, int64_t max_kv,
                   int64_t window) {
  AttnPlan p{};
  const int64_t g = hq / hk, bm = 32 * attn_tile_waves(d);
  const int64_t cap = d == 256 ? 16 : 32;  // rows whose registers fit
  const int64_t limit = int64_t(1) << 31;
  // a product of counts, cut at the limit (three of them pass 2^63 within what the caller accepts)
  auto times = [&](int64_t x, int64_t y) { return y > 0 && x >= (limit + y - 1) / y ? limit : x * y; };
  // longest span of an item; any window from max_kv on hides nothing
  const int64_t span = window > 0 && window < max_kv ? std::min(max_kv, window + max_q - 1) : max_kv;
  auto nc_of = [](int64_t rows) { return rows <= 16 ? 1 : 2; };
  if (max_q * g <= cap) {
    p.nc = nc_of(max_q * g);
  } else {
    p.tile = true;
    // tokens that fill every sequence to max_q leave none for the few-row kernel
    if (g <= cap && t != n_seqs * max_q) p.nc = nc_of(g);
  }
  p.few_rows = 16 * p.nc;
  p.ok = true;
  size_t at = 0;
  if (p.nc) {
    const int64_t tiles = span / kAttnFewKeys + 10;
    const int64_t units = times(times(n_seqs, hk), tiles);
    p.ok = p.ok && units < limit;
    // two resident workgroups a compute unit, one at 256 values a head (their LDS; four at 64 values
    // would fit, but the pieces cost more than they hide: 16 x 5 drafted tokens 34 against 28 us)
    p.nw_few = (int)std::min<int64_t>(d == 256 ? 256 : 512, units);
    p.cap_few = 16 * p.nc;
    p.part_floats = p.cap_few * (d + 2);
    p.join_few = max_kv > kAttnFewKeys;  // a span inside one tile is never cut
  }
  if (p.tile) {
    const int64_t slots = 256;  // resident workgroups
    const int64_t full = t * g / bm;
    const int64_t seqs = std::min<int64_t>(n_seqs, t * g / (p.few_rows + 1));
    const int64_t tiles = full + seqs;
    p.plan_tiles = (int)tiles;
    const int64_t grid = times(tiles, hk);
    p.ok = p.ok && grid < limit;
    // whole items to workgroups where that fills them: two items or more each, or a last round that
    // is four fifths full (4096 tokens, 28 heads on 4: 448 items 151 us, cut into runs 181; 1000 tokens
    // at 32767, 32 heads on 8: 128 items would leave half the chip idle)
    const int64_t items = times(full, hk), rounds = (items + slots - 1) / slots;
    if (items >= 2 * slots || (items > 0 && 5 * items >= 4 * slots * rounds) || tiles + n_seqs > 4096) {
      p.items_tile = (int)std::min(grid, limit - 1);
    } else {
      p.ok = p.ok && times(grid, span / kAttnTileKeys + 16) < limit;
      p.nw_tile = (int)slots;
      p.join_tile = max_kv > kAttnTileKeys;
    }
  }
  auto take = [&](size_t n) {
    const size_t o = at;
    at = (at + n + 255) / 256 * 256;
    return o;
  };
  take((size_t)(p.nw_few + p.nw_tile) * sizeof(AttnRecord));
  p.part_off = take((size_t)2 * p.nw_few * p.part_floats * 4);
  p.part_tile_off = take((size_t)2 * p.nw_tile * bm * (d + 2) * 4);
  p.bytes = at;
  return p;
}

AttnArgs attn_record_kind(AttnArgs a) {
  a.few_by_item = (int64_t)a.n_seqs * a.hk <= a.nw_few;
  a.tile_by_item = (int64_t)a.plan_tiles * a.hk <= a.nw_tile;
  return a;
}

hipError_t launch_attn_tile(const AttnArgs& args, int dt, int d, hipStream_t s) {
  const AttnArgs a = attn_record_kind(args);
  if (dt == DT_BF16) return d == 64 ? tile<BF16, 64>(a, s) : d == 128 ? tile<BF16, 128>(a, s) : tile<BF16, 256>(a, s);
  return d == 64 ? tile<F16, 64>(a, s) : d == 128 ? tile<F16, 128>(a, s) : tile<F16, 256>(a, s);
}
hipError_t launch_attn_join(const AttnArgs& args, int dt, int d, hipStream_t s) {
  const AttnArgs a = attn_record_kind(args);
  if (dt == DT_BF16) return d == 64 ? join<BF16, 64>(a, s) : d == 128 ? join<BF16, 128>(a, s) : join<BF16, 256>(a, s);
  return d == 64 ? join<F16, 64>(a, s) : d == 128 ? join<F16, 128>(a, s) : join<F16, 256>(a, s);
}

}  // namespace ql
