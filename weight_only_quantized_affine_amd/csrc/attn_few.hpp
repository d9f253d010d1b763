// Shared by the few-row kernels (attn_few.hip, attn_few4.hip): which run of units a workgroup takes, and
// the end of an item.
#pragma once
#include "attn_common.hpp"

namespace ql {

// A workgroup's run of units [u0, u1) of W, cut between nw workgroups, this one the w-th; the sequence s
// of u0 and that sequence's first unit; item_units before each item's first tile; its record.
struct FewRun {
  int u0, u1, s, base, W, nw, w, item_units;
  AttnRecord* rec;
};
// False where the workgroup has nothing to do.  Units are tiles of KEYS positions; an item counts ITEM units for
// its start and end where a workgroup has LONG tiles or more; 256 threads.
template <int KEYS, int ITEM, int LONG>
__device__ __forceinline__ bool few_run(const AttnArgs& a, int* ssh, int* sfound, FewRun& run) {
  const int tid = threadIdx.x;
  // This workgroup's run of units: all sequences' tiles, head by head, end to end.
  // Short runs are better off with the tiles spread evenly, without units for start and end.
  int& item_units = run.item_units;
  item_units = 0;
  auto cost = [&](int s) -> int {
    if (s >= a.n_seqs) return 0;
    const AttnSeq q = attn_seq(a, s);
    if (q.nq < 1 || !attn_is_few(a, q.nq)) return 0;
    int lo, hi, first;
    attn_span(a, q, 0, q.nq - 1, lo, hi);
    return (item_units + attn_tiles<KEYS>(lo, hi, first)) * a.hk;
  };
  int W = 0, mine = 0, before = 0;  // the thread's own sequence tid: its units and those before it
  auto measure = [&] {
    W = 0;
    for (int s0 = 0; s0 < a.n_seqs; s0 += 256) {
      int total;
      const int c = cost(s0 + tid), e = block_scan<4>(c, ssh, total);
      if (s0 == 0) mine = c, before = e;
      W += total;
    }
  };
  measure();
  if (W >= LONG * a.nw_few) {
    item_units = ITEM;
    measure();
  }
  const int nw = min(a.nw_few, W);
  // workgroups of one XCD (every 8th) take neighbouring runs (one sequence of 131071: 102 -> 97 us)
  const int w = a.nw_few % 8 == 0 ? (blockIdx.x & 7) * (a.nw_few >> 3) + (blockIdx.x >> 3) : blockIdx.x;
  run.rec = a.rec + w;
  if (a.few_by_item) {  // the first workgroup clears the records of sequences that are not taken here
    if (blockIdx.x == 0)
      for (int i = tid; i < a.n_seqs; i += 256)
        if (cost(i) == 0)
          for (int h = 0; h < a.hk; ++h) a.rec[i * a.hk + h].pieces = 0;
  } else if (w >= nw && tid == 0) {
    run.rec->pieces = 0;
  }
  if (w >= nw) return false;
  const int u0 = attn_cut(w, nw, W), u1 = attn_cut(w + 1, nw, W);
  // sequence of unit u0 and its first unit; beyond 256 sequences the scan is run again
  for (int s0 = 0, sum = 0; s0 < a.n_seqs && sum <= u0; s0 += 256) {
    if (s0 > 0) {
      int total;
      mine = cost(s0 + tid);
      before = sum + block_scan<4>(mine, ssh, total);
      sum += total;
    } else if (a.n_seqs > 256) {
      int total;
      block_scan<4>(mine, ssh, total);
      sum += total;
    }
    if (before <= u0 && u0 < before + mine) sfound[0] = s0 + tid, sfound[1] = before;
  }
  __syncthreads();
  run.u0 = u0, run.u1 = u1, run.s = sfound[0], run.base = sfound[1], run.W = W, run.nw = nw, run.w = w;
  return true;
}

// The end of an item, by thread tid of 256: joins the waves' sums (m, l, o of the wave's columns) in LDS, wave_bytes apart from
// sm, and stores the rows, or the piece where the item is not `whole`; `starts`: the piece is its first.
template <int D, int NC, class Store>
__device__ __forceinline__ void few_finish(const AttnArgs& a, int tid, uint8_t* sm, int wave_bytes, float (*sml)[16 * NC][2],
                                           f32x4_t (*o)[D / 16], const float* m, float* l, int w, const AttnSeq& q,
                                           int head, int rows, bool starts, bool whole, Store&& store) {
  constexpr int ND = D / 16;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int g = lane >> 4, col = lane & 15;
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    l[n] = join32(join16(l[n], SumF()), SumF());
    if (g == 0) sml[wave][16 * n + col][0] = m[n], sml[wave][16 * n + col][1] = l[n];
  }
  __syncthreads();
  const int slot = starts ? 2 * w + 1 : 2 * w;
  float* part = a.part + (int64_t)slot * a.part_floats;
#pragma unroll
  for (int n = 0; n < NC; ++n) {
    float mt = kNegInf;
#pragma unroll
    for (int v = 0; v < 4; ++v) mt = fmaxf(mt, sml[v][16 * n + col][0]);
    const float f = join_factor(m[n], l[n], mt);
    float* so = (float*)(sm + wave * wave_bytes);  // [16][D], 4-value chunks placed by the row
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      f32x4_t x = o[n][d];
      for (int r = 0; r < 4; ++r) x[r] = f == 0.f ? 0.f : x[r] * f;
      *(f32x4_t*)(so + col * D + 4 * ((4 * d + g) ^ col)) = x;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16 * (D / 4) / 256; ++i) {
      const int e = i * 256 + tid, r = e / (D / 4), c = e % (D / 4), row = 16 * n + r;
      f32x4_t x = {0, 0, 0, 0};
      float mr = kNegInf, lr = 0.f;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        x += *(const f32x4_t*)((const float*)(sm + v * wave_bytes) + r * D + 4 * (c ^ r));
        mr = fmaxf(mr, sml[v][row][0]);
      }
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const float mv = sml[v][row][0];
        const float lv = sml[v][row][1];
        lr += lv == 0.f ? 0.f : lv * join_factor(mv, lv, mr);
      }
      if (row < rows) {
        if (whole) {
          const int tok = (int)a.g_div.div((uint32_t)row);
          const int hq = head * a.g + row - tok * a.g;
          const float inv = attn_scale(a.sinks, hq, mr, lr);
          uint8_t* op = a.out + ((int64_t)(q.q0 + tok) * a.out_ts + (int64_t)hq * a.out_hs) + c * 8;
          store(op, x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv);
        } else {
          if (c == 0) part[row] = mr, part[16 * NC + row] = lr;
          *(f32x4_t*)(part + 32 * NC + row * D + c * 4) = x;
        }
      }
    }
    __syncthreads();
  }
}

// The record of an item whose first piece this workgroup holds; `end`: the unit after its last tile.
__device__ __forceinline__ void few_record(const AttnArgs& a, FewRun& run, int s, int head, int q0, int rows, int end,
                                           bool whole, bool& recorded) {
  if (whole && !a.few_by_item) return;
  recorded = true;
  if (threadIdx.x == 0) {
    AttnRecord r = {};
    if (a.few_by_item) run.rec = a.rec + s * a.hk + head;
    r.pieces = whole ? 0 : attn_last(end, run.nw, run.W) - run.w + 1;
    r.w = run.w;
    r.q0 = q0;
    r.row0 = 0;
    r.rows = rows;
    r.head = head;
    *run.rec = r;
  }
}

}  // namespace ql
