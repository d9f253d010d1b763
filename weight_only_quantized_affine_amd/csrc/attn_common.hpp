// Shared parts of the paged attention kernels (attn_few.hip, attn_tile.hip): the split of the work
// over workgroups, the copy of cache rows into LDS and the register tiles of the two products.
//
// Mathematics: the softmax with a running maximum (Milakov and Gimelshein 2018).  For one query row
// with scores s_j (log2 units: scale * log2(e) * q.k_j) the kernels hold M (a reference not below the
// maximum by more than kLazy), l = sum 2^(s_j - M) and O = sum 2^(s_j - M) v_j in fp32, the weights
// 2^(s_j - M) rounded once to the cache's 16-bit type (the matrix cores' operand) in the sum l as in O,
// so that the normalized weights sum to one; pieces of a row join as
//   sum_p 2^(M_p - M) O_p / sum_p 2^(M_p - M) l_p.
// Both products run transposed, S^T = K Q^T and O^T = V^T P^T, so that a lane holds one query column:
// the maximum, the sum and the rescaling of a row are per-lane scalars, and the lane's scores are
// already the P^T operand of the second product under a permutation of the keys that the V^T reads
// follow.
#pragma once
#include "head_common.hpp"

namespace ql {

typedef __attribute__((address_space(3))) void at_lds_void;
typedef __attribute__((ext_vector_type(4))) short s16x4_t;
typedef __attribute__((address_space(3))) s16x4_t at_lds_s16x4;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_inff();
// The reference M is raised only when a tile's maximum passes it by more than 2^8: P stays below
// 256 (exact range of both 16-bit types), and most tiles skip the rescaling of O.
constexpr float kLazy = 8.0f;

// 16-bit products with fp32 accumulation.
__device__ __forceinline__ f32x4_t mfma16(BF16, u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                 0, 0, 0);
}
__device__ __forceinline__ f32x4_t mfma16(F16, u32x4_t a, u32x4_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                0, 0);
}
__device__ __forceinline__ f32x16_t mfma32(BF16, u32x4_t a, u32x4_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                 0, 0, 0);
}
__device__ __forceinline__ f32x16_t mfma32(F16, u32x4_t a, u32x4_t b, f32x16_t c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                0, 0);
}
// acc plus the two 16-bit values of a word.
__device__ __forceinline__ float add2(BF16, uint32_t w, float acc) { return dot2(BF16{}, w, 0x3f803f80u, acc); }
__device__ __forceinline__ float add2(F16, uint32_t w, float acc) { return dot2(F16{}, w, 0x3c003c00u, acc); }
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// x joined with its value in the other half (lanes +-32) or the other 16 of each 32 lanes.
template <typename F> __device__ __forceinline__ float join32(float x, F f) {
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return f(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
template <typename F> __device__ __forceinline__ float join16(float x, F f) {
  const uint32_t u = __float_as_uint(x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return f(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
// The largest of three, ignoring NaN (fmaxf would first quiet each operand).  The compiler puts no
// wait between a matrix product and an inline instruction that reads its result: a chain over
// scores begins with fmaxf of a value of each product, which is waited for, and every max3 takes
// the chain's last result.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
  return r;
}
struct MaxF {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct SumF {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};

// Factor of a piece with reference m and sum l when pieces join under the reference mt.  A piece
// that saw nothing has m = -inf and l = 0; one whose every score is NaN has m = -inf and l = NaN,
// and keeps its NaN.
__device__ __forceinline__ float join_factor(float m, float l, float mt) {
  return m == kNegInf ? (l == 0.f ? 0.f : 1.f) : exp2_fast(m - mt);
}

// What a row's O is multiplied by: 1 / (l + 2^(sink - m)).  A sink of -infinity is no term, one of
// +infinity leaves nothing for the keys (f = 0), and a row that saw nothing (m = -inf, l = 0) is zero
// with any sink: neither infinity's difference from the reference is used.
__device__ __forceinline__ float attn_scale(const float* sinks, int head, float m, float l) {
  float f = 1.f, z = l;
  if (sinks) {
    const float sink = sinks[head] * kLog2e, mn = fmaxf(m, sink);
    if (sink != kNegInf) f = join_factor(m, l, mn), z = l * f + exp2_fast(sink - mn);
  }
  return f == 0.f || z == 0.f ? 0.f : f / z;
}

// A V row that some query rows of a tile see and others do not may hold infinities or NaN, and zero
// times those is not zero.  Tiles with such rows are checked; if one holds any, its non-finite
// values are added one key at a time to the rows that see them, and the product takes zeros there.
template <typename T> struct Bits16;
template <> struct Bits16<BF16> {
  static constexpr uint32_t expo = 0x7f80u, step = 0x0080u;
};
template <> struct Bits16<F16> {
  static constexpr uint32_t expo = 0x7c00u, step = 0x0400u;
};
// Bit 15 of a half is set when that half of w is infinite or NaN.
template <typename T> __device__ __forceinline__ uint32_t nonfinite2(uint32_t w) {
  return (w & (Bits16<T>::expo * 0x10001u)) + Bits16<T>::step * 0x10001u;
}
// The word with its infinite and NaN halves as zero.
template <typename T> __device__ __forceinline__ uint32_t finite2(uint32_t w) {
  const uint32_t nf = (nonfinite2<T>(w) & 0x80008000u) >> 15;  // 1 in a half that is not finite
  return w & ~(nf * 0xffffu);
}
// The halves of w that are infinite or NaN, as floats, where `on`; zero otherwise.
template <typename T> __device__ __forceinline__ void only_nonfinite(uint32_t w, bool on, float& a, float& b) {
  const uint32_t nf = nonfinite2<T>(w);
  a = on && (nf & 0x8000u) ? param_to_f32<T>(w & 0xffffu) : 0.f;
  b = on && (nf & 0x80000000u) ? param_to_f32<T>(w >> 16) : 0.f;
}

// Position of 16-byte chunk c of row r in a tile of rows of D values.  The LDS has 256 bytes of banks:
// K is read 16 rows at one chunk per pass, V (transposing, 32 bytes of a row) either 8 rows at one
// chunk pair or 4 rows at two neighbouring pairs; the positions of each set are distinct modulo 256
// bytes.  (V's pairs by r & 7 alone: the tile kernel's reads met banks twice, a third of its LDS
// cycles.)
template <int D> __device__ __forceinline__ int swz_k(int r) { return D >= 128 ? (r & 15) : ((r >> 1) & 7); }
template <int D> __device__ __forceinline__ int swz_v(int r) {
  if (D >= 128) return ((r & 3) << 2) | ((r & 4) >> 1);
  return ((r & 2) << 1) | ((r & 4) >> 1);
}

// One sequence: its query rows [q0, q0 + nq) and cached length kv, kept inside the arrays whatever
// the device values say.
struct AttnSeq {
  int q0, nq, kv;
};
__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs& a, int s) {
  AttnSeq r;
  const int t = (int)a.t;
  const int c0 = a.cu_q[s], c1 = a.cu_q[s + 1];
  r.q0 = min(max(c0, 0), t);
  r.nq = min(min(max(c1, r.q0), t) - r.q0, a.max_q);
  r.kv = min(max(a.kv_lens[s], 0), a.max_kv);
  return r;
}
// Whether the few-row kernel takes a sequence (the tile kernel takes the others with nq >= 1).
__device__ __forceinline__ bool attn_is_few(const AttnArgs& a, int nq) { return nq * a.g <= a.few_rows; }

// Cached positions [lo, hi) that the queries i0 .. i1 of a sequence may see.
__device__ __forceinline__ void attn_span(const AttnArgs& a, const AttnSeq& q, int i0, int i1, int& lo, int& hi) {
  hi = max(0, q.kv - q.nq + i1 + 1);
  const int first = q.kv - q.nq + i0 + 1 - a.window;
  lo = a.window > 0 ? min(max(0, first), hi) : 0;
}
// Tiles of N positions that cover [lo, hi): first tile and count (at least one: a row that sees
// nothing is still written).
template <int N> __device__ __forceinline__ int attn_tiles(int lo, int hi, int& first) {
  first = lo / N;
  return max(1, (hi + N - 1) / N - first);
}

// Rows that are not to be seen are copied from here: their V must be zero, since zero times an
// infinity or a NaN left in an unused slot would not be.
__device__ __attribute__((aligned(16))) static uint32_t kZeroRow[128] = {};

__device__ __forceinline__ uint32_t lds_at(const uint8_t* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(at_lds_void*)p);
}
// The copies set m0, which the compiler keeps for itself: it never holds a value there over other
// instructions, and the clobber list keeps it from placing its own use of m0 around them.  It warns
// of the name in the list.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// Starts a copy of 16 bytes a lane into LDS, lane l's from src to dst + 16 l (dst is uniform).
// Written as an instruction because the compiler, which cannot tell the stages apart, would wait for
// every copy in flight at each LDS read; the kernels wait by count (attn_wait_vm) for the stage they
// read.  The copy writes no register; the wait state between m0 and its use is in the text.
//
// NT: the non-temporal policy, for rows that no other workgroup reads (few-row kernel: one sequence
// of 131071 114 -> 102 us, 64 ragged ones 163 -> 147 us; the tile kernel's row tiles share their
// keys, and lose 10 % by it).
template <bool NT> __device__ __forceinline__ void copy16(const uint8_t* src, uint8_t* dst) {
  if constexpr (NT)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off nt"
                 :
                 : "s"(lds_at(dst)), "v"(src)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :
                 : "s"(lds_at(dst)), "v"(src)
                 : "memory", "m0");
}
__device__ __forceinline__ int64_t uniform64(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x), hi = __builtin_amdgcn_readfirstlane((uint32_t)(x >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}
// Two of them, 1 KB apart in LDS, from a uniform base plus the lane's offsets (off1 is not used for
// one).  A scalar written by a vector instruction needs 5 wait states before a load takes it.
template <bool NT, bool TWO>
__device__ __forceinline__ void copy16_from(int64_t base, uint32_t off0, uint32_t off1, uint8_t* dst) {
  if constexpr (TWO && NT)
    asm volatile(
        "s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %3 nt\n\t"
        "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3 nt"
        :
        : "s"(lds_at(dst)), "v"(off0), "v"(off1), "s"(base)
        : "memory", "m0", "scc");
  else if constexpr (TWO)
    asm volatile(
        "s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %3\n\t"
        "s_add_u32 m0, m0, 0x400\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3"
        :
        : "s"(lds_at(dst)), "v"(off0), "v"(off1), "s"(base)
        : "memory", "m0", "scc");
  else if constexpr (NT)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2 nt"
                 :
                 : "s"(lds_at(dst)), "v"(off0), "s"(base)
                 : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds_at(dst)), "v"(off0), "s"(base)
                 : "memory", "m0");
}
#pragma clang diagnostic pop

// The cache rows of a tile that one wave copies, U runs of R rows (positions base .. base + U R; R
// divides 16 and base is a multiple of R), K and V alike; tiles are STEP positions apart.
//
// Where pages are multiples of 16 slots (a.page16) a run lies in one page: the ids of the next 64 / U
// tiles are read at once, one per lane, and the copies take a scalar base and lane offsets that
// never change.  (One scalar load per tile instead shares its counter with the LDS reads: every
// read after it waits for it.)  Else, and for runs that end inside, row r is looked up by the lanes
// with lane % (U R) == r, and handed to the lanes that copy it.
template <int D, int R, int U, int STEP, bool NT> struct TileCopy {
  static constexpr int CH = D / 8;      // 16-byte chunks of a row
  static constexpr int RPI = 64 / CH;   // rows of an instruction (1 KB)
  static constexpr int NI = R / RPI;    // instructions of a run
  static constexpr int ROWS = U * R, BLOCK = 64 / U;
  struct Place {       // where a tile's rows lie
    int64_t row;       // the lane's row, -1 for a row that is not to be seen
    int64_t at[U];     // uniform: the runs, -1: by rows
  };
  uint32_t off_k[NI], off_v[NI];  // lane offsets within a run
  int pos, id;                    // the lane's row: position, page (a.page16: unused)
  int ids, block;                 // a.page16: pages of the runs of BLOCK tiles, position of the first
  int base, uid[U];               // uniform: first position, pages of the runs
  Place now;
  uint32_t seen;                  // bit r: row r is to be seen

  // row0: place of the first row in the tile, whose swizzle the chunks follow.
  __device__ __forceinline__ void init(const AttnArgs& a, int row0, int lane) {
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int r = i * RPI + lane / CH, c = lane % CH;
      off_k[i] = (uint32_t)r * (uint32_t)a.token_stride + (c ^ swz_k<D>(row0 + r)) * 16;
      off_v[i] = (uint32_t)r * (uint32_t)a.token_stride + (c ^ swz_v<D>(row0 + r)) * 16;
    }
  }
  // Reads the page ids of the rows of the tile at `first` that lie in [lo, hi); `begins` at the
  // first of a sequence's tiles.
  __device__ __forceinline__ void lookup(const AttnArgs& a, const int32_t* table, int first, int lo, int hi, int lane,
                                         bool begins) {
    base = first;
    pos = first + (lane & (ROWS - 1));
    if (a.page16) {
      if (begins || first - block >= BLOCK * STEP) {
        block = first;
        const int p = first + (lane % BLOCK) * STEP + (lane / BLOCK) * R;
        ids = -1;
        if (p + R > lo && p < hi) ids = table[a.page_div.div((uint32_t)p)];
        asm volatile("" : "+v"(ids));  // the wait for the load is here
      }
      const int i = (first - block) / STEP;
#pragma unroll
      for (int u = 0; u < U; ++u) uid[u] = __builtin_amdgcn_readlane(ids, i + u * BLOCK);
    } else {
      id = -1;
      if (pos >= lo && pos < hi) id = table[a.page_div.div((uint32_t)pos)];
    }
  }
  // Turns the page ids into places; sets seen.
  __device__ __forceinline__ void resolve(const AttnArgs& a, int lo, int hi, int lane) {
    constexpr uint32_t kAll = (uint32_t)((1ull << ROWS) - 1);
    bool by_rows = true;
    if (a.page16) {
      by_rows = false;
      seen = kAll;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int p = base + R * u;
        const bool known = (uint32_t)uid[u] < (uint32_t)a.n_pages;
        now.at[u] = known ? (int64_t)uid[u] * a.page_stride +
                                (int64_t)(p - (int)a.page_div.div((uint32_t)p) * a.page_size) * a.token_stride
                          : -1;
        by_rows |= !(known && p >= lo && p + R <= hi);
      }
      if (by_rows) {
        int64_t b = now.at[0];
        if (U > 1 && (lane & (ROWS - 1)) >= R) b = now.at[U - 1];
        now.row = b >= 0 && pos >= lo && pos < hi ? b + (int64_t)(lane & (R - 1)) * a.token_stride : -1;
      }
    } else {
      const uint32_t in = (uint32_t)pos - a.page_div.div((uint32_t)pos) * (uint32_t)a.page_size;
      now.row = id >= 0 && id < a.n_pages ? (int64_t)id * a.page_stride + (int64_t)in * a.token_stride : -1;
    }
    if (by_rows) {
      seen = (uint32_t)__ballot(now.row >= 0) & kAll;
      now.at[0] = -1;
    }
    static_assert(U <= 2 && ROWS <= 32, "places of one or two runs");
  }
  // Starts the copies of the rows into LDS at dst (rows back to back, chunks placed by the swizzle).
  template <bool IS_V>
  __device__ __forceinline__ void copy(const Place& pl, const uint8_t* head, uint8_t* dst, int row0, int lane) const {
    if (pl.at[0] >= 0) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t b = uniform64((int64_t)(uintptr_t)head + pl.at[u]);
#pragma unroll
        for (int i = 0; i < NI; i += 2)
          copy16_from<NT, (NI > 1)>(b, IS_V ? off_v[i] : off_k[i], IS_V ? off_v[(i + 1) % NI] : off_k[(i + 1) % NI],
                                    dst + (u * NI + i) * 1024);
      }
    } else {
      asm volatile("" : "+v"(lane));  // the lane's places are worked out here, not kept in registers
#pragma unroll
      for (int i = 0; i < U * NI; ++i) {
        const int r = i * RPI + lane / CH;
        const int lo = __shfl((int)pl.row, r), hi = __shfl((int)(pl.row >> 32), r);
        const int64_t o = ((int64_t)hi << 32) | (uint32_t)lo;
        const int c = (lane % CH) ^ (IS_V ? swz_v<D>(row0 + r) : swz_k<D>(row0 + r));
        copy16<NT>((hi < 0 ? (const uint8_t*)kZeroRow : head + o) + c * 16, dst + i * 1024);
      }
    }
  }
};

__device__ __forceinline__ s16x4_t read_tr(const uint8_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((at_lds_s16x4*)p);
}
// s_waitcnt with only the vector-memory count.
template <int N> __device__ __forceinline__ void attn_wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
  asm volatile("" ::: "memory");
}

// The wave's LDS reads so far are done: copies over what they read may start.
__device__ __forceinline__ void attn_wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// Workgroup barrier after this wave's LDS accesses (not its copies: those are waited for by count).
__device__ __forceinline__ void attn_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// Sum over the workgroup's threads, and the exclusive prefix; sh holds an int per wave.
template <int WAVES> __device__ __forceinline__ int block_scan(int v, int* sh, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 63) sh[wave] = x;
  __syncthreads();
  int before = 0, sum = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    const int s = sh[w];
    before += w < wave ? s : 0;
    sum += s;
  }
  total = sum;
  return before + x - v;
}

// A split item: the workgroup that began it writes where its rows and pieces are.  Records are kept
// by item where there are at most as many as workgroups (few records to look through), else by
// the workgroup that began the item, which begins at most one that it does not finish.
struct AttnRecord {
  int32_t pieces;  // 0: nothing to join
  int32_t q0;      // first query token of the sequence
  int32_t row0;    // first row of the item among the sequence's nq * g rows
  int32_t rows;    // rows of the item
  int32_t head;    // kv head
  int32_t w;       // the workgroup that began it
  int32_t pad_[2];
};
// Range of units [u0, u1) of workgroup w of nw over W units, and the last workgroup that holds a
// unit below `end` (nw <= W: none is empty).
__device__ __forceinline__ int attn_cut(int w, int nw, int W) { return (int)((int64_t)w * W / nw); }
__device__ __forceinline__ int attn_last(int end, int nw, int W) { return (int)(((int64_t)end * nw - 1) / W); }

// Stores 4 neighbouring output values of a row.
template <typename T> __device__ __forceinline__ void store4(T t, void* p, float a, float b, float c, float d) {
  *(u32x2_t*)p = u32x2_t{pack2(t, a, b), pack2(t, c, d)};
}

}  // namespace ql
