// The tables of a batch from its token counts: lengths, pages, positions and slots of a paged cache's next
// step.
//
// Prefix sums over the sequences (new tokens, pages given back, pages needed) place everything: token i of
// sequence s is row cu_q[s] + i, page j that s gives back is entry F + back_before[s] + j of the free
// list, page j that it takes entry F + back - 1 - (need_before[s] + j).  All of it is a few words a
// sequence and 16 bytes a token, so what bounds it is latency: one workgroup decides and lays out the
// sequences, and the tokens follow in the same workgroup where they are few, else in a second launch over
// all of the chip.  Pages are moved one a thread, whose sequence it finds in the prefix (a wave taking sequence
// after sequence: 300 of them, 100 with chunks, 14 us against 12).
//
// Measured (in a graph): 64 single tokens 5 us, 300 sequences, 20 of which give back all their pages, and 13000
// tokens 15.
#include "attn_launch.hpp"
#include "device_common.hpp"

namespace ql {
namespace {

// The exclusive prefixes of x and y over the workgroup's threads; sh holds a pair per wave.  The sums are
// within 2^31: the batch has been found to fit.
struct Pair {
  int x, y;
};
template <int kWaves> __device__ __forceinline__ Pair block_scan2(Pair v, Pair* sh, Pair& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  Pair p = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const Pair q = {__shfl_up(p.x, d), __shfl_up(p.y, d)};
    if (lane >= d) p.x += q.x, p.y += q.y;
  }
  __syncthreads();
  if (lane == 63) sh[wave] = p;
  __syncthreads();
  Pair before = {0, 0};
  total = {0, 0};
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const Pair q = sh[w];
    if (w < wave) before.x += q.x, before.y += q.y;
    total.x += q.x, total.y += q.y;
  }
  return {before.x + p.x - v.x, before.y + p.y - v.y};
}
__device__ __forceinline__ int64_t wave_sum(int64_t x) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) x += __shfl_xor((long long)x, d);
  return x;
}

// What sequence s asks for: its length before, new tokens, pages that go back, held and needed; and
// whether its lengths lie in a row of the table.
struct Ask {
  int old, now, back, have, need;
  bool fits;
};
__device__ __forceinline__ Ask ask(const ExtendArgs& a, int s) {
  const int64_t c = a.counts[s], len = a.lens[s], most = a.max_pages * a.page_size;
  Ask k;
  k.fits = len >= 0 && len <= most && (c < 0 || len + c <= most);
  const int l = k.fits ? (int)len : 0;
  k.old = c < 0 ? 0 : l;
  k.now = k.fits && c > 0 ? (int)c : 0;
  auto pages = [&](int n) { return n > 0 ? (int)a.page_div.div((uint32_t)(n - 1)) + 1 : 0; };
  k.have = pages(k.old);
  k.back = a.free_pages ? pages(l) - k.have : 0;
  k.need = a.free_pages ? pages(k.old + k.now) - k.have : 0;
  return k;
}

// The last of n ascending numbers that is at most i (the first is).
__device__ __forceinline__ int last_at_most(const int* x, int n, int64_t i) {
  int b = 0, e = n;
  while (e - b > 1) {
    const int m = (b + e) / 2;
    if (x[m] <= i) b = m; else e = m;
  }
  return b;
}

// Row i of positions and slots, cu and lens the prefix and the lengths after of the sequences [0, n).
__device__ __forceinline__ void token(const ExtendArgs& a, int64_t i, int total, const int* cu, const int* lens) {
  int64_t pos = 0, slot = -1;
  if (i < total) {
    const int b = last_at_most(cu, a.n_seqs, i);
    pos = (int64_t)lens[b] - cu[b + 1] + i;  // its length before, and the tokens before this one
    const int64_t page = a.page_div.div((uint32_t)pos);
    slot = (int64_t)a.table[b * a.table_stride + page] * a.page_size + (pos - page * a.page_size);
  }
  a.positions[i] = pos;
  a.slots[i] = slot;
}

// Sequences whose prefix and lengths are searched in LDS.
constexpr int kHeld = 4096;

// THREADS: one workgroup.  Where the sequences are at most as many as the threads each thread asks once.
template <int THREADS> __global__ __launch_bounds__(THREADS) void extend_kernel(const ExtendArgs a, int with_tokens) {
  constexpr int kWaves = THREADS / 64;
  __shared__ Pair sh[kWaves];
  __shared__ int64_t sums[kWaves][3];
  __shared__ int scu[THREADS + 1], slen[THREADS], spre[THREADS], shave[THREADS];
  const int tid = threadIdx.x;
  const bool list = a.free_pages != nullptr, once = a.n_seqs <= THREADS;
  const int64_t f0 = list ? a.free_count[0] : 0;
  // what the whole batch asks for
  int64_t tok = 0, back = 0, need = 0;
  bool fits = true;
  Ask mine = {};
  mine.fits = true;
  for (int s = tid; s < a.n_seqs; s += THREADS) {
    mine = ask(a, s);
    tok += mine.now, back += mine.back, need += mine.need;
    fits &= mine.fits;
  }
  tok = wave_sum(tok), back = wave_sum(back), need = wave_sum(need);
  if ((tid & 63) == 0) sums[tid >> 6][0] = tok, sums[tid >> 6][1] = back, sums[tid >> 6][2] = need;
  const bool misfit = __syncthreads_or(!fits) != 0;
  tok = back = need = 0;
  for (int w = 0; w < kWaves; ++w) tok += sums[w][0], back += sums[w][1], need += sums[w][2];
  int why = (tok > a.rows ? 1 : 0) | (misfit ? 4 : 0);
  if (list) why |= (need > f0 + back ? 2 : 0) | (f0 < 0 || f0 + back > a.free_cap ? 8 : 0);
  auto asked = [&](int s) {
    if (once) return mine;
    return ask(a, s);
  };
  // pages that come back
  if (why == 0 && back > 0) {
    int before = (int)f0;
    for (int s0 = 0; s0 < a.n_seqs; s0 += THREADS) {
      const int s = s0 + tid;
      Pair v = {0, 0}, total;
      if (s < a.n_seqs) v.x = asked(s).back;
      spre[tid] = block_scan2<kWaves>(v, sh, total).x;
      __syncthreads();
      for (int i = tid; i < total.x; i += THREADS) {
        const int b = last_at_most(spre, min(THREADS, a.n_seqs - s0), i);
        a.free_pages[before + i] = a.table[(s0 + b) * a.table_stride + i - spre[b]];
      }
      __syncthreads();
      before += total.x;
    }
  }
  // lengths, prefix and pages that are taken
  int row = 0, taken = 0;
  for (int s0 = 0; s0 < a.n_seqs; s0 += THREADS) {
    const int s = s0 + tid;
    Pair v = {0, 0}, total;
    Ask k = {};
    if (s < a.n_seqs && why == 0) {
      k = asked(s);
      v = {k.now, k.need};
    }
    const Pair e = block_scan2<kWaves>(v, sh, total);
    if (s < a.n_seqs) {
      const int len = why == 0 ? k.old + k.now : a.lens[s];
      a.cu_q[s] = row + e.x;
      a.lens_out[s] = len;
      if (once) scu[tid] = row + e.x, slen[tid] = len;
    }
    if (total.y > 0) {  // uniform
      spre[tid] = e.y, shave[tid] = k.have;
      __syncthreads();
      for (int i = tid; i < total.y; i += THREADS) {
        const int b = last_at_most(spre, min(THREADS, a.n_seqs - s0), i);
        a.table[(s0 + b) * a.table_stride + shave[b] + i - spre[b]] = a.free_pages[(int)(f0 + back) - 1 - taken - i];
      }
      __syncthreads();
    }
    row += total.x, taken += total.y;
  }
  if (tid == 0) {
    const int left = (int)(why ? f0 : f0 + back - need);
    a.cu_q[a.n_seqs] = row;
    if (once) scu[a.n_seqs] = row;
    if (list) a.free_count_out[0] = left;
    a.info[0] = row;
    a.info[1] = taken;
    a.info[2] = why;
    a.info[3] = left;
  }
  if (with_tokens) {
    __syncthreads();
    for (int64_t i = tid; i < a.rows; i += THREADS)
      if (once)
        token(a, i, row, scu, slen);
      else
        token(a, i, row, a.cu_q, a.lens_out);
  }
}

__global__ __launch_bounds__(1024) void extend_tokens_kernel(const ExtendArgs a) {
  __shared__ int scu[kHeld + 1], slen[kHeld];
  const int64_t i = (int64_t)blockIdx.x * 1024 + threadIdx.x;
  if (a.n_seqs <= kHeld) {
    for (int s = threadIdx.x; s <= a.n_seqs; s += 1024) {
      scu[s] = a.cu_q[s];
      if (s < a.n_seqs) slen[s] = a.lens_out[s];
    }
    __syncthreads();
    if (i < a.rows) token(a, i, scu[a.n_seqs], scu, slen);
  } else if (i < a.rows) {
    token(a, i, a.cu_q[a.n_seqs], a.cu_q, a.lens_out);
  }
}

}  // namespace

hipError_t launch_kv_extend(const ExtendArgs& a, hipStream_t s) {
  // small steps in one launch, by as few waves as hold a sequence a thread (their barriers cost most)
  const bool one = a.rows <= 4096;
  if (a.n_seqs <= 256 && (a.rows <= 1024 || !one))
    extend_kernel<256><<<1, 256, 0, s>>>(a, one ? 1 : 0);
  else
    extend_kernel<1024><<<1, 1024, 0, s>>>(a, one ? 1 : 0);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || one) return e;
  extend_tokens_kernel<<<(unsigned)((a.rows + 1023) / 1024), 1024, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace ql
