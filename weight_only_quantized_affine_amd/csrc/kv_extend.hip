// The tables of a batch from its token counts: lengths, pages, positions and slots of a paged cache's next
// step.
//
// Prefix sums over the sequences (new tokens, pages given back, pages needed) place everything: token i of
// sequence s is row cu_q[s] + i, page j that s gives back is entry F + back_before[s] + j of the free
// list, page j that it takes entry F + back - 1 - (need_before[s] + j).  All of it is a few words a
// sequence and 16 bytes a token, so what bounds it is latency: one workgroup decides and lays out the
// sequences, and the tokens follow in the same workgroup where they are few, else in a second launch over
// all of the chip.
#include "attn_launch.hpp"
#include "device_common.hpp"

namespace ql {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;

// The exclusive prefixes of x and y over the workgroup's threads; sh holds a pair per wave.  The sums are
// within 2^31: the batch has been found to fit.
struct Pair {
  int x, y;
};
__device__ __forceinline__ Pair block_scan2(Pair v, Pair* sh, Pair& total) {
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

// Moves the n pages of each lane's sequence: move(s, x, y, j) its page j.  Few pages are moved by their own
// lane, more by all lanes of the wave, sequence after sequence.
template <class Move> __device__ __forceinline__ void move_pages(int s, int n, int x, int y, Move&& move) {
  const bool few = n <= 4;
  if (few)
    for (int j = 0; j < n; ++j) move(s, x, y, j);
  uint64_t many = __ballot(!few);
  while (many) {
    const int from = __builtin_ctzll(many);
    many &= many - 1;
    const int s1 = __builtin_amdgcn_readlane(s, from), n1 = __builtin_amdgcn_readlane(n, from);
    const int x1 = __builtin_amdgcn_readlane(x, from), y1 = __builtin_amdgcn_readlane(y, from);
    for (int j = threadIdx.x & 63; j < n1; j += 64) move(s1, x1, y1, j);
  }
}

// Rows [first, last) of positions and slots, by the threads of this workgroup.
__device__ __forceinline__ void tokens(const ExtendArgs& a, int64_t first, int64_t last) {
  const int total = a.cu_q[a.n_seqs];
  for (int64_t i = first + threadIdx.x; i < last; i += kThreads) {
    int64_t pos = 0, slot = -1;
    if (i < total) {
      int b = 0, e = a.n_seqs;  // the last sequence with cu_q <= i
      while (e - b > 1) {
        const int m = (b + e) / 2;
        if (a.cu_q[m] <= i) b = m; else e = m;
      }
      pos = (int64_t)a.lens_out[b] - a.cu_q[b + 1] + i;  // its length before, and the tokens before this one
      const int64_t page = a.page_div.div((uint32_t)pos);
      slot = (int64_t)a.table[b * a.table_stride + page] * a.page_size + (pos - page * a.page_size);
    }
    a.positions[i] = pos;
    a.slots[i] = slot;
  }
}

__global__ __launch_bounds__(kThreads) void extend_kernel(const ExtendArgs a, int with_tokens) {
  __shared__ Pair sh[kWaves];
  __shared__ int64_t sums[kWaves][3];
  const int tid = threadIdx.x;
  const bool list = a.free_pages != nullptr;
  const int64_t f0 = list ? a.free_count[0] : 0;
  // what the whole batch asks for
  int64_t tok = 0, back = 0, need = 0;
  bool fits = true;
  for (int s = tid; s < a.n_seqs; s += kThreads) {
    const Ask k = ask(a, s);
    tok += k.now, back += k.back, need += k.need;
    fits &= k.fits;
  }
  tok = wave_sum(tok), back = wave_sum(back), need = wave_sum(need);
  if ((tid & 63) == 0) sums[tid >> 6][0] = tok, sums[tid >> 6][1] = back, sums[tid >> 6][2] = need;
  const bool misfit = __syncthreads_or(!fits) != 0;
  tok = back = need = 0;
  for (int w = 0; w < kWaves; ++w) tok += sums[w][0], back += sums[w][1], need += sums[w][2];
  int why = (tok > a.rows ? 1 : 0) | (misfit ? 4 : 0);
  if (list) why |= (need > f0 + back ? 2 : 0) | (f0 < 0 || f0 + back > a.free_cap ? 8 : 0);
  // pages that come back
  if (why == 0 && back > 0) {
    int before = (int)f0;
    for (int s0 = 0; s0 < a.n_seqs; s0 += kThreads) {
      const int s = s0 + tid;
      Pair v = {0, 0}, total;
      if (s < a.n_seqs) v.x = ask(a, s).back;
      const Pair e = block_scan2(v, sh, total);
      move_pages(s, v.x, before + e.x, 0,
                 [&](int s, int to, int, int j) { a.free_pages[to + j] = a.table[s * a.table_stride + j]; });
      before += total.x;
    }
    __syncthreads();
  }
  // lengths, prefix and pages that are taken
  int row = 0, taken = 0;
  for (int s0 = 0; s0 < a.n_seqs; s0 += kThreads) {
    const int s = s0 + tid;
    Pair v = {0, 0}, total;
    Ask k = {};
    if (s < a.n_seqs && why == 0) {
      k = ask(a, s);
      v = {k.now, k.need};
    }
    const Pair e = block_scan2(v, sh, total);
    if (s < a.n_seqs) {
      a.cu_q[s] = row + e.x;
      const int len = why == 0 ? k.old + k.now : a.lens[s];
      a.lens_out[s] = len;
    }
    move_pages(s, v.y, (int)(f0 + back) - 1 - (taken + e.y), k.have,
               [&](int s, int top, int have, int j) { a.table[s * a.table_stride + have + j] = a.free_pages[top - j]; });
    row += total.x, taken += total.y;
  }
  if (tid == 0) {
    const int left = (int)(why ? f0 : f0 + back - need);
    a.cu_q[a.n_seqs] = row;
    if (list) a.free_count_out[0] = left;
    a.info[0] = row;
    a.info[1] = taken;
    a.info[2] = why;
    a.info[3] = left;
  }
  if (with_tokens) {
    __syncthreads();
    tokens(a, 0, a.rows);
  }
}

__global__ __launch_bounds__(kThreads) void extend_tokens_kernel(const ExtendArgs a) {
  const int64_t first = (int64_t)blockIdx.x * kThreads;
  tokens(a, first, min(first + kThreads, a.rows));
}

}  // namespace

hipError_t launch_kv_extend(const ExtendArgs& a, hipStream_t s) {
  const bool one = a.rows <= 4 * kThreads;
  extend_kernel<<<1, kThreads, 0, s>>>(a, one ? 1 : 0);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || one) return e;
  extend_tokens_kernel<<<(unsigned)((a.rows + kThreads - 1) / kThreads), kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace ql
