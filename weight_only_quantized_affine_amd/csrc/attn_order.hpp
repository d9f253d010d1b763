// The order in which a wave of the tile kernel goes through the key tiles of an item: its copies into
// LDS, its products and the barriers that keep them apart.  A template over the steps, so that the
// host can run the same text with steps that record what is read and written between barriers.
#pragma once

#ifdef __HIPCC__
#define QL_ORDER __host__ __device__ __forceinline__
#else
#define QL_ORDER inline
#endif

namespace ql {

enum class AttnStep {
  kBarrier,
  kPages,     // page ids of the item's first tile
  kCopyK,     // start the copy of K of tile t, and note which of its keys are to be seen
  kCopyV,     // start the copy of V of tile t
  kWait,      // the wave's copies have arrived
  kScores,    // scores of tile t (before the first weights)
  kWeights,   // weights of tile t from its scores
  kProducts,  // output of tile t, then scores of tile t + 1
  kIdle,      // a wave without rows: its share of what all waves do for the products of tile t
};
template <AttnStep S> struct AttnStepOf {
  static constexpr AttnStep value = S;
};

// Where tile t lies: stages of K and of V, and places of the bits of the keys to be seen.
template <int ST> QL_ORDER int attn_stage(int t) { return t % ST; }
QL_ORDER int attn_seen_at(int t) { return t & 3; }
// The finite copy of a V tile.
QL_ORDER int attn_clean_at(int t) { return t & 1; }

// n tiles with ST stages.  `copier`: the wave copies; `late`: it runs half a tile behind (not with
// two stages); `idle`: it has no rows.  A period ends with a barrier, which early waves meet after
// their products and late ones after their weights.  Copies start with a period and are waited for
// at its end, and what they write was last read a period before.
template <int ST, class Step>
QL_ORDER void attn_tile_order(int n, bool copier, bool late, bool idle, Step&& step) {
  using S = AttnStep;
  auto copies = [&](int t) {
    if (t < n) step(AttnStepOf<S::kCopyV>{}, t);
    if (t + 1 < n) step(AttnStepOf<S::kCopyK>{}, t + 1);
  };
  step(AttnStepOf<S::kBarrier>{}, 0);  // the last item's reads are done
  if (copier) {
    step(AttnStepOf<S::kPages>{}, 0);
    step(AttnStepOf<S::kCopyK>{}, 0);
    copies(0);
    step(AttnStepOf<S::kWait>{}, 0);
  }
  step(AttnStepOf<S::kBarrier>{}, 0);
  if (!idle) step(AttnStepOf<S::kScores>{}, 0);
  // With two stages K of tile 2 takes the place of K of tile 0, whose scores some waves may still be
  // at while others start its copy: they wait for each other once an item.
  if (ST == 2) step(AttnStepOf<S::kBarrier>{}, 0);
  if (idle) {
    for (int t = 0; t < n; ++t) {
      if (copier) copies(t + 1);
      step(AttnStepOf<S::kIdle>{}, t);
      if (copier) step(AttnStepOf<S::kWait>{}, t);
      step(AttnStepOf<S::kBarrier>{}, t);
    }
  } else {
    for (int t = 0; t < n; ++t) {
      if (copier) copies(t + 1);
      step(AttnStepOf<S::kWeights>{}, t);
      if (late) step(AttnStepOf<S::kBarrier>{}, t);
      step(AttnStepOf<S::kProducts>{}, t);  // (after the last tile the scores are of stale keys and unused)
      if (!late) {
        step(AttnStepOf<S::kWait>{}, t);
        step(AttnStepOf<S::kBarrier>{}, t);
      }
    }
  }
}

}  // namespace ql
