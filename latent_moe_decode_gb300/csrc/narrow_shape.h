// What a CTA of the narrow BF16 product takes of an SM: stages, runs of K, TMEM columns, shared memory (plain C++).
#pragma once

#include <cstddef>

namespace moe {
namespace linear_impl {

constexpr int kMaxSmem = 227 * 1024;  // shared memory a CTA may have
constexpr int kSmSmem = 228 * 1024;   // ... and an SM, 1 KB of it reserved per CTA
constexpr int kSmTmemCols = 512;      // TMEM columns of an SM
constexpr int kStaticSmem = 1536;     // an upper bound on a kernel's static shared memory and its reserve
constexpr int kBlockK = 64;           // K of a pipeline stage: one 128-byte swizzle row

constexpr int kLanes = 128;                    // rows of b a tile
constexpr int kBBytes = kLanes * kBlockK * 2;  // of a stage
constexpr int kNarrowStages = 12;
constexpr int kMaxRunBlocks = 8;               // blocks of K of a run, where TMEM has the columns
constexpr int kEnoughStages = 5;               // (beside the partials)

// Shared memory of a CTA beside its alignment, where an SM holds `per_sm` of them.
constexpr int room(int per_sm) { return (per_sm == 1 ? kMaxSmem : kSmSmem / per_sm) - kStaticSmem - 1024; }
constexpr int partial_bytes(int bn, int splits) { return ((bn / 4 - 1) / splits + 1) * splits * kLanes * 16; }
constexpr int narrow_stage_bytes(int bn) { return kBBytes + bn * kBlockK * 2; }

struct NarrowShape {
  int stages, runs, tmem_cols;
  bool apart;     // the partials stay beside the stages
  size_t smem;    // dynamic
};

// Of tiles of bn rows of a, nbk blocks of K split over `splits` CTAs; bn <= 512 / per_sm and
// partial_bytes(bn, splits) <= room(per_sm).
constexpr NarrowShape narrow_shape(int bn, int splits, int per_sm, int nbk) {
  NarrowShape s = {};
  const int blocks = (nbk - 1) / splits + 1;  // of a CTA, at most
  s.runs = (blocks - 1) / kMaxRunBlocks + 1;
  if (s.runs > kSmTmemCols / per_sm / bn) s.runs = kSmTmemCols / per_sm / bn;
  s.tmem_cols = 32;
  while (s.tmem_cols < s.runs * bn) s.tmem_cols *= 2;
  // The partials stay beside the stages where enough of these are left.
  const int stage = narrow_stage_bytes(bn), part = partial_bytes(bn, splits), beside = (room(per_sm) - part) / stage;
  s.apart = beside >= kEnoughStages || beside >= blocks;
  s.stages = s.apart ? beside : room(per_sm) / stage;
  if (s.stages > kNarrowStages) s.stages = kNarrowStages;
  if (s.stages > blocks) s.stages = blocks;
  // A CTA takes at least its TMEM columns' share of an SM's shared memory, so that the CTAs an SM holds never ask for
  // more than its 512 columns: tcgen05.alloc would make one wait for another, in a ring of waits where clusters meet
  // at barriers.
  s.smem = (size_t)s.stages * stage + (s.apart ? part : 0);
  const size_t least = (size_t)s.tmem_cols * (kSmSmem / kSmTmemCols) - kStaticSmem - 1024;
  if (s.smem < (size_t)part) s.smem = part;
  if (s.smem < least) s.smem = least;
  if (s.smem > (size_t)room(1)) s.smem = room(1);
  s.smem += 1024;
  return s;
}

}  // namespace linear_impl
}  // namespace moe
