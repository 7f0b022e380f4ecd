"""What the narrow BF16 product's CTAs take of an SM (csrc/narrow_shape.h), over every tile, split and K that its plan may
choose, in a small host program: CTAs that share an SM never ask for more TMEM columns than it has."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
#include "narrow_shape.h"
#include <cstdio>
using namespace moe::linear_impl;
#define HOLDS(c) do { if (!(c)) { std::printf("bn %d splits %d per_sm %d nbk %d: %s\n", bn, splits, per_sm, nbk, #c); return 1; } } while (0)
int main() {
  size_t least[kSmTmemCols + 1] = {};  // the least shared memory of a CTA of so many columns
  long long seen = 0;
  for (int bn = 16; bn <= 256; bn += 16)
    for (int splits = 1; splits <= 8; ++splits)
      for (int per_sm = 1; per_sm <= 2; ++per_sm) {
        if (bn > kSmTmemCols / per_sm || partial_bytes(bn, splits) > room(per_sm)) continue;
        for (int nbk = splits; nbk < 40000; nbk += nbk < 2000 ? 1 : 997) {
          const NarrowShape s = narrow_shape(bn, splits, per_sm, nbk);
          const int blocks = (nbk - 1) / splits + 1;
          HOLDS(s.stages >= 1 && s.stages <= kNarrowStages && s.stages <= blocks);
          HOLDS(s.runs >= 1 && s.runs * bn <= s.tmem_cols && s.tmem_cols <= kSmTmemCols / per_sm);
          HOLDS((s.tmem_cols & (s.tmem_cols - 1)) == 0 && s.tmem_cols >= 32);
          HOLDS(s.smem <= (size_t)kMaxSmem - kStaticSmem);
          // 1024 for the stages' alignment, then stages and partials, one behind the other or in one place
          const size_t stages = (size_t)s.stages * narrow_stage_bytes(bn), part = partial_bytes(bn, splits);
          HOLDS(s.smem >= 1024 + (s.apart ? stages + part : stages > part ? stages : part));
          HOLDS(per_sm == 1 || 2 * (s.smem + kStaticSmem) <= (size_t)kSmSmem);
          size_t& l = least[s.tmem_cols];
          if (l == 0 || s.smem < l) l = s.smem;
          ++seen;
        }
      }
  // An SM filled with such CTAs, of one launch or of several, each with its 1 KB reserve and no static memory counted: every
  // two kinds, as many of the first as fit and then of the second; TMEM columns within 512.
  const int bn = 0, splits = 0, per_sm = 0, nbk = 0;
  for (int a = 32; a <= kSmTmemCols; a *= 2)
    for (int b = 32; b <= kSmTmemCols; b *= 2) {
      if (!least[a] || !least[b]) continue;
      const int na = (int)(kSmSmem / (least[a] + 1024));
      for (int i = 0; i <= na; ++i) {
        const int nb = (int)((kSmSmem - i * (least[a] + 1024)) / (least[b] + 1024));
        if (i * a + nb * b > kSmTmemCols) { std::printf("%d of %d columns and %d of %d\n", i, a, nb, b); return 1; }
      }
    }
  HOLDS(seen > 100000 && least[32] && least[512]);
  return 0;
}
"""


def test_narrow_shape(tmp_path):
    (tmp_path / "main.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", os.path.join(ROOT, "latent_moe_decode_gb300", "csrc"), str(tmp_path / "main.cpp"),
                    "-o", str(tmp_path / "main")], check=True)
    run = subprocess.run([str(tmp_path / "main")], capture_output=True, text=True)
    assert run.returncode == 0, run.stdout
