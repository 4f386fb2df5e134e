// Runs gbb_rope_table over sizes, scalings and refusals for the sanitizers.
#include <cmath>
#include <cstdio>
#include <vector>

#include "gbb.h"

int main() {
  const gbb_rope_scaling all[] = {{GBB_ROPE_PLAIN, 1, 0, 0, 0, 1},
                                  {GBB_ROPE_LINEAR, 4, 0, 0, 0, 0.5},
                                  {GBB_ROPE_BANDS, 8, 8192, 1, 4, 1},
                                  {GBB_ROPE_YARN, 16, 4096, 1, 32, 1.2},
                                  {GBB_ROPE_YARN, 2, 1e-3, 1e-6, 1e6, 1}};
  const int rots[] = {2, 6, 64, 128, 1024};
  const int lens[] = {1, 2, 17, 1000, 5001};
  for (const auto& s : all)
    for (int rot : rots)
      for (int n : lens) {
        std::vector<float> t(size_t(n) * rot);
        if (gbb_rope_table(rot, n, 10000.0, &s, t.data()) != GBB_OK) return 1;
        for (float v : t)
          if (!std::isfinite(v)) return 2;
      }
  std::vector<float> t(64);
  if (gbb_rope_table(8, 8, 10000.0, nullptr, t.data()) != GBB_OK || t[0] != 1.f || t[1] != 0.f) return 3;
  gbb_rope_scaling bad = {9, 1, 0, 0, 0, 1};
  if (gbb_rope_table(8, 8, 10000.0, &bad, t.data()) != GBB_E_ARG) return 4;
  if (gbb_rope_table(7, 8, 10000.0, nullptr, t.data()) != GBB_E_ARG) return 5;
  if (gbb_rope_table(8, 8, NAN, nullptr, t.data()) != GBB_E_ARG) return 6;
  if (gbb_rope_table(8, 8, 10000.0, nullptr, nullptr) != GBB_E_ARG) return 7;
  std::puts("ok");
  return 0;
}
