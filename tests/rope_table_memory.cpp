// Runs gbb_rope_table with the k-th allocation refused, for every k up to the
// last one it makes: an error or the whole table, never the end of the process.
#include <atomic>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <new>
#include <vector>

#include "gbb.h"

static std::atomic<long> left{-1};   // allocations that succeed from here; below 0: all

void* operator new(size_t n) {
  if (left.load() >= 0 && left.fetch_sub(1) <= 0) {
    left = 0;   // and every later one is refused too
    throw std::bad_alloc();
  }
  if (void* p = std::malloc(n ? n : 1)) return p;
  throw std::bad_alloc();
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, size_t) noexcept { std::free(p); }

int main() {
  const int rot = 128, n_pos = 9001;   // work for several threads
  std::vector<float> want(size_t(rot) * n_pos), got(want.size());
  if (gbb_rope_table(rot, n_pos, 10000.0, nullptr, want.data()) != GBB_OK) return 1;
  int errors = 0, tables = 0;
  for (long k = 0; k < 40; ++k) {
    std::memset(got.data(), 0xff, got.size() * 4);
    left = k;
    const gbb_status st = gbb_rope_table(rot, n_pos, 10000.0, nullptr, got.data());
    left = -1;
    if (st == GBB_E_SPACE) {
      ++errors;
    } else if (st == GBB_OK) {
      ++tables;
      if (std::memcmp(got.data(), want.data(), got.size() * 4)) return 2;
    } else {
      return 3;
    }
  }
  if (!errors || !tables) return 4;
  std::puts("ok");
  return 0;
}
