// Host tables of rotations for the rotary positions (gbb_rope_table).
#include <algorithm>
#include <cmath>
#include <exception>
#include <new>
#include <thread>
#include <vector>

#include "internal.h"

using namespace gbb;

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;

// Frequency of pair i after scaling (the formulas are at gbb_rope_scaling).
double frequency(int i, int rot, double base, const gbb_rope_scaling& s) {
  const double f = std::pow(base, -2.0 * i / rot);
  if (s.kind == GBB_ROPE_LINEAR) return f / s.factor;
  if (s.kind == GBB_ROPE_BANDS) {
    const double w = kTwoPi / f;
    if (w < s.original_len / s.high) return f;
    if (w > s.original_len / s.low) return f / s.factor;
    const double t = (s.original_len / w - s.low) / (s.high - s.low);
    return (1 - t) * f / s.factor + t * f;
  }
  if (s.kind == GBB_ROPE_YARN) {
    const auto index = [&](double turns) {
      return rot * std::log(s.original_len / (kTwoPi * turns)) / (2 * std::log(base));
    };
    const double a = std::max(std::floor(index(s.high)), 0.0);
    const double b = std::min(std::ceil(index(s.low)), double(rot - 1));
    const double t = std::min(std::max((i - a) / std::max(b - a, 0.001), 0.0), 1.0);
    return (1 - t) * f + t * f / s.factor;
  }
  return f;
}

gbb_status check_scaling(const gbb_rope_scaling& s) {
  if (s.kind < GBB_ROPE_PLAIN || s.kind > GBB_ROPE_YARN) return fail(GBB_E_ARG, "unknown rope scaling %d", s.kind);
  if (!std::isfinite(s.attention) || s.attention == 0)
    return fail(GBB_E_ARG, "the attention factor must be finite and not 0 (%g)", s.attention);
  if (s.kind == GBB_ROPE_PLAIN) return GBB_OK;
  if (!(std::isfinite(s.factor) && s.factor >= 1)) return fail(GBB_E_ARG, "the factor must be at least 1 (%g)", s.factor);
  if (s.kind == GBB_ROPE_LINEAR) return GBB_OK;
  if (!(std::isfinite(s.original_len) && s.original_len > 0))
    return fail(GBB_E_ARG, "original_len must be positive (%g)", s.original_len);
  if (!(std::isfinite(s.high) && s.low > 0 && s.low < s.high))
    return fail(GBB_E_ARG, "low and high must satisfy 0 < low < high (%g, %g)", s.low, s.high);
  return GBB_OK;
}

}  // namespace

extern "C" gbb_status gbb_rope_table(int rot, int n_pos, double base, const gbb_rope_scaling* scaling, float* table) {
  if (!table) return fail(GBB_E_ARG, "table is NULL");
  if (rot < 2 || rot % 2) return fail(GBB_E_ARG, "rot must be even and positive (%d)", rot);
  if (n_pos <= 0) return fail(GBB_E_ARG, "n_pos must be positive (%d)", n_pos);
  if (!(std::isfinite(base) && base > 1)) return fail(GBB_E_ARG, "base must be above 1 (%g)", base);
  gbb_rope_scaling s = {GBB_ROPE_PLAIN, 1, 0, 0, 0, 1};
  if (scaling) {
    s = *scaling;
    const gbb_status st = check_scaling(s);
    if (st != GBB_OK) return st;
  }
  const int half = rot / 2;
  try {
    std::vector<double> f(half);
    for (int i = 0; i < half; ++i) f[i] = frequency(i, rot, base, s);
    const auto rows = [&](int p0, int p1) {
      float* t = table + size_t(p0) * rot;
      for (int p = p0; p < p1; ++p)
        for (int i = 0; i < half; ++i) {
          const double a = p * f[i];
          *t++ = float(std::cos(a) * s.attention);
          *t++ = float(std::sin(a) * s.attention);
        }
    };
    const size_t pairs = size_t(n_pos) * half;
    const int want = int(std::min<size_t>(std::min(16u, std::max(1u, std::thread::hardware_concurrency())), 1 + pairs / 65536));
    const int step = n_pos / want + (n_pos % want != 0);
    std::vector<std::thread> pool;
    pool.reserve(want);
    int p0 = 0;
    try {
      for (; p0 + step < n_pos; p0 += step) pool.emplace_back(rows, p0, p0 + step);
    } catch (const std::exception&) {
      // no further thread, or no memory for its state, to be had: this one
      // does the rest, and those that run are joined below
    }
    rows(p0, n_pos);
    for (auto& t : pool) t.join();
  } catch (const std::bad_alloc&) {
    return fail(GBB_E_SPACE, "out of host memory");
  }
  return GBB_OK;
}
