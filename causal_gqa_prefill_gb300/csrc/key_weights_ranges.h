// key_weights_ranges.h — how the steps of the key weights' kernel are cut into
// ranges, one per CTA. Plain C++ apart from the qualifiers, so that the arithmetic
// can be built and checked without CUDA.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define KEY_WEIGHTS_FN __host__ __device__ __forceinline__
#else
#define KEY_WEIGHTS_FN inline
#endif

namespace gb300_key_weights {

constexpr int kUnitKeys = 256;        // keys per unit
constexpr int kRows = 128;            // rows (query positions x heads) per step
constexpr int kCtas = 152;            // one CTA per SM on a 152-SM GB300

// The units of one (b, K/V head): unit t holds keys 256 t .. 256 t + 255, and its
// steps are first_step(t) .. steps - 1, nr query positions each; position i of the
// rows is off + i.
struct Shape {
  int off, nr, steps, T, causal;
};

// The first step of which a row sees the unit's first key.
KEY_WEIGHTS_FN int first_step(int t, int off, int nr, int causal) {
  const int past = t * kUnitKeys - off;
  return causal && past > 0 ? static_cast<int>(static_cast<unsigned>(past) / static_cast<unsigned>(nr))
                            : 0;
}

// Steps of units 0 .. t - 1, for any t. Units up to s0 - 1 have all of them; unit
// s0 + j lacks its first f(j) = floor((256 j + b) / nr) ones, b = 256 s0 - off. nr
// units further on f has grown by 256 exactly, so with j = nr i + r
//   f(j) = 256 i + f(r),
// and a sum over whole periods is one over the first and an arithmetic series.
class StepsBefore {
 public:
  explicit StepsBefore(const Shape& s)
      : steps_(s.steps), nr_(s.nr), s0_(s.causal ? s.off / kUnitKeys + 1 : s.T) {
    int64_t sum = 0;
    for (int r = 0; r <= nr_ && s0_ + r <= s.T; ++r) {
      lacking_[r] = sum;
      sum += first_step(s0_ + r, s.off, s.nr, s.causal);
    }
  }
  int64_t operator()(int t) const {
    const int64_t all = static_cast<int64_t>(t) * steps_;
    if (t <= s0_) return all;
    const int64_t i = (t - s0_) / nr_, r = (t - s0_) % nr_;
    int64_t lacking = lacking_[r] + i * r * kUnitKeys;
    if (i > 0) lacking += i * lacking_[nr_] + i * (i - 1) / 2 * nr_ * kUnitKeys;
    return all - lacking;
  }

 private:
  int steps_, nr_, s0_;
  int64_t lacking_[kRows + 1];        // [r]: steps that units s0 .. s0 + r - 1 lack
};

// Where each CTA's range starts: unit (of all heads' in order), step, and the number
// of steps.
struct Starts {
  int unit[kCtas], step[kCtas], count[kCtas];
};

// Cuts the steps of `heads` (b, K/V head) into equal ranges; returns how many. *cut:
// does a range start inside a unit?
inline int cut_ranges(const Shape& s, int64_t heads, Starts* st, bool* cut) {
  const StepsBefore before(s);
  const int64_t per_head = before(s.T), W = per_head * heads;
  const int G = static_cast<int>(W < kCtas ? W : kCtas);
  *cut = false;
  int64_t last_head = -1;
  int last_unit = 0;
  for (int c = 0; c < G; ++c) {
    const int64_t x = c * W / G, head = x / per_head, rest = x - head * per_head;
    st->count[c] = static_cast<int>((c + 1) * W / G - x);
    // the unit that holds step `rest` (starts only move on)
    int lo = head == last_head ? last_unit : 0, hi = s.T;
    while (hi - lo > 1) {
      const int mid = lo + (hi - lo) / 2;
      if (before(mid) <= rest)
        lo = mid;
      else
        hi = mid;
    }
    last_head = head;
    last_unit = lo;
    const int first = first_step(lo, s.off, s.nr, s.causal);
    st->unit[c] = static_cast<int>(head * s.T + lo);
    st->step[c] = first + static_cast<int>(rest - before(lo));
    *cut |= st->step[c] != first;
  }
  return G;
}

}  // namespace gb300_key_weights
