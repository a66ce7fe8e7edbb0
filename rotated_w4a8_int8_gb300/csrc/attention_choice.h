// How many CTAs share keys in the kernel for few rows (host code only).
#pragma once

#include <cstdint>

namespace cratt {

constexpr int MOST_FEW_SLICES = 16;

// CTAs that share the keys of a sequence's K head (`units` of them, `tiles` of 64
// keys each) on `sms` SMs, at most `largest`, the largest cluster that fits the
// device: as many as fit the SMs twice (152 of them; one token, 56 heads x 19989
// keys: 4 or 5 CTAs 83 us, 2 97 us, 6, which take two rounds, 99 us; 2 heads x
// 32768 keys: 16 CTAs 20 us, 8 33 us), two tiles or more for each; with more heads
// than that, four where the keys are long, so that the last round is short (512 x
// 8191 keys: 213 us, whole 242 us; 512 x 512: 26 to 41 us in parts, whole 16 us).
[[maybe_unused]] static int few_slices(int64_t units, int64_t tiles, int sms, int largest) {
  int64_t n = 2 * sms / units, most = tiles / 2;
  if (n < 2) n = 4, most = tiles / 32;
  // larger clusters than eight fit less well: only where they have the SMs for themselves (30 heads x 4096 keys: by
  // eight 10 us, by ten 18 us)
  if (n > 8) n = sms / units > 8 ? sms / units : 8;
  n = n < most ? n : most;
  n = n < MOST_FEW_SLICES ? n : MOST_FEW_SLICES;
  n = n < largest ? n : largest;
  return static_cast<int>(n < 1 ? 1 : n);
}

}  // namespace cratt
