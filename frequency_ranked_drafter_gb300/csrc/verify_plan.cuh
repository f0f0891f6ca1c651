// How many CTAs vt_verify_draft gives a sequence (host code, no CUDA).
#pragma once

#include <cstdint>

namespace vt {

constexpr int kVerifyMaxCluster = 16;

// CTAs a sequence, a power of two with 1024 ids a CTA at least, and no more than
// `largest`, the clusters that the device can hold.  An SM holds four CTAs.  Up
// to eight a sequence, two rounds of shorter segments beat one of longer ones
// (V = 128256, B = 100: 27.4 us with eight, 31.9 with four; V = 32003, B = 64:
// 9.1 and 11.9); sixteen have to fit at once (V = 128256, B = 24: 10.3 us with
// sixteen, 14.6 with eight; B = 64: 21.1 and 18.0).
inline int verify_ctas(int B, int V, int num_sms, int largest) {
  int C = 1;
  while (2 * C <= largest && 2 * C <= kVerifyMaxCluster && V > C * 1024 &&
         (int64_t)B * C * 2 <= (C < 8 ? 8ll : 4ll) * num_sms)
    C *= 2;
  return C;
}

}  // namespace vt
