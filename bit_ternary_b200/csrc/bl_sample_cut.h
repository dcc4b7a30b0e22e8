// bl_sample_cut.h - how the sampler cuts a batch of rows: CTAs per row, and the
// kernel form. Plain C++.
#pragma once

#include <initializer_list>

#include <stddef.h>
#include <stdint.h>

namespace bl {

constexpr int kMaxCluster = 16;
constexpr int kPortableCluster = 8;  // every device takes clusters up to this size
constexpr int kPackMax = 16383;      // tokens per CTA whose count and places fit 14 + 18 bits
constexpr size_t kSampleSmemMax = 225 * 1024;

struct SampleCut {
  int cluster;    // CTAs per row
  int per;        // tokens per CTA
  bool resident;  // the CTA keeps its tokens in shared memory
  bool wide;      // 1024 threads, one CTA an SM, instead of 512
  size_t smem;
};

// fixed: shared memory beside the logits. at_once(cut): how many clusters of this
// form the device runs at a time. A cluster needs its SMs in one part of the chip, so
// that is fewer than the SMs would hold (B200: 7 of 16 wide CTAs, 14 of 16 narrow
// ones, 15 and 33 of 8), and none of 16 CTAs is sure of. The first of the cuts below
// that runs all rows at once is taken: a row more than that waits for a whole row's
// time (128000 tokens, top-p: 7 rows 22 us; 8 rows 43 as 16 wide CTAs, 25 as 16
// narrow ones; 15 rows 40 as 16 narrow ones, 25 as 8 wide ones).
template <typename AtOnce>
SampleCut sample_cut(int64_t B, int64_t V, int num_sms, size_t fixed, AtOnce at_once) {
  const auto form = [&](int C, bool wide) {
    SampleCut c;
    c.cluster = C;
    c.per = (int)((V + C - 1) / C);
    c.smem = fixed + 4 * (size_t)(c.per + 16);
    c.resident = c.smem <= kSampleSmemMax;
    if (!c.resident) c.smem = fixed;
    c.wide = wide && c.resident;
    return c;
  };
  // So many CTAs that a stretch packs its histogram and two CTAs fit an SM, then
  // more while rows alone leave SMs idle and stretches stay long.
  int C = 1;
  while (C < kMaxCluster && ((V + C - 1) / C > kPackMax || (B * C * 2 <= 2 * num_sms && V / (2 * C) >= 2048))) C *= 2;
  while (C > kPortableCluster && at_once(form(C, false)) == 0) C /= 2;
  // Fewer, as far as stretches still pack, where those do not run at once.
  for (int c = C;; c /= 2) {
    for (const bool wide : {true, false}) {
      const SampleCut cut = form(c, wide);
      if (cut.wide == wide && at_once(cut) >= B) return cut;
    }
    if (c == 1 || (V + c / 2 - 1) / (c / 2) > kPackMax) break;
  }
  const SampleCut wide = form(C, true);
  return B * C <= num_sms && at_once(wide) > 0 ? wide : form(C, false);
}

}  // namespace bl
