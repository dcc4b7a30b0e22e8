// bl_sample_cut.h - how the sampler cuts a batch of rows: CTAs per row, and the
// kernel form. Plain C++.
#pragma once

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
  bool wide;      // every SM has one CTA at most: 1024 threads instead of 512
  size_t smem;
};

// fixed: shared memory beside the logits. fits(cut): whether a cluster of more than
// kPortableCluster CTAs of this form can run on the device; where it cannot, the
// next smaller ones take the row.
template <typename Fits>
SampleCut sample_cut(int64_t B, int64_t V, int num_sms, size_t fixed, Fits fits) {
  SampleCut c;
  for (int most = kMaxCluster;; most /= 2) {
    // So many CTAs that a stretch packs its histogram and two CTAs fit an SM, then
    // more while rows alone leave SMs idle and stretches stay long.
    int C = 1;
    while (C < most && ((V + C - 1) / C > kPackMax || (B * C * 2 <= 2 * num_sms && V / (2 * C) >= 2048))) C *= 2;
    c.cluster = C;
    c.per = (int)((V + C - 1) / C);
    c.smem = fixed + 4 * (size_t)(c.per + 16);
    c.resident = c.smem <= kSampleSmemMax;
    if (!c.resident) c.smem = fixed;
    c.wide = c.resident && B * C <= num_sms;
    if (C <= kPortableCluster || fits(c)) return c;
  }
}

}  // namespace bl
