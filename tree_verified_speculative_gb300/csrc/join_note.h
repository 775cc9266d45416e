// join_note.h -- what a CTA of the attention leaves for the join, and when the
// join may use it.  No CUDA header is needed, so host code can check it too.
#pragma once

#ifdef __CUDACC__
#define MFD_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MFD_HOST_DEVICE inline
#endif

namespace mfd {

// Whether a CTA holds parts (of the item its stretch starts in, of the one it
// ends in), and of the latter, if this CTA has its first part, where it is and
// how many CTAs it reaches over.  All zeros: nothing to join.
struct Cut {
  int has[2];
  int reach;  // 0: no first part
  int q, h, pair, nn;
};

// Whether CTA `cta` of n_cta left the first part of an item of this call.  The
// note lies in scratch that nobody zeroes, and its numbers become bounds and
// addresses: a note that is not of this call must never be followed.
// (In signed comparisons one after the other it cost a call 0.4 us, and 0.2 like
// this: the join is short and fetches each of its instructions for the first time.)
MFD_HOST_DEVICE bool cut_usable(const Cut &c, int cta, int n_cta, int n_req, int Hk, int n_pair, int N) {
  return ((unsigned)c.reach - 1u < (unsigned)(n_cta - cta)) & ((unsigned)c.q < (unsigned)n_req) &
         ((unsigned)c.h < (unsigned)Hk) & ((unsigned)c.pair < (unsigned)n_pair) & ((unsigned)c.nn - 1u < (unsigned)N);
}

// A part's weight in the join's sum: `w` over the row's sum (inv: one over it).
// A CTA's stretch of the item may hold no key tile; there is no part then (slot
// -1), and it must have weight zero, which is what keeps it from being read,
// whatever the sum is: a row with a NaN has a NaN for inv.  TINY_WEIGHT stands
// for a weight that is more than zero but nothing in 32 bits.
constexpr float TINY_WEIGHT = -1.f;
MFD_HOST_DEVICE float join_weight(int slot, float w, float inv) {
  return slot < 0 ? 0.f : w == TINY_WEIGHT ? w : w * inv;
}

}  // namespace mfd
