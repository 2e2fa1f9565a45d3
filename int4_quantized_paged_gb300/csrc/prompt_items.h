// The items of an attention over whole prompts and the search of one by its number.
//
// A sequence of n tokens is cut into items of `per` positions, one for each KV head.
// Items are numbered by levels, the highest first: level q has the items that begin at
// position q * per, of each sequence longer than that, in the sequences' order, the
// KV heads of one together.  So those with the most keys come first.
//
// A search starts where the last one ended, which costs nothing while the numbers
// ascend.  That is how they usually come, but nothing says in which order the launches
// of a grid are cancelled: a smaller number starts the search again from the top.
//
// Plain C++, so that it also runs without a GPU.  A warp searches together; Lanes gives
// it 32 sequences at a time:
//   unsigned longer(int b0, int than)   bit i: sequence b0 + i has more than `than` tokens
//   int nth(unsigned m, int r)          position of set bit r (from 0) of m, -1 if there is none
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define KVQ_HD __host__ __device__ __forceinline__
#else
#define KVQ_HD inline
#endif

namespace kvq {

struct PromptSeqs {
  const int* start;                            // [B + 1]
  long long T;                                 // tokens that there are
  int B, max_len;                              // sequences, the caller's bound of their lengths
  int Hkv, per;
};

// Positions [p0, end) of the sequence that starts at token t0, KV head g; p0 < 0: none.
struct PromptItem {
  int t0, p0, end, g;
};

// Tokens of sequence b that are computed: none past the bound, none of a sequence that
// does not lie within the tokens.  *wrong is set where that leaves some out.
KVQ_HD int prompt_length(const PromptSeqs& s, int b, bool* wrong) {
  if (b >= s.B) return 0;
  const long long t = s.start[b], e = s.start[b + 1];
  const bool bad = t < 0 || e < t || e > s.T;
  const bool over = !bad && e - t > s.max_len;
  *wrong |= bad || over;
  return bad ? 0 : over ? s.max_len : (int)(e - t);
}

template <class Lanes>
struct PromptSearch {
  const PromptSeqs& s;
  const Lanes& lanes;
  int levels;                                  // level `levels` and those above it are empty
  int level;                                   // where the search stands,
  int at_level;                                // the sequences that have an item there,
  long long before;                            // and the items of the levels above

  // longest: the tokens of the longest sequence
  KVQ_HD PromptSearch(const PromptSeqs& s, const Lanes& lanes, int longest)
      : s(s), lanes(lanes), levels((longest + s.per - 1) / s.per) {
    restart();
  }

  KVQ_HD void restart() {
    level = levels;
    at_level = 0;
    before = 0;
  }

  // Item w; none where there are no more than w.
  KVQ_HD PromptItem find(long long w) {
    PromptItem it = {0, -1, 0, 0};
    if (w < before) restart();
    while (w - before >= (long long)at_level * s.Hkv) {
      if (level == 0) return it;
      before += (long long)at_level * s.Hkv;
      --level;
      at_level = 0;
      for (int b0 = 0; b0 < s.B; b0 += 32) at_level += bits(lanes.longer(b0, level * s.per));
    }
    const unsigned n = (unsigned)(w - before);             // below 2^32, as at_level * Hkv is
    int r = (int)(n / (unsigned)s.Hkv);                    // which of the level's sequences
    const int g = (int)(n - (unsigned)r * (unsigned)s.Hkv);
    for (int b0 = 0; b0 < s.B; b0 += 32) {
      const unsigned m = lanes.longer(b0, level * s.per);
      const int i = lanes.nth(m, r);
      if (i >= 0) {
        const int b = b0 + i;
        bool ignored = false;
        it.t0 = s.start[b];
        it.p0 = level * s.per;
        it.g = g;
        const int n_b = prompt_length(s, b, &ignored);
        it.end = n_b - it.p0 < s.per ? n_b : it.p0 + s.per;
        return it;
      }
      r -= bits(m);
    }
    return it;
  }

 private:
  KVQ_HD static int bits(unsigned m) {
#ifdef __CUDA_ARCH__
    return __popc(m);
#else
    return __builtin_popcount(m);
#endif
  }
};

}  // namespace kvq
