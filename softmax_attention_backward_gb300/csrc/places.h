// Where the segments of packed sequences lie in linear attention's workspace
// (linear_attn.cu).  Free of CUDA types, so that a host program can go over the
// arrays that no caller should pass.
#pragma once

#include <cstdint>

#include "fastdiv.h"   // ATTN_HD

namespace attn {

constexpr int kLinearChunk = 128;   // tokens of a chunk

ATTN_HD int chunks_of(int len) { return static_cast<int>((static_cast<uint32_t>(len) + kLinearChunk - 1) / kLinearChunk); }
ATTN_HD int segments_of(int len, int seg_chunks) {
  const int n = (chunks_of(len) + seg_chunks - 1) / seg_chunks;
  return n > 1 ? n : 1;
}

// The end of a sequence whose entry of cu_seqlens is `e`, `before` the one of the
// sequence before: entries count within [0, tokens] and never decrease.  So whatever
// the array holds sequences are disjoint, and their lengths add up to `tokens` at most.
ATTN_HD int packed_end(int e, int before, int tokens) {
  const int kept = e < 0 ? 0 : e > tokens ? tokens : e;
  return kept > before ? kept : before;
}

// The CTAs that the segments of all sequences take at most: a sequence has one more than `len` fills.
ATTN_HD int packed_walks(int tokens, int num_seqs, int seg_chunks) {
  return tokens / (seg_chunks * kLinearChunk) + num_seqs;
}
// And the states that segments hand on, all but the last of each sequence: the workspace's places.
ATTN_HD int packed_places(int tokens, int seg_chunks) { return tokens / (seg_chunks * kLinearChunk); }

}  // namespace attn
