// attn_split.cuh -- attention of requests that share prefixes with several kinds of
// CTAs: some attend the prefixes, on the tensor cores, with one query tile or with two
// that share K and V (attn_tree.cuh; over an e4m3 cache there can be both); others each
// request's own keys, with one query tile or, for single tokens with few heads, as
// attn_few.cuh does.  How many of each is found by every CTA from the lengths, by what a
// step of its kind takes.
#pragma once

#include "attn_few.cuh"

namespace b2pa {

// tiles: query tiles of a prefix; sets: rows of own keys in attn_few.cuh, in sets of
// eight (0: one query tile).  Instantiated in attn_split.cu, attn_split64.cu
// and attn_split8.cu.
template <int D, bool FP8, int kTiles, int kSets>
cudaError_t launch_split(const TreeParams& p, cudaStream_t stream);

}  // namespace b2pa
