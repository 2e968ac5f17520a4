// The places of an accepted path, as kv_compact_tokens8's kernel takes them:
// plain arithmetic, for the host too.
#pragma once

#ifdef __CUDACC__
#define SMC_BOTH __host__ __device__ __forceinline__
#else
#define SMC_BOTH inline
#endif

namespace smcsd {

struct PathPlaces {
  int first;  // the table's place of new token 0
  int held;   // new tokens of the sequence; first + held tokens are in its table
  int n;      // entries of the path (may be more: what is past `held` is refused)
  int block;  // tokens of a block

  // Places [i0, end) are taken at a time: whole blocks, as many as there is
  // `room` for (at least a block's).
  SMC_BOTH int end(int i0, int room) const {
    const int off = i0 < held ? (first + i0) % block : 0;
    const int most = (off + room) / block * block - off;
    return n - i0 < most ? n : i0 + most;
  }
  // Tokens move into places before this one only: an entry that counts is less
  // than `held` and no less than its place.  Past it lies the table's end.
  SMC_BOTH int moves_end(int end) const { return end < held ? end : held; }
  // The table's slot of a place before moves_end, and the end of its places.
  SMC_BOTH int slot(int i) const { return (first + i) / block; }
  SMC_BOTH int slot_end(int i, int end) const {
    const int off = (first + i) % block;
    return end - i < block - off ? end : i + (block - off);
  }
};

}  // namespace smcsd
