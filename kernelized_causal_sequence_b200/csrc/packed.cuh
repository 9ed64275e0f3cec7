// packed.cuh — where the sequences of a packed token axis lie.
#pragma once
#include <stdint.h>

namespace la {

// cu[s] clamped to the N tokens there are, so that no value of the caller's
// array leads outside the tensors.
__device__ __forceinline__ int seq_start(const int32_t *cu, int s, int N) {
    const int x = cu[s];
    return x < 0 ? 0 : x > N ? N : x;
}

// The sequence of token t: the last s with cu[s] <= t (0 if there is none).
__device__ __forceinline__ int seq_of_token(const int32_t *cu, int n_seq, int N, int t) {
    int lo = 0, hi = n_seq;   // cu[lo] <= t < cu[hi], where cu is in order
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (seq_start(cu, mid, N) <= t) lo = mid; else hi = mid;
    }
    return lo;
}

// Tiles of BM queries over all sequences without a count of tiles: sequence s
// gets the tile numbers from cu[s] / BM + s on.  It has room for
// floor(cu[s+1] / BM) - floor(cu[s] / BM) + 1 >= ceil(len / BM) of them, so
// N / BM + n_seq numbers serve any lengths, and the sequence of a number is
// found by bisection.  A number without a tile gives q0 >= end.
struct SeqTile {
    int begin, end;   // the sequence's tokens
    int q0;           // the tile's first token
};
template <int BM> __device__ __forceinline__ SeqTile seq_tile(const int32_t *cu, int n_seq, int N, int x) {
    int lo = 0, hi = n_seq;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (seq_start(cu, mid, N) / BM + mid <= x) lo = mid; else hi = mid;
    }
    SeqTile t;
    t.begin = seq_start(cu, lo, N);
    t.end = seq_start(cu, lo + 1, N);
    const int i = x - (t.begin / BM + lo);
    // (i < 0 or past the end only where cu is out of order; N < 2^30 keeps this in 32 bits)
    t.q0 = i < 0 ? t.end : t.begin + i * BM;
    return t;
}
inline int seq_tiles(int N, int n_seq, int BM) { return N / BM + n_seq; }

}  // namespace la
