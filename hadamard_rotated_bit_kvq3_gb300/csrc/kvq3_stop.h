// How the warps of a decode CTA leave its chunk loop together when a copy has
// not arrived in time.
//
// The warps meet at one barrier per chunk.  A warp whose wait for chunk i runs
// out marks i before that barrier, and every warp reads the mark after it.  A
// mark without the chunk would not do: a warp that is quick through chunk i
// can run out of polls at chunk i + 1 and mark it while a slower one has yet
// to read for chunk i; the slow one would leave a chunk before the others,
// which then wait at a barrier that it never reaches.  With the chunk in the
// mark that reader goes on to chunk i + 1 and leaves there with the rest: a
// mark of chunk i is written before the barrier of chunk i, so it is seen by
// all of them after it, and nobody gets past it to mark a later one.
//
// Plain C++, so that the protocol can be explored on a host.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define KVQ3_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define KVQ3_HOST_DEVICE inline
#endif

namespace kvq3 {

constexpr uint32_t kNoStop = 0;   // no wait has run out

// The mark of chunk i of a CTA (fewer than 2^32 - 1 of them).
KVQ3_HOST_DEVICE uint32_t stop_mark(int64_t i) { return (uint32_t)i + 1u; }

// Whether a warp that has passed the barrier of chunk i and read `mark` leaves there.
KVQ3_HOST_DEVICE bool stops_at(uint32_t mark, int64_t i) { return mark == stop_mark(i); }

}  // namespace kvq3
