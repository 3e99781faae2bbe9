// extend_ring.h -- which of a row block's r.P distances the band kernel of
// relattn_extend (extend_band.cu) holds in shared memory, and where.  Plain
// arithmetic, on the host as on the device.
//
// Distances come in chunks of 64, a half of 32 to each of a row's two threads; half h
// of the n-th chunk that a CTA takes lies in slot (2 n + h) % slots.  The item's first step reads
// the distances D0 - 63 .. D0 + tokens - 1 (D0: the first row's to the step's first
// key; those below 0 are masked), of up to three chunks, each later step 64 more.
#pragma once

#ifdef __CUDACC__
#define RELATTN_HD __host__ __device__ __forceinline__
#else
#define RELATTN_HD inline
#endif

namespace relattn {

struct BandChunks {
  int start, first;       // the oldest chunk that the first step reads, the newest
};
RELATTN_HD BandChunks band_chunks(int D0, int tokens) {
  const int start = (D0 - 63) >> 6;
  return {start > 0 ? start : 0, (D0 + tokens - 1) >> 6};
}
RELATTN_HD int band_slot(int n, int half, int slots) { return (2 * n + half) % slots; }

// Is this half of chunk c stored?  Three chunks fill six slots.  Of five slots the
// oldest half and the newest would share one: the threads that write them do not
// wait for each other at an item's start, and the older might come last.  With five
// slots an item has at most 32 tokens, so that three chunks are read only where D0 is
// 33 or more past a multiple of 64, and then nothing reads the oldest half.
RELATTN_HD bool band_stored(int c, int half, int first, int slots) { return slots >= 6 || half == 1 || c > first - 2; }

}  // namespace relattn
