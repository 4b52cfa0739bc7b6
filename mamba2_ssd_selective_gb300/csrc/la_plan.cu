// Linear attention: the table of units of packed sequences, and the words that a
// call's kernels share (status, work counters, flags) cleared in the same launch.
// One thread works a unit out from all sequences' lengths, which costs nseq reads each: a launch's latency
// for up to kLaMaxCutSeqs sequences (8 us for 24 sequences in 35 units); more are not cut.
#include "retention.h"

namespace ssd {

namespace {

constexpr int kThreads = 256;

// Thread y takes unit y in sequence order, finds its sequence and segment, and
// its place in the order by levels:
//     sum_s min(segments_s, level) + (sequences before its own with more segments than level).
__global__ void __launch_bounds__(kThreads) la_table_kernel(LaPlanDev pl, LaEntry *table, int *table_units, int nflags) {
  __shared__ int nseg[kLaMaxCutSeqs];
  const int y = blockIdx.x * kThreads + threadIdx.x, stride = gridDim.x * kThreads;
  if (y == 0) *pl.status = 0;
  if (y < kLaCounterWords) pl.counters[y] = 0;
  for (int i = y; i < nflags; i += stride) pl.flags[i] = 0;
  for (int s = threadIdx.x; s < pl.nseq; s += kThreads) {
    int a, len;
    la_seq_bounds(pl, s, a, len);
    nseg[s] = la_segments(len, pl.seg_len);
  }
  __syncthreads();
  long long n = 0;
  for (int s = 0; s < pl.nseq; ++s) n += nseg[s];
  if (n > pl.units) {
    // Only sequences that overlap have more units than there is room for: each is then taken whole, so that every
    // entry below the number of units is written and names rows of its own sequence.
    __syncthreads();
    for (int s = threadIdx.x; s < pl.nseq; s += kThreads) nseg[s] = 1;
    __syncthreads();
    n = pl.nseq;
  }
  if (y == 0) *table_units = (int)n;
  if (y >= n) return;
  int seq = 0, first = 0;
  while (first + nseg[seq] <= y) first += nseg[seq++];
  const int level = y - first;
  int at = 0, next = 0;  // places of this level and of the next
  for (int s = 0; s < pl.nseq; ++s) {
    at += min(nseg[s], level) + (s < seq && nseg[s] > level);
    next += min(nseg[s], level + 1) + (s < seq && nseg[s] > level + 1);
  }
  LaEntry e;
  e.seq = seq;
  e.level = level;
  e.nseg = nseg[seq];
  la_seq_bounds(pl, seq, e.a, e.len);
  e.next = level + 1 < nseg[seq] ? next : -1;
  table[at] = e;
}

}  // namespace

void launch_la_table(const LaPlanDev &pl, LaEntry *table, int *table_units, int nflags, cudaStream_t s) {
  long long blocks = ((long long)pl.units + kThreads - 1) / kThreads;
  if (blocks < (nflags + 4095) / 4096) blocks = (nflags + 4095) / 4096;
  la_table_kernel<<<(unsigned)blocks, kThreads, 0, s>>>(pl, table, table_units, nflags);
}

}  // namespace ssd
