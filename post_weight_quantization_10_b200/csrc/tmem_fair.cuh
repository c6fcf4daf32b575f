// tmem_fair.cuh -- how many CTAs of a kernel that allocates tensor memory run at
// once, and how much shared memory such a kernel asks for.
#pragma once
#include "host.cuh"

namespace admmq {

// CTAs that run at once, one per SM, in clusters of a power of two.  Clusters do
// not straddle the GPU's processing clusters, whose sizes leave some SMs over:
// 48 clusters of three (144 CTAs) took two rounds where 48 pairs took one, and
// 32 clusters of four are the most that run together.
inline int cluster_ctas(int size, int sms) { return size <= 2 ? sms / size * size : 128; }

// Shared memory to ask for, so that blocks which fit an SM together never ask
// for more than its 512 tensor-memory columns: the CTAs of a cluster wait for
// one another, and one of them that waited for columns held by another cluster
// could close a circle.  Columns and shared memory (228 KB with 1 KB a block)
// run out together; the 40 KB keep it off the SMs of the layer solve's engine,
// whose blocks hold all columns and leave 29 KB.
inline int tmem_fair_smem(int bytes, int cols) {
  const int fair = cols * (228 * 1024 / 512) - 1024;
  if (bytes < fair) bytes = fair;
  return bytes < 40 * 1024 ? 40 * 1024 : bytes;
}

}  // namespace admmq
