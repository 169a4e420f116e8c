// The tiles of the attention over the paged 8-bit cache (dsa_kv8_tiles.cuh), for requests of their own.

#include <atomic>

#include "dsa_kv8.cuh"

namespace dsa_kv8 {
constexpr int LAUNCH_REGS = 128;   // of a thread of the tiles' kernel
}

#include "dsa_kv8_tiles.cuh"

namespace dsa_kv8 {

// How many clusters of a size the current device holds at a time: a property of the device,
// asked for once.
template <int D>
static int resident_clusters(int size) {
  constexpr int DEVICES = 64;
  static std::atomic<int> known[DEVICES][MAX_CLUSTER + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev < DEVICES && known[dev][size].load(std::memory_order_relaxed) > 0) return known[dev][size].load(std::memory_order_relaxed) - 1;
  Params P = {};
  P.n_ctas = P.cluster = size;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (configure<D, true, false>(P, cfg, attr, nullptr) != DSA_OK) return 0;
  cfg.attrs = attr + 1;   // the cluster's
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&n, tiles_kernel<D, true, false>, &cfg) != cudaSuccess) {
    cudaGetLastError();   // a size that this device cannot hold
    n = 0;
  }
  if (dev < DEVICES) known[dev][size].store(n + 1, std::memory_order_relaxed);
  return n;
}

int cluster_size(int d, long long units, int blocks) {
  if (blocks < 4) return 0;   // no two pieces of two blocks
  for (const int size : {12, 10, 8, 6, 4, 2})
    if ((size <= blocks / 2 || size == 2) && units <= (d == 128 ? resident_clusters<128>(size) : resident_clusters<64>(size)))
      return size;
  return 0;
}

int launch_tiles(int d, const Params& P, cudaStream_t st) { return launch_tiles_of<false>(d, P, st); }

}  // namespace dsa_kv8
