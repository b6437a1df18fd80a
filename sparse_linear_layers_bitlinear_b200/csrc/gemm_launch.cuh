// Host-side launch of the CTA-pair GEMM kernel (gemm_pair.cuh), shared by the
// translation units that define configurations of it.
#pragma once

#include <mutex>

#include "gemm_pair.cuh"
#include "sbl_kernels.h"

namespace sbl {

// Pair kernels: grid = two CTAs per concurrently resident cluster, capped by
// the tile count.
template <class Cfg>
static cudaError_t pair_setup(int num_sms, int* max_clusters_out) {
  constexpr int smem = pair_smem_bytes<Cfg>();
  static_assert(smem <= 227 * 1024, "shared memory budget");
  // the attribute and the occupancy belong to a device
  static std::once_flag once[kMaxDevices];
  static cudaError_t attr_errs[kMaxDevices];
  static int max_clusters_of[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  cudaError_t& attr_err = attr_errs[dev];
  int& max_clusters = max_clusters_of[dev];
  std::call_once(once[dev], [num_sms, &attr_err, &max_clusters] {
    attr_err = cudaFuncSetAttribute(k_gemm_pair<Cfg>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (attr_err != cudaSuccess) return;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms & ~1);
    cfg.blockDim = dim3(pair_threads<Cfg>());
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    attr_err = cudaOccupancyMaxActiveClusters(&n, k_gemm_pair<Cfg>, &cfg);
    max_clusters = n;
  });
  if (attr_err != cudaSuccess) return attr_err;
  if (max_clusters <= 0) return cudaErrorInvalidConfiguration;
  *max_clusters_out = max_clusters;
  return cudaSuccess;
}

// pdl: launch with programmatic stream serialisation (the kernel's producer
// waits for the predecessor before its first load).
template <class Cfg>
static cudaError_t launch_pair(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& e,
                               const typename Cfg::Params& p, int m_rows, int n_cols, int num_sms, cudaStream_t s,
                               bool pdl = false) {
  int max_clusters = 0;
  const cudaError_t err = pair_setup<Cfg>(num_sms, &max_clusters);
  if (err != cudaSuccess) return err;
  const int tiles = ((m_rows + 255) / 256) * ((n_cols + Cfg::BN - 1) / Cfg::BN);
  const int pairs = tiles < max_clusters ? tiles : max_clusters;
  if (pairs <= 0) return cudaSuccess;
  if (pdl)
    return launch_pdl(k_gemm_pair<Cfg>, dim3(2 * pairs), dim3(pair_threads<Cfg>()), pair_smem_bytes<Cfg>(), s, a, b,
                      e, e, p);
  k_gemm_pair<Cfg><<<2 * pairs, pair_threads<Cfg>(), pair_smem_bytes<Cfg>(), s>>>(a, b, e, e, p);
  return counted(cudaGetLastError());
}

}  // namespace sbl
