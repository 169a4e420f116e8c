// Latent rows read back from the cache (include/dsa_kv_gather.h).
//
// What bounds it: memory, 656 bytes in and 1152 out a row (24 contexts, 105 k rows, 190 MB: 33.3 us, 5.7 TB/s,
// 0.84 of a copy).  A warp has ROWS neighbouring rows of the output.  Its lanes first find the rows' places
// in the pool, a lane for each (a search in cu_rows, then the table entry), and then the warp moves the
// rows, their loads in flight together.  Lane l takes codes 8 l .. 8 l + 7 of each half of the 512, so that
// loads and stores of a warp are contiguous.  Rows of a warp, us: 2 33.3, 4 34.0, 8 34.5, 16 35.4 (8 at a
// time).

#include <cuda_runtime.h>
#include <stdint.h>

#include "device.cuh"
#include "dsa_kv_gather.h"
#include "ptx_sm103.cuh"

namespace dsa_gather {

constexpr int WARPS = 8;
constexpr int ROWS = 2;          // of a warp
constexpr int ROW_BYTES = 656;

struct Params {
  const uint8_t* pool;
  long long n_rows, table_ld, ld;
  const int32_t *table, *cu, *lens;
  uint16_t* out;
  uint32_t* status;
  int cols, page, n_req, n_out;
};

__device__ __forceinline__ uint32_t bf16x2(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
// 8 codes times their scale
__device__ __forceinline__ uint4 dequantise(uint2 codes, float scale) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = dsa::e4m3x2_to_f16x2(((i < 2 ? codes.x : codes.y) >> (16 * (i & 1))) & 0xFFFFu);
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
    o[i] = bf16x2(v.x * scale, v.y * scale);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__global__ void __launch_bounds__(32 * WARPS) gather_kernel(const __grid_constant__ Params P) {
  const int lane = threadIdx.x & 31;
  const long long first = ((long long)blockIdx.x * WARPS + (threadIdx.x >> 5)) * ROWS;
  constexpr long long LEAVE = -1, ZERO = -2;
  long long from = LEAVE;
  if (lane < ROWS && first + lane < P.n_out) {
    const int t = (int)(first + lane);
    auto cu = [&](int r) { return min(max(__ldg(P.cu + r), 0), P.n_out); };
    // the request with cu[lo] <= t < cu[lo + 1]: the last one that begins at or before t
    int lo = 0, hi = P.n_req;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (cu(mid) <= t) lo = mid; else hi = mid;
    }
    if (t >= cu(lo) && t < cu(lo + 1)) {
      const int i = t - cu(lo);
      if (!P.lens || i < __ldg(P.lens + lo)) {
        const int col = i / P.page;
        const int page = col < P.cols ? __ldg(P.table + lo * P.table_ld + col) : -1;
        from = (long long)page * P.page + (i - col * P.page);
        if (page < 0 || from >= P.n_rows) {
          from = ZERO;
          if (P.status) atomicOr(P.status, DSA_STATUS_SLOT_OUT_OF_RANGE);
        }
      }
    }
  }
  uint2 codes[ROWS][2];
  float scale[ROWS][2];
  uint32_t rope[ROWS];
  long long src[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    src[r] = __shfl_sync(0xFFFFFFFFu, from, r);
    codes[r][0] = codes[r][1] = make_uint2(0u, 0u);
    scale[r][0] = scale[r][1] = 0.f;
    rope[r] = 0u;
    if (src[r] < 0) continue;
    const uint8_t* row = P.pool + src[r] * ROW_BYTES;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      codes[r][h] = dsa::ldg_nc_v2(row + 256 * h + 8 * lane);
      scale[r][h] = __ldg(reinterpret_cast<const float*>(row + 512) + 2 * h + (lane >> 4));
    }
    rope[r] = __ldg(reinterpret_cast<const uint32_t*>(row + 528) + lane);
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    if (src[r] == LEAVE) continue;
    uint16_t* dst = P.out + (first + r) * P.ld;
#pragma unroll
    for (int h = 0; h < 2; ++h) *reinterpret_cast<uint4*>(dst + 256 * h + 8 * lane) = dequantise(codes[r][h], scale[r][h]);
    reinterpret_cast<uint32_t*>(dst + 512)[lane] = rope[r];
  }
}

static bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

}  // namespace dsa_gather

extern "C" int dsa_kv_gather(const void* pool, int64_t n_rows, const int32_t* block_table, int64_t table_ld,
                             int32_t table_cols, int32_t page_size, const int32_t* cu_rows, const int32_t* lens,
                             int32_t n_req, void* out, int64_t ld, int32_t n_out, uint32_t* status, void* stream) {
  using namespace dsa_gather;
  if (n_rows < 0 || n_req < 0 || n_out < 0 || table_cols < 0 || page_size < 1 || ld < 576 || ld % 8 != 0 ||
      (status && !aligned(status, 4)))
    return DSA_ERR_INVALID_ARG;
  if (n_req == 0 || n_out == 0) return DSA_OK;
  if (!cu_rows || !out || !aligned(cu_rows, 4) || !aligned(out, 16) || (lens && !aligned(lens, 4)) ||
      (n_rows > 0 && (!pool || !aligned(pool, 16))) ||
      (table_cols > 0 && (!block_table || !aligned(block_table, 4) || (n_req > 1 && table_ld < table_cols))))
    return DSA_ERR_INVALID_ARG;
  int sms = 0;
  const int device_rc = dsa::gb300_sms(&sms);
  if (device_rc != DSA_OK) return device_rc;
  Params P;
  P.pool = static_cast<const uint8_t*>(pool);
  P.n_rows = (long long)n_rows;
  P.table_ld = (long long)table_ld;
  P.ld = (long long)ld;
  P.table = block_table;
  P.cu = cu_rows;
  P.lens = lens;
  P.out = static_cast<uint16_t*>(out);
  P.status = status;
  P.cols = table_cols;
  P.page = page_size;
  P.n_req = n_req;
  P.n_out = n_out;
  const unsigned grid = (unsigned)(((long long)n_out + WARPS * ROWS - 1) / (WARPS * ROWS));
  gather_kernel<<<grid, 32 * WARPS, 0, (cudaStream_t)stream>>>(P);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
