// Block-wide top-k selection and the warp butterfly of the decode routing kernels
// (blocks of 256 threads).
#pragma once

#include "common.cuh"

namespace ssa {

// Butterfly over 32 values a lane: lane l returns the sum over the lanes of v[l].
__device__ __forceinline__ float reduce32_transpose(float (&v)[32]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int half = 16; half >= 1; half >>= 1) {
    const bool upper = (lane & half) != 0;
#pragma unroll
    for (int k = 0; k < half; ++k) {
      const float send = upper ? v[k] : v[k + half];
      const float keep = upper ? v[k + half] : v[k];
      v[k] = keep + __shfl_xor_sync(0xffffffffu, send, half);
    }
  }
  return v[0];
}

// Exclusive prefix sum of one int per thread over a 256-thread block.
__device__ __forceinline__ int block_excl_scan(int v, int* wsum, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    const int x = wsum[w];
    base += (w < warp) ? x : 0;
    all += x;
  }
  __syncthreads();
  *total = all;
  return base + incl - v;
}

// Top-k by all 256 threads of the block over n scores in shared memory; same
// result as warp_select_topk: the k highest scores, equal scores going to the
// lower index, written ascending as first + e to out[0 ..).  4-pass MSB-first
// radix select (8 bits per pass) on a shared histogram, then an index-ordered
// compaction (block scans) of the keys above the threshold and the first
// `need` keys equal to it.  Returns the number written.
static __device__ int block_select_topk(const float* sc, int n, int k, int first, int32_t* out,
                                 uint32_t* hist, int* sbuf) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (k <= 0 || n <= 0) return 0;
  if (k >= n) {
    for (int e = t; e < n; e += 256) out[e] = first + e;
    return n;
  }
  uint32_t prefix = 0, pmask = 0;
  int need = k;
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    hist[t] = 0;
    __syncthreads();
    for (int e = t; e < n; e += 256) {
      const uint32_t key = order_key(sc[e]);
      if ((key & pmask) == prefix) atomicAdd(&hist[(key >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (warp == 0) {
      uint32_t c[8], local = 0;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        c[q] = hist[255 - (lane * 8 + q)];
        local += c[q];
      }
      uint32_t incl = local;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const uint32_t excl = incl - local;
      if (excl < (uint32_t)need && (uint32_t)need <= incl) {
        uint32_t run = excl;
        for (int q = 0; q < 8; ++q) {
          if (run + c[q] >= (uint32_t)need) {
            sbuf[8] = 255 - (lane * 8 + q);
            sbuf[9] = (int)run;
            break;
          }
          run += c[q];
        }
      }
    }
    __syncthreads();
    prefix |= (uint32_t)sbuf[8] << shift;
    pmask |= 255u << shift;
    need -= sbuf[9];
    __syncthreads();
  }
  // index-ordered compaction: thread t owns the contiguous range [e0, e1)
  const int per = (n + 255) / 256;
  const int e0 = min(t * per, n), e1 = min(e0 + per, n);
  int neq = 0;
  for (int e = e0; e < e1; ++e) neq += (order_key(sc[e]) == prefix);
  int total;
  int eqr = block_excl_scan(neq, sbuf, &total);
  int ntake = 0;
  for (int e = e0; e < e1; ++e) {
    const uint32_t key = order_key(sc[e]);
    if (key > prefix) ++ntake;
    else if (key == prefix) ntake += (eqr++ < need);
  }
  int pos = block_excl_scan(ntake, sbuf, &total);
  eqr = block_excl_scan(neq, sbuf, &total);  // recompute this thread's equal-key rank base
  for (int e = e0; e < e1; ++e) {
    const uint32_t key = order_key(sc[e]);
    bool take = key > prefix;
    if (key == prefix) take = (eqr++ < need);
    if (take) out[pos++] = first + e;
  }
  return k;
}

}  // namespace ssa
