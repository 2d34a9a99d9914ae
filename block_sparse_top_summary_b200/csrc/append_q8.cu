// New tokens of a ragged batch into pages of 8-bit codes.
//
// A unit is one block of one sequence that receives rows, for one KV head and for
// K or V: rows [r0, r1) of its page are new.  One block of 256 threads takes a
// unit, holds the new rows in registers (each is read once), reduces the largest
// magnitude, chooses the scale, and writes codes.  What a part-filled block held
// before is read again only when the scale grows (its codes are then rounded
// again under the larger scale) or when the block is complete and its keys'
// mean is due.
//
// Units of sequence b start at floor(cu[b] / B) + 2 b: n new tokens touch at most
// floor(n / B) + 2 blocks, so the ranges do not meet, and a block finds its
// sequence by bisection without another pass over the batch.
//
// The largest magnitude is a maximum over sign-less bits: a NaN or an infinity
// beats every finite value and marks the block by a NaN scale.
#include "common.cuh"
#include "kernels.h"
#include "q8.cuh"

namespace ssa {

namespace {

constexpr int kQ8Threads = 256;

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* f) {
  if constexpr (sizeof(T) == 2) {
    unpack16(ldg16_stream(p), f, p);
  } else {
    unpack16(ldg16_stream(p), f, p);
    unpack16(ldg16_stream(p + 4), f + 4, p);
  }
}

}  // namespace

template <typename T, int D, int F>
__global__ void __launch_bounds__(kQ8Threads) append_q8_kernel(
    uint8_t* __restrict__ Kp, float* __restrict__ Ks, uint8_t* __restrict__ Vp,
    float* __restrict__ Vs, float* __restrict__ S, const int32_t* __restrict__ slots,
    const int32_t* __restrict__ cu, const int32_t* __restrict__ seqlens, const T* __restrict__ kn,
    const T* __restrict__ vn, long long tok_stride, long long head_stride, int batch, int T_max,
    int Hkv, int B, int max_blocks, int num_pages) {
  constexpr int CPR = D / 8;             // 8-element chunks a row
  constexpr int RPS = kQ8Threads / CPR;  // rows a step of the block
  constexpr int NCH = 128 / RPS;         // most chunks a thread (B <= 128)
  __shared__ uint32_t s_max[kQ8Threads / 32];
  __shared__ float s_sum[kQ8Threads / 32][D];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int g = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const int u = blockIdx.x;

  // the sequence: the last b with floor(cu[b] / B) + 2 b <= u
  int lo = 0, hi = batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] / B + 2 * mid <= u) lo = mid;
    else hi = mid - 1;
  }
  const int b = lo;
  const int c0 = cu[b], c1 = cu[b + 1];
  const int len = seqlens[b], p0 = len - (c1 - c0);
  if (c0 < 0 || c1 <= c0 || c1 > T_max || p0 < 0) return;
  const int j = p0 / B + (u - (c0 / B + 2 * b));
  if (j < 0 || j >= max_blocks || j * B >= len) return;
  const int r0 = max(p0 - j * B, 0), r1 = min(len - j * B, B);
  const int t0 = c0 + j * B + r0 - p0;  // token of row r0
  const int slot = slots[t0];
  if (slot < 0 || slot % B != r0 || slot / B >= num_pages) return;  // refused, or not this block's
  const int page = slot / B;

  uint8_t* P = (is_v ? Vp : Kp) + ((int64_t)page * Hkv + g) * B * D;
  float* Ps = (is_v ? Vs : Ks) + (int64_t)page * Hkv + g;
  const T* x = (is_v ? vn : kn) + (int64_t)t0 * tok_stride + (int64_t)g * head_stride;
  const int cc = t % CPR, rr = t / CPR;

  float f[NCH][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int r = r0 + rr + i * RPS;
    if (r < r1) {
      load8(x + (int64_t)(r - r0) * tok_stride + cc * 8, f[i]);
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(f[i][e]) & 0x7fffffffu);
    }
  }
  const float old = r0 > 0 ? *Ps : 0.f;
  m = __reduce_max_sync(0xffffffffu, m);
  if (lane == 0) s_max[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kQ8Threads / 32; ++w) m = max(m, s_max[w]);
  const bool nan = m >= 0x7f800000u || old != old;
  const float scale = nan ? __uint_as_float(0x7fc00000u) : fmaxf(old, q8_scale<F>(m));
  if (t == 0) *Ps = scale;
  // scales are powers of two, so the product with the reciprocal is x / scale
  const float inv = nan ? 0.f : 1.f / scale;
  const bool mean = !is_v && S != nullptr && r1 == B;
  float sum[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = 0.f;
  auto put = [&](int r, float* y) {
    const uint2 c = q8_pack8<F>(y);
    *reinterpret_cast<uint2*>(P + (int64_t)r * D + cc * 8) = c;
    if (mean) {
      float v[8];
      q8_unpack8<F>(c, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += v[e];
    }
  };
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int r = r0 + rr + i * RPS;
    if (r < r1) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[i][e] = nan ? 0.f : f[i][e] * inv;
      put(r, f[i]);
    }
  }
  // the rows that the block held before
  const bool grown = r0 > 0 && !nan && scale > old;
  if (grown || (mean && r0 > 0)) {
    const float ratio = grown ? old * inv : 1.f;
    for (int r = rr; r < r0; r += RPS) {
      float y[8];
      q8_unpack8<F>(*reinterpret_cast<const uint2*>(P + (int64_t)r * D + cc * 8), y);
      if (grown) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= ratio;
        put(r, y);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] += y[e];
      }
    }
  }
  if (!mean) return;
  // mean of the B held rows: lanes of one column chunk, then the warps
#pragma unroll
  for (int o = CPR; o < 32; o <<= 1)
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], o);
  if (lane < CPR) {
#pragma unroll
    for (int e = 0; e < 8; ++e) s_sum[warp][lane * 8 + e] = sum[e];
  }
  __syncthreads();
  if (t < D) {
    float a = 0.f;
#pragma unroll
    for (int w = 0; w < kQ8Threads / 32; ++w) a += s_sum[w][t];
    S[(((int64_t)b * Hkv + g) * max_blocks + j) * D + t] = a * (scale / (float)B);
  }
}

template <typename T, int D, int F>
static cudaError_t launch_append_q8_t(void* Kp, float* Ks, void* Vp, float* Vs, float* S,
                                      const int32_t* slots, const int32_t* cu,
                                      const int32_t* seqlens, const void* kn, const void* vn,
                                      long long tok_stride, long long head_stride, int batch,
                                      int T_max, int Hkv, int B, int max_blocks, int num_pages,
                                      cudaStream_t st) {
  const dim3 grid((unsigned)(T_max / B + 2 * batch), (unsigned)(2 * Hkv));
  append_q8_kernel<T, D, F><<<grid, kQ8Threads, 0, st>>>(
      (uint8_t*)Kp, Ks, (uint8_t*)Vp, Vs, S, slots, cu, seqlens, (const T*)kn, (const T*)vn,
      tok_stride, head_stride, batch, T_max, Hkv, B, max_blocks, num_pages);
  return cudaGetLastError();
}

cudaError_t launch_append_q8(void* Kp, float* Ks, void* Vp, float* Vs, ssa_qformat fmt, float* S,
                             const int32_t* slots, const int32_t* cu, const int32_t* seqlens,
                             const void* kn, const void* vn, ssa_dtype dt, long long tok_stride,
                             long long head_stride, int batch, int T_max, int Hkv, int d, int B,
                             int max_blocks, int num_pages, cudaStream_t st) {
#define SSA_APPEND_Q8(T, D, F)                                                                    \
  return launch_append_q8_t<T, D, F>(Kp, Ks, Vp, Vs, S, slots, cu, seqlens, kn, vn, tok_stride,   \
                                     head_stride, batch, T_max, Hkv, B, max_blocks, num_pages, st)
  if (dt == SSA_BF16) {
    if (d == 128) {
      if (fmt == SSA_E4M3) SSA_APPEND_Q8(__nv_bfloat16, 128, SSA_E4M3);
      SSA_APPEND_Q8(__nv_bfloat16, 128, SSA_I8);
    }
    if (fmt == SSA_E4M3) SSA_APPEND_Q8(__nv_bfloat16, 64, SSA_E4M3);
    SSA_APPEND_Q8(__nv_bfloat16, 64, SSA_I8);
  }
  if (d == 128) {
    if (fmt == SSA_E4M3) SSA_APPEND_Q8(float, 128, SSA_E4M3);
    SSA_APPEND_Q8(float, 128, SSA_I8);
  }
  if (fmt == SSA_E4M3) SSA_APPEND_Q8(float, 64, SSA_E4M3);
  SSA_APPEND_Q8(float, 64, SSA_I8);
#undef SSA_APPEND_Q8
}

}  // namespace ssa
