// One decode step over a paged cache of 8-bit codes (ssa_decode_paged_q8).
//
// With k = Ks[page, g] * code, the scale of a block is a factor of its logits, and
// the scale of V a factor of the block's share of the output:
//   x_t = (scale ks) (q . kcode_t),   O = sum_blocks vs (sum_t p_t vcode_t) / l,
// so the codes go to the tensor cores unscaled: both formats are exact in f16, and
// int8 has tiles of its own.  HBM-bound; two launches, or one for few short rows:
//   1. route: a cluster of 1 to 8 blocks a sequence and KV head (a pair) scores the
//      summaries of rows that have more candidates than are kept, and selects; rows
//      that keep every block are not scored and need no list.
//   2. split attention.  The work is cut into slices of 16 keys; block x of the
//      grid takes an equal contiguous run of all slices, whatever the sequences'
//      lengths, and each of its 12 warps an equal contiguous run of those.  A warp
//      copies its own slices into its own ring of shared memory (cp.async, 16
//      bytes a thread; 96 KB of a block's are under way) and keeps its own m, l and O,
//      so nothing is waited for across warps until the block's run is done.  A pair that
//      lies within a warp's run is written at once; the others' records are joined
//      in shared memory, and a pair that is split between blocks is finished by the
//      last of them, from the blocks' records in order.  The kernel starts while the
//      route kernel runs (programmatic dependent launch) and waits only for lists, and
//      before its end.  Until then it reads what the kernels before the call have written and
//      writes O, idx and records: that is safe because every block of the route kernel lets it in
//      only behind its own wait for those kernels.  Whatever is launched between the two has
//      to keep to that.
// Both rules on row lengths go by the table's width, as the lengths are on the device: a
// wide table takes the two kernels however short its rows.
// Measured (B200, calls back to back in a CUDA graph): 128K keys of 8 heads, d = 128, e4m3,
// read whole (0.27 GB): 54 us, of which the blocks' streams take 38 to 46 (24 of the 148 SMs
// are a tenth slower under load), start and joins the rest; 32 ragged rows of up to 16K
// keys, int8 (0.67 GB): 115 us cool, 127 under a sustained load, which meets the power limit;
// 64 rows of 65536 keys, top-32 (0.27 GB of summaries, 0.28 GB of codes): 104.8 us; one row of
// 128K keys, top-32: 18.0 us.  A first form with a barrier of all warps at every pair's end,
// the heads as the tiles' rows and a serial join took 74, 175, 138 and 39 us.
//
// Fragments.  m16n8k16 tiles, f16 in and fp32 out, with the cache as the row operand:
// S^T = K q^T has a tile's 16 rows for the slice's keys and its 8 columns for the
// group's heads, O^T = V^T P^T its rows for 16 coordinates.  So no row is idle (with
// the heads as rows half of them are), and the f16 pairs of a code word are its
// operands as they come.  P is held as the sum of two f16, 22 bits, and so is q in fp32: two
// products with one row operand and one accumulator.  q in bf16 is exact in one f16.  (P
// in one f16, 11 bits, would take a third off the tensor work, 32 ragged rows of int8 under a
// sustained load 127 -> 113 us, but an eighth of a step of the bf16 result shows in one result
// in ten and, where the values cancel, in far more than a step.)  A thread reads 16 bytes of
// a key row at a time: the order of the coordinates within a product is free, as long as
// q has the same.  The order of the keys is pi(row), chosen with the chunk swizzle so that
// neither K nor V reads have bank conflicts.  P^T is the S^T tile transposed (movmatrix).
#include "common.cuh"
#include "kernels.h"
#include "ptx.cuh"
#include "q8.cuh"
#include "select_block.cuh"

namespace ssa {

namespace {

constexpr int kQW = 12;                 // warps of the split kernel
constexpr int kQThreads = 32 * kQW;
constexpr int kSlice = 16;              // keys a slice
constexpr int kWholeSlices = 96;        // most slices of a pair that a block takes whole,
constexpr size_t kWholePairs = 148;     // and most pairs then
constexpr int kQGridMax = 160;          // most blocks of the split grid (148 SMs, one each)
constexpr int kTogether = 32;           // most slices whose sums are formed in registers alone
// Slices in flight or in use a warp: 144 KB (d = 128) or 192 KB (d = 64) a block.
__host__ __device__ constexpr int q8_stages(int d) { return d == 128 ? 3 : 8; }

// Slices of the pairs (sequence, KV head) of one sequence: s blocks, the last
// of them with `tail` keys.
__device__ __forceinline__ int pair_slices(int L, int B, int kk, int Lmax, int* blocks) {
  if (L < 1 || L > Lmax) {
    *blocks = 0;
    return 0;
  }
  const int last = (L - 1) / B;
  const int nb = min(max(last - 1, 0), kk) + (last > 0 ? 2 : 1);
  *blocks = nb;
  const int tail = L - last * B;
  return (nb - 1) * (B / kSlice) + (tail + kSlice - 1) / kSlice;
}

// a / b for whole numbers that leave an int; in 32 bits where a fits (a 64-bit division is
// a fifth of a microsecond).
__device__ __forceinline__ int quotient(long long a, int b) {
  return a >> 32 ? (int)(a / b) : (int)((uint32_t)a / (uint32_t)b);
}

// *p += v, as a release of what this thread knows written and an acquire of what others
// have released there; the old value.  (__threadfence on both sides: 0.5 us more.)
__device__ __forceinline__ int add_acq_rel(int* p, int v) {
  int old;
  asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], %2;"
               : "=r"(old)
               : "l"(p), "r"(v)
               : "memory");
  return old;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// The first `bytes` (0 or 16) from src, zeros for the rest.
__device__ __forceinline__ void cp16_part(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ uint4 lds16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(at));
  return v;
}

__device__ __forceinline__ uint2 lds8(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}

__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One m16n8k32 tile on int8 operands: c += A . B, exact.
__device__ __forceinline__ void mma32(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// |x| < 64 as d0 + 2^-7 d1 + 2^-14 d2, whole numbers up to 64: exact for a bf16 x from
// 2^-7 up, and off by at most 2^-15 below.
__device__ __forceinline__ void digits3(float x, uint32_t (&d)[3]) {
  const float a = rintf(x), y = (x - a) * 128.f, b = rintf(y), c = rintf((y - b) * 128.f);
  d[0] = (uint32_t)(int)a & 255u;
  d[1] = (uint32_t)(int)b & 255u;
  d[2] = (uint32_t)(int)c & 255u;
}

// c = A . B (no accumulator to clear).
__device__ __forceinline__ void mma16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                            uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The f16 pair of (a, b), and that of what it leaves out.
__device__ __forceinline__ void split_half2(float a, float b, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(a, b);
  const float2 f = __half22float2(h);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = half2_bits(a - f.x, b - f.y);
}

// Four outputs v * f on end.
__device__ __forceinline__ void store4(float* p, float4 v, float f) {
  *reinterpret_cast<float4*>(p) = make_float4(v.x * f, v.y * f, v.z * f, v.w * f);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v, float f) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x * f, v.y * f);
  const __nv_bfloat162 b = __floats2bfloat162_rn(v.z * f, v.w * f);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                            *reinterpret_cast<const uint32_t*>(&b));
}

// The 8 x 8 tile of 16-bit values held by the warp, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Key of row n (0 .. 7) of a tile.  Bits (n2 n1 n0) -> (n0 ^ n1, n2, n1).
__device__ __forceinline__ int key_of(int n) {
  return (((n ^ (n >> 1)) & 1) << 2) | ((n >> 2) << 1) | ((n >> 1) & 1);
}

// Byte offset of 16-byte chunk c of row r in a slice's K (or V) tile.  d = 128: the
// usual XOR with the row; d = 64 (two rows to 128 bytes): K rows r and r ^ 4, and
// V rows r and r ^ 2, must differ.
template <int D, bool V>
__device__ __forceinline__ int tile_at(int r, int c) {
  if constexpr (D == 128) return r * 128 + ((c ^ (r & 7)) << 4);
  const int x = V ? ((r >> 1) & 1) << 1 : ((r >> 2) & 1) << 2;
  return ((r * 4 + c) ^ x) << 4;
}

}  // namespace

// ---------------------------------------------------------------- 1. route
namespace {

constexpr int kListCap = 512;  // candidates that the quick selection can list

// v to the same shared word of the cluster's first block.
__device__ __forceinline__ void st_first(float* p, float v) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p), r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(a));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(r), "f"(v) : "memory");
}

// Entries of keys[u0], keys[u0 + 1], .. 4 of every `step` below n (n up to a multiple of 4,
// the rest 0), that come before key at position i: the larger ones, and the equal ones
// of a lower position.
__device__ __forceinline__ int rank_of(const uint32_t* keys, int u0, int step, int n, uint32_t key,
                                       int i) {
  int r = 0;
#pragma unroll 4
  for (int u = u0; u < n; u += step) {
    const uint4 k = *reinterpret_cast<const uint4*>(keys + u);
    r += (k.x > key || (k.x == key && u < i)) + (k.y > key || (k.y == key && u + 1 < i)) +
         (k.z > key || (k.z == key && u + 2 < i)) + (k.w > key || (k.w == key && u + 3 < i));
  }
  return r;
}

// block_select_topk with few passes over the scores, for k <= 128.  The candidates
// are dealt to 32, 64 or 128 >= k groups; T, the least of the groups' largest scores, is
// not above the k-th largest score, so whatever is selected is >= T.  The
// candidates >= T, in index order, are few (about 110 of 1000 or 2000 for k <= 32),
// and each counts those before it.  A list longer than kListCap (many equal scores)
// is left to block_select_topk.  2046 candidates, k = 32: 2.8 us (4.4 us with the
// k-th of 256 groups' maxima, found by ranking them, for T); with the chosen placed by
// rank and put in order among themselves, not by a scan over the list, 0.4 us less.
// keys: 256 + kListCap words, list: kListCap entries of shared memory.
__device__ int block_select_quick(const float* sc, int n, int k, int first, int32_t* out,
                                  uint32_t* keys, uint16_t* list, uint32_t* hist, int* sbuf) {
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (k <= 0 || k > 128 || k >= n) return block_select_topk(sc, n, k, first, out, hist, sbuf);
  uint32_t best = 0;
  for (int e = t; e < n; e += 256) best = max(best, order_key(sc[e]));
  keys[t] = best;
  __syncthreads();
  // group l: the threads l, l + groups, ...; every warp forms the minimum for itself
  const int groups = k <= 32 ? 32 : k <= 64 ? 64 : 128;
  uint32_t T = 0xffffffffu;
  for (int l = lane; l < groups; l += 32) {
    uint32_t m = 0;
    for (int u = l; u < 256; u += groups) m = max(m, keys[u]);
    T = min(T, m);
  }
  T = __reduce_min_sync(0xffffffffu, T);
  // a warp lists a contiguous run
  const int seg = ((n + 255) / 256) * 32, e0 = warp * seg, e1 = min(e0 + seg, n);
  int c = 0;
  for (int e = e0 + lane; e - lane < e1; e += 32)
    c += __popc(__ballot_sync(0xffffffffu, e < e1 && order_key(sc[e]) >= T));
  if (lane == 0) sbuf[warp] = c;
  __syncthreads();
  int pos = 0, m = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    if (w < warp) pos += sbuf[w];
    m += sbuf[w];
  }
  if (m > kListCap) {
    __syncthreads();
    return block_select_topk(sc, n, k, first, out, hist, sbuf);
  }
  uint32_t* lk = keys + 256;
  for (int e = e0 + lane; e - lane < e1; e += 32) {
    const uint32_t key = e < e1 ? order_key(sc[e]) : 0u;
    const bool in = e < e1 && key >= T;
    const uint32_t mask = __ballot_sync(0xffffffffu, in);
    if (in) {
      const int at = pos + __popc(mask & lanemask_lt());
      list[at] = (uint16_t)e;
      lk[at] = key;
    }
    pos += __popc(mask);
  }
  if (t < 4 && m + t < kListCap) lk[m + t] = 0;  // up to a multiple of 4
  __syncthreads();
  // two threads a candidate, each against half of the list; the first k by rank
  uint32_t* sel = keys;  // (the maxima have been read)
  for (int i = t >> 1; i - (t >> 1) < m; i += 128) {
    const uint32_t key = i < m ? lk[i] : 0u;
    int r = i < m ? rank_of(lk, (t & 1) * 4, 8, m, key, i) : k;
    r += __shfl_xor_sync(0xffffffffu, r, 1);
    if ((t & 1) == 0 && r < k) sel[r] = list[i];
  }
  if (t < 4) sel[k + t] = 0xffffffffu;
  __syncthreads();
  // by index
  if (t < k) {
    const uint32_t v = sel[t];
    int at = 0;
#pragma unroll 4
    for (int u = 0; u < k; u += 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(sel + u);
      at += (x.x < v) + (x.y < v) + (x.z < v) + (x.w < v);
    }
    out[at] = first + (int)v;
  }
  return k;
}

}  // namespace

// One cluster of CS blocks a (sequence, KV head); each scores a share of the
// candidates into the first block's shared memory, which then selects.  The last
// cluster sums the slices of the batch.
template <typename T, int D>
__global__ void __launch_bounds__(256, 4) q8_route_kernel(
    const T* __restrict__ q, const float* __restrict__ S, const int32_t* __restrict__ seqlens,
    int batch, int Hq, int Hkv, int Lmax, int B, int nsum, int kk, int width, int CS,
    int32_t* __restrict__ ws_idx, int* __restrict__ ws_ctr, int32_t* __restrict__ ws_off,
    T* __restrict__ O, int32_t* __restrict__ idx_out, float inv_sqrt_d) {
  constexpr int SL = D / 32;
  extern __shared__ __align__(16) float smem[];
  __shared__ int sbuf[16];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int bg = blockIdx.x / CS, rank = blockIdx.x - bg * CS;
  grid_wait();         // the kernels before
  grid_launch_next();  // the split kernel's blocks may come in as these leave
  if (bg == batch * Hkv) {
    if (rank > 0) return;
    // slices of the sequences before each, per KV head
    int base = 0;
    for (int b0 = 0; b0 < batch; b0 += 256) {
      int nb, tot;
      const int v = b0 + t < batch ? pair_slices(seqlens[b0 + t], B, kk, Lmax, &nb) : 0;
      const int off = block_excl_scan(v, sbuf, &tot);
      if (b0 + t < batch) ws_off[b0 + t] = base + off;
      base += tot;
    }
    if (t == 0) ws_off[batch] = base;
    return;
  }
  if (t == 0 && rank == 0) ws_ctr[bg] = 0;
  const int b = bg / Hkv, g = bg - (bg / Hkv) * Hkv, G = Hq / Hkv;
  const int L = seqlens[b];
  float qsum = 0.f;  // (read beside the length)
  if (kk < nsum - 2 && t < D) {
#pragma unroll 4
    for (int h = 0; h < G; ++h) qsum += (float)q[((int64_t)b * Hq + g * G + h) * D + t];
  }
  const bool valid = L >= 1 && L <= Lmax;
  const int last = valid ? (L - 1) / B : 0;
  const int n = valid ? max(last - 1, 0) : 0;  // candidates 1 .. last - 1
  if (n <= kk) {
    if (rank > 0) return;
    if (!valid) {  // no slices: nothing else writes these rows
      for (int e = t; e < G * D; e += 256) store_out(O + ((int64_t)b * Hq + g * G) * D + e, 0.f);
    }
    // every block: the list is 0 .. last, and the split pass knows it
    if (idx_out != nullptr) {
      const int c = valid ? last + 1 : 0;
      for (int p = t; p < width; p += 256) idx_out[(int64_t)bg * width + p] = p < c ? p : -1;
    }
    return;
  }
  cluster_arrive();  // every block of the cluster has begun
  float* qb = smem;                                                  // [D]
  uint32_t* hist = reinterpret_cast<uint32_t*>(qb + D);              // [256]
  uint32_t* keys = hist + 256;                                       // [256 + kListCap]
  uint16_t* list = reinterpret_cast<uint16_t*>(keys + 256 + kListCap);  // [kListCap]
  float* sc = reinterpret_cast<float*>(list + kListCap);             // [nsum]
  if (t < D) qb[t] = qsum / (float)G;
  __syncthreads();
  float qs[SL];
#pragma unroll
  for (int e = 0; e < SL; ++e) qs[e] = qb[lane * SL + e];
  cluster_wait();
  const float* Sg = S + ((int64_t)b * Hkv + g) * nsum * D + lane * SL;
  // steps of 16 candidates, dealt to the warps of all blocks
  for (int j0 = 1 + (rank * 8 + warp) * 16; kk > 0 && j0 <= n; j0 += 16 * 8 * CS) {
    float v[16];
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      const int j = min(j0 + c, n);
      float x[SL], a = 0.f;
      if constexpr (SL == 4) {
        const float4 y = __ldg(reinterpret_cast<const float4*>(Sg + (int64_t)j * D));
        x[0] = y.x; x[1] = y.y; x[2 % SL] = y.z; x[3 % SL] = y.w;
      } else {
        const float2 y = __ldg(reinterpret_cast<const float2*>(Sg + (int64_t)j * D));
        x[0] = y.x; x[1] = y.y;
      }
#pragma unroll
      for (int e = 0; e < SL; ++e) a = fmaf(x[e], qs[e], a);
      v[c] = a;
    }
    // lane l and l ^ 16 end with the sum of candidate l % 16
#pragma unroll
    for (int half = 8; half >= 1; half >>= 1) {
      const bool upper = (lane & half) != 0;
#pragma unroll
      for (int k = 0; k < half; ++k) {
        const float send = upper ? v[k] : v[k + half];
        const float keep = upper ? v[k + half] : v[k];
        v[k] = keep + __shfl_xor_sync(0xffffffffu, send, half);
      }
    }
    const float dot = v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
    if (lane < 16 && j0 + lane <= n) st_first(sc + j0 + lane - 1, dot * inv_sqrt_d);
  }
  cluster_arrive();
  cluster_wait();
  if (rank > 0) return;
  int32_t* row = ws_idx + (int64_t)bg * width;
  // the list by way of shared memory where that holds it (hist is free by then)
  int32_t* out = kk <= 128 ? reinterpret_cast<int32_t*>(hist) : row + 1;
  block_select_quick(sc, n, kk, 1, out, keys, list, hist, sbuf);
  __syncthreads();
  for (int p = t; p < width; p += 256) {
    const int j = p == 0 ? 0 : p == kk + 1 ? last : out[p - 1];
    row[p] = j;
    if (idx_out != nullptr) idx_out[(int64_t)bg * width + p] = j;
  }
}

// --------------------------------------------------------- 2. split attention
// The state of a warp, a block or the whole pair: m[G'], l[G'], o[G'][D] (log2 domain,
// o unnormalised).  Records of warps are in shared memory (G' = 8), those of blocks
// in the workspace (G' = G); a block of the grid owns two, for the pair that
// begins before its run and for the one that goes on behind it.
template <typename T, int D, int F>
__global__ void __launch_bounds__(kQThreads, 1) q8_split_kernel(
    const T* __restrict__ q, const uint8_t* __restrict__ Kp, const float* __restrict__ Ks,
    const uint8_t* __restrict__ Vp, const float* __restrict__ Vs,
    const int32_t* __restrict__ table, const int32_t* __restrict__ seqlens, int batch, int Hq,
    int Hkv, int B, int max_blocks, int num_pages, int kk, int width, int lists, int whole_pairs,
    int32_t* __restrict__ idx_out, const int32_t* __restrict__ ws_idx,
    const int32_t* __restrict__ ws_off, float* __restrict__ ws_part, int* __restrict__ ws_ctr,
    T* __restrict__ O, float scale_log2) {
  constexpr int TILE = kSlice * D;       // bytes of K (or V) of a slice
  constexpr int KS = D / 16;             // k steps of S
  constexpr int OT = D / 16;             // tiles of O^T
  constexpr int CPR = D / 16;            // 16-byte chunks of a row
  constexpr int NCP = kSlice * CPR / 32; // chunks a lane copies
  constexpr int REC = 8 * (D + 2);       // floats of a warp's record
  // P is p vs f in f16, vs the scale of V and f a power of two of each head that has the
  // largest weight p vs met so far at 2^kUp or below 2^(kUp + 1).  m (log2) and f change when p
  // passes 2^kLazy or vs f passes kMost, so P stays within 2^15.
  // Half of f16's last bit, 2^-25, is 2^-34 of the largest weight so: 16 K keys just below that
  // are 2^-20 together.  (kLazy = 8 and kUp = 4 leave 2^-29, and 2^-15.)
  constexpr float kLazy = 4.0f, kMost = 2048.0f;
  constexpr int kUp = 9;
  static_assert(kMost * 16.0f <= 32768.0f, "kMost 2^kLazy is within f16");
  constexpr int stages = q8_stages(D);
  static_assert(stages * 2 * TILE >= REC * 4, "a warp's ring holds its record");
  // the last block's room for two pairs: each m and l of all records, the threads' sums
  // and kJoinStage float4 of records
  constexpr int kJoinRoom = kQW * stages * 2 * TILE / 4;
  constexpr int kJoinStage = (kJoinRoom / 2 - 16 * kQGridMax - 8 * kQThreads) / 4;
  static_assert(kQThreads >= 8 * D / 4 && kJoinStage >= kQThreads, "PS and cap are 1 at least");
  // q against e4m3 codes, or in fp32: f16 against keys turned into f16, with a low part
  // in fp32.  q in bf16 against int8 codes: three int8 digits against the codes
  // themselves, which saves turning K (410 -> 392 instructions a slice; 32 ragged rows under a
  // sustained load, where int8 meets the power limit, 132 -> 127 us).
  // e4m3 has no such tile: the one that PTX offers here turns its operands into f16 as
  // well (9 to 12 cycles an SM quarter for k = 32 at a latency of 47, f16 8.3 for k = 16 at
  // 24), and was slower (56 -> 65 us for 128K keys).
  constexpr bool kDigits = sizeof(T) == 2 && F == SSA_I8;
  constexpr bool kLow = sizeof(T) == 4;
  extern __shared__ __align__(128) unsigned char q8_smem[];
  __shared__ int s_b, s_groups;
  __shared__ int s_pair[kQW][2];             // pair of a warp's first and last record, or -1
  __shared__ int s_list[2 * kQW];            // records in use
  __shared__ int s_from[kQW + 2], s_gpair[kQW + 1];  // a group's records in s_list, its pair
  __shared__ int s_split[2], s_first[2], s_parts[2];  // split pairs, their blocks
  __shared__ int s_last[2];                           // those that this block joins
  __shared__ int32_t s_off[kQThreads + 1];
  __shared__ uint32_t s_tmem;

  const int G = Hq / Hkv, spb = B / kSlice;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (whole_pairs && !lists) grid_wait();  // the kernels before (there is no route kernel)
  // Slices of the sequences before each, per KV head: formed here up to kQThreads
  // sequences, so that only block lists (where there are any) are waited for.
  const int32_t* off = ws_off;
  if (batch <= kQThreads) {
    int nb;
    const int v = t < batch ? pair_slices(seqlens[t], B, kk, max_blocks * B, &nb) : 0;
    int in = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, in, o);
      if (lane >= o) in += y;
    }
    if (lane == 31) s_list[warp] = in;
    __syncthreads();
    int base = 0;
#pragma unroll
    for (int w = 0; w < kQW; ++w) base += w < warp ? s_list[w] : 0;
    if (t < batch) s_off[t + 1] = base + in;
    if (t == 0) s_off[0] = 0;
    __syncthreads();
    off = s_off;
  } else {
    grid_wait();
  }
  const long long total = (long long)off[batch] * Hkv;
  // no more blocks than leave each warp a slice; the first `extra` take run + 1 slices, the
  // others run
  const int grid = total < (long long)gridDim.x * kQW ? ((int)total + kQW - 1) / kQW
                                                      : (int)gridDim.x;
  int run = 0, extra = 0;
  long long s0, s1;
  if (whole_pairs) {
    // one pair a block, with what the route kernel does where there is one
    const int pb = blockIdx.x / Hkv, per = off[pb + 1] - off[pb];
    s0 = (long long)off[pb] * Hkv + (long long)(blockIdx.x - pb * Hkv) * per;
    s1 = s0 + per;
    if (!lists) {
      const int L = per > 0 ? seqlens[pb] : 0, c = (L + B - 1) / B;
      if (idx_out != nullptr)
        for (int i = t; i < width; i += kQThreads)
          idx_out[(int64_t)blockIdx.x * width + i] = i < c ? i : -1;
      if (per == 0)
        for (int e = t; e < G * D; e += kQThreads)
          store_out(O + (int64_t)blockIdx.x * G * D + e, 0.f);
    }
    if (per == 0) {
      grid_wait();  // this kernel's end is to mean that the route kernel has ended too
      return;
    }
  } else {
    if ((int)blockIdx.x >= grid) {  // also when there is nothing at all
      grid_wait();
      return;
    }
    run = quotient(total, grid);
    extra = (int)(total - (long long)run * grid);
    s0 = (long long)blockIdx.x * run + min((int)blockIdx.x, extra);
    s1 = s0 + run + ((int)blockIdx.x < extra ? 1 : 0);
  }
  const int ns = (int)(s1 - s0);
  // the warp's run
  const int w0 = (int)((long long)warp * ns / kQW), w1 = (int)((long long)(warp + 1) * ns / kQW);

  unsigned char* ring = q8_smem + (size_t)warp * stages * 2 * TILE;  // [kQW][stages][K, V]
  float* rec0 = reinterpret_cast<float*>(q8_smem + (size_t)kQW * stages * 2 * TILE);  // [kQW][REC]
  float4* minfo = reinterpret_cast<float4*>(rec0 + kQW * REC) + warp * 8;  // [kQW][8]: rows, ks, vs

  // Sums of more than kTogether slices.  A tile's product is added to its accumulator with the
  // bits below that one's last cut off: one long sum loses a tail of small weights behind a
  // large one, and drifts down by up to a step a product (1 K slices, 16 K keys, of weights of
  // any size: 3e-4 of the result).  So after kTogether slices a warp adds what it has to its
  // sums in tensor memory and begins anew; nobody else wants that memory here, while the
  // registers and shared memory are full.  128K keys whole: 53.5 -> 54.1 us (with loads of 8
  // columns instead of 16 the fp32 form takes 0.4 us more).
  constexpr int kCols = OT * 4 + 8;  // of a warp: O, then l, m and f of two heads
  static_assert(kQW / 4 * kCols <= 128, "three warps share a quarter of the lanes");
  const bool tmem = ns > kQW * kTogether;
  if (tmem && warp == 0) {
    ptx::tmem_alloc(&s_tmem, 128);
    ptx::tmem_relinquish();
  }
  // the sequence of the block's first slice
  if (t < kQW * 2) s_pair[t >> 1][t & 1] = -1;
  for (int b0 = 0; b0 < batch; b0 += kQThreads) {
    const int b = b0 + t;
    if (b < batch && (long long)off[b] * Hkv <= s0 && (long long)off[b + 1] * Hkv > s0)
      s_b = b;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const int b_first = s_b;
  const uint32_t sums_at = tmem ? s_tmem + ((uint32_t)(warp & 3) << 21) + (warp >> 2) * kCols : 0u;
  if (lists) grid_wait();  // (else at the end: see the top for what makes that safe)

  // What a slice is: page * Hkv + g (or -1: no keys), first row | rows << 8.
  struct Slice {
    int pg, rows;
  };
  auto resolve = [&](int i) -> Slice {
    Slice r{-1, 0};
    if (i >= w1) return r;
    const long long s = s0 + i;
    int b = b_first;
    while ((long long)off[b + 1] * Hkv <= s) ++b;
    const int L = seqlens[b];
    const int per = off[b + 1] - off[b];
    const long long in = s - (long long)off[b] * Hkv;  // (all heads' slices pass 32 bits)
    const int g = quotient(in, per), k = (int)(in - (long long)g * per);
    const int e = k / spb, sub = k - e * spb;
    const int last = (L - 1) / B;
    const int j = last - 1 > kk ? ws_idx[((int64_t)b * Hkv + g) * width + e] : e;
    const int rows = min(kSlice, L - j * B - sub * kSlice);
    const int page = table[(int64_t)b * max_blocks + j];
    if (page < 0 || page >= num_pages || rows <= 0) return r;
    r.pg = page * Hkv + g;
    r.rows = sub * kSlice | rows << 8;
    return r;
  };

  // Lane l resolves the warp's slice 32 c + l, a batch ahead of its use.
  Slice cur = resolve(w0 + lane), nxt = resolve(w0 + 32 + lane);
  // A slice is 16 rows of d bytes on end: lane l copies the chunks l, l + 32, ...,
  // row l / CPR + 32 i / CPR, whose swizzle depends on i only by its parity.
  const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
  const uint32_t info_s = (uint32_t)__cvta_generic_to_shared(minfo);
  uint32_t kdst[2], vdst[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int c = lane + 32 * (i % NCP);
    kdst[i] = ring_s + tile_at<D, false>(c / CPR, c % CPR);
    vdst[i] = ring_s + TILE + tile_at<D, true>(c / CPR, c % CPR);
  }
  auto issue = [&](int n, int st) {  // the warp's n-th slice into stage st = n % stages
    if (w0 + n < w1) {
      const int pg = __shfl_sync(0xffffffffu, cur.pg, n & 31);
      const int rr = __shfl_sync(0xffffffffu, cur.rows, n & 31);
      const int rows = rr >> 8;
      if (pg >= 0) {
        const int64_t at = ((int64_t)pg * B + (rr & 255)) * D + lane * 16;
        const uint32_t so = (uint32_t)st * (2 * TILE);
        if (rows == kSlice) {
#pragma unroll
          for (int i = 0; i < NCP; ++i) {
            cp16(kdst[i & 1] + so + (i >> 1) * 1024, Kp + at + i * 512);
            cp16(vdst[i & 1] + so + (i >> 1) * 1024, Vp + at + i * 512);
          }
        } else {
          // rows past the sequence read as zeros
#pragma unroll
          for (int i = 0; i < NCP; ++i) {
            const bool in = (lane + 32 * i) / CPR < rows;
            const int64_t from = in ? at + i * 512 : at - lane * 16;
            cp16_part(kdst[i & 1] + so + (i >> 1) * 1024, Kp + from, in ? 16 : 0);
            cp16_part(vdst[i & 1] + so + (i >> 1) * 1024, Vp + from, in ? 16 : 0);
          }
        }
        if (lane < 2) cp4(info_s + st * 16 + 4 + 4 * lane, (lane ? Vs : Ks) + pg);
      }
      if (lane == 2) minfo[st].x = __int_as_float(rows);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if ((n & 31) == 31) {
      cur = nxt;
      nxt = resolve(w0 + n + 33 + lane);
    }
  };
  for (int n = 0; n < stages - 1; ++n) issue(n, n);

  const int gr = lane >> 2, tq = lane & 3;
  const int ka = key_of(gr), va = key_of(2 * tq), vb = key_of(2 * tq + 1);
  // this lane's chunks of a slice: K row ka (and 8 on; the
  // second half of a row of 128 at ^ 64), V rows va, vb (and 8 on), columns of gr
  const uint32_t k_at = ring_s + tile_at<D, false>(ka, tq);
  const uint32_t k_at2 = D == 128 ? k_at ^ 64u : k_at;
  const uint32_t v_at = ring_s + TILE + (D == 128 ? tile_at<D, true>(va, gr)
                                                  : tile_at<D, true>(va, gr >> 1) + 8 * (gr & 1));
  const uint32_t v_at2 = ring_s + TILE + (D == 128 ? tile_at<D, true>(vb, gr)
                                                   : tile_at<D, true>(vb, gr >> 1) + 8 * (gr & 1));
  // O^T: [i][e + 2 y] is head 2 tq + e, coordinate gr D / 8 + 2 i + y
  float oc[OT][4];
  int n = 0, st = 0;  // the warp's next slice and its stage
  int b = b_first;
  while (w0 + n < w1) {
    // ---- the pair at the warp's slice n
    const long long pos = s0 + w0 + n;
    while ((long long)off[b + 1] * Hkv <= pos) ++b;
    const int per = off[b + 1] - off[b];
    const int g = (int)((pos - (long long)off[b] * Hkv) / per);
    const long long pair0 = (long long)off[b] * Hkv + (long long)g * per;
    const bool begins = pair0 >= s0 + w0, ends = pair0 + per <= s0 + w1;
    const int stop = ends ? (int)(pair0 + per - s0) - w0 : w1 - w0;

    // Fragments of q: lane (gr, tq) holds coordinates 64 c + 16 tq + i of head gr.  A
    // power of two brings the head's largest coordinate into [2^kTop, 2^(kTop + 1)).
    // Digits: k step 2 c + p of 32 has i = 8 p ..; f16: k step 4 c + s
    // of 16 has i = 4 s ..
    uint32_t qa[kDigits ? 3 * (D / 32) : KS][2], ql[kLow ? KS : 1][2];
    float qscale[2];  // of heads 2 tq and 2 tq + 1; NaN for one with a NaN or infinity
    {
      constexpr int kTop = kDigits ? 5 : 14;
      float v[D / 64][16];
      uint32_t m = 0;
      const T* qp = q + ((int64_t)b * Hq + g * G + (gr < G ? gr : 0)) * D + 16 * tq;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
#pragma unroll
        for (int e = 0; e < 16; e += Vec16<T>::n) unpack16(ldg16(qp + 64 * c + e), v[c] + e, qp);
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          v[c][e] = gr < G ? v[c][e] : 0.f;
          m = max(m, __float_as_uint(v[c][e]) & 0x7fffffffu);
        }
      }
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int ex = max((int)(m >> 23) - 127 - kTop, -126);
      const float up = __uint_as_float((uint32_t)(127 - ex) << 23);
      const float back = m >= 0x7f800000u
                             ? __uint_as_float(0x7fc00000u)
                             : __uint_as_float((uint32_t)(127 + ex) << 23) * scale_log2;
      qscale[0] = __shfl_sync(0xffffffffu, back, 8 * tq);
      qscale[1] = __shfl_sync(0xffffffffu, back, 8 * tq + 4);
      if constexpr (!kDigits) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const float* x = v[ks >> 2] + 4 * (ks & 3);
          if constexpr (kLow) {
            split_half2(x[0] * up, x[1] * up, qa[ks][0], ql[ks][0]);
            split_half2(x[2] * up, x[3] * up, qa[ks][1], ql[ks][1]);
          } else {
            qa[ks][0] = half2_bits(x[0] * up, x[1] * up);
            qa[ks][1] = half2_bits(x[2] * up, x[3] * up);
          }
        }
      } else {
#pragma unroll
        for (int w = 0; w < D / 16; ++w) {  // word w & 1 of k step w >> 1
          uint32_t word[3] = {0, 0, 0};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t dg[3];
            digits3(v[w >> 2][4 * (w & 3) + e] * up, dg);
#pragma unroll
            for (int i = 0; i < 3; ++i) word[i] |= dg[i] << (8 * e);
          }
#pragma unroll
          for (int i = 0; i < 3; ++i) qa[i * (D / 32) + (w >> 1)][w & 1] = word[i];
        }
      }
    }
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    // O is kept times f; w: the largest weight so far, with m the reference of its p
    float f[2] = {1.f, 1.f}, w[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < OT; ++i) oc[i][0] = oc[i][1] = oc[i][2] = oc[i][3] = 0.f;

    bool held = false;  // tensor memory has sums of this pair
    // Adds them to the present ones, or (keep) these to them, under the present m and f.
    auto together = [&](bool keep) {
      float s[8], r[2] = {0.f, 0.f};
      if (held) {
        ptx::tmem_ld8(sums_at + OT * 4, s);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float a = s[2 + e] == m_run[e] ? 1.f : ex2(s[2 + e] - m_run[e]);
          l_run[e] = fmaf(s[e], a, l_run[e]);
          r[e] = a * f[e] * __uint_as_float(0x7f000000u - __float_as_uint(s[4 + e]));
        }
      }
#pragma unroll
      for (int i = 0; i < OT; i += 4) {
        if (held) {
          float o[16];
          ptx::tmem_ld16(sums_at + 4 * i, o);
#pragma unroll
          for (int c = 0; c < 16; ++c) oc[i + c / 4][c & 3] = fmaf(o[c], r[c & 1], oc[i + c / 4][c & 3]);
        }
        if (keep) {
#pragma unroll
          for (int j = i; j < i + 4; j += 2) {
            const float o[8] = {oc[j][0], oc[j][1], oc[j][2], oc[j][3],
                                oc[j + 1][0], oc[j + 1][1], oc[j + 1][2], oc[j + 1][3]};
            ptx::tmem_st8(sums_at + 4 * j, o);
          }
#pragma unroll
          for (int c = 0; c < 16; ++c) oc[i + c / 4][c & 3] = 0.f;
        }
      }
      if (keep) {
        const float z[8] = {l_run[0], l_run[1], m_run[0], m_run[1], f[0], f[1], 0.f, 0.f};
        ptx::tmem_st8(sums_at + OT * 4, z);
        ptx::tmem_wait_st();
        l_run[0] = l_run[1] = 0.f;
      }
      held = keep;
    };
    for (int upto = min(n + kTogether, stop);; ++n) {
      if (n == upto) {
        if (held || n < stop) together(n < stop);
        if (n == stop) break;
        upto = min(n + kTogether, stop);
      }
      issue(n + stages - 1, st == 0 ? stages - 1 : st - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(stages - 1) : "memory");
      __syncwarp();
      const float4 mi = minfo[st];
      const int rows = __float_as_int(mi.x);
      const uint32_t so = (uint32_t)st * (2 * TILE);
      if (rows > 0) {
        // S^T = K q^T of 16 keys
        float sv[4];
        if constexpr (!kDigits) {
          float se[4], sd[4];  // even and odd k steps
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const uint4 u = lds16((c == 0 ? k_at : k_at2) + so);
            const uint4 v = lds16((c == 0 ? k_at : k_at2) + so + 8 * D);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              uint32_t a0, a1, a2, a3;
              q8_to_half4<F>(s == 0 ? u.x : s == 1 ? u.y : s == 2 ? u.z : u.w, a0, a2);
              q8_to_half4<F>(s == 0 ? v.x : s == 1 ? v.y : s == 2 ? v.z : v.w, a1, a3);
              const int ks = 4 * c + s;
              if (ks == 0) mma16_first(se, a0, a1, a2, a3, qa[ks][0], qa[ks][1]);
              else if (ks == 1) mma16_first(sd, a0, a1, a2, a3, qa[ks][0], qa[ks][1]);
              else mma16(s & 1 ? sd : se, a0, a1, a2, a3, qa[ks][0], qa[ks][1]);
              if constexpr (kLow) mma16(s & 1 ? sd : se, a0, a1, a2, a3, ql[ks][0], ql[ks][1]);
            }
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) sv[e] = se[e] + sd[e];
        } else {
          int sg[3][4] = {};  // by digit
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const uint4 u = lds16((c == 0 ? k_at : k_at2) + so);
            const uint4 v = lds16((c == 0 ? k_at : k_at2) + so + 8 * D);
#pragma unroll
            for (int i = 0; i < 3; ++i) {
              const uint32_t(*w)[2] = qa + i * (D / 32) + 2 * c;
              mma32(sg[i], u.x, v.x, u.y, v.y, w[0][0], w[0][1]);
              mma32(sg[i], u.z, v.z, u.w, v.w, w[1][0], w[1][1]);
            }
          }
          // |sums of d0| <= 2^20, so 2^7 times that and the sums of d1 fit 32 bits
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sv[e] = fmaf((float)(sg[0][e] * 128 + sg[1][e]), 1.f / 128.f,
                         (float)sg[2][e] * (1.f / 16384.f));
        }
        uint32_t r[4][D / 32];  // V rows va, vb, va + 8, vb + 8: columns gr D / 8 ...
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint32_t at = (y & 1 ? v_at2 : v_at) + so + (y >> 1) * (8 * D);
          if constexpr (D == 128) {
            const uint4 w = lds16(at);
            r[y][0] = w.x; r[y][1] = w.y; r[y][2 % (D / 32)] = w.z; r[y][3 % (D / 32)] = w.w;
          } else {
            const uint2 w = lds8(at);
            r[y][0] = w.x; r[y][1] = w.y;
          }
        }
        // softmax, log2 domain: x[y][e] is key row gr + 8 y, head 2 tq + e
        float x[2][2];
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int e = 0; e < 2; ++e) x[y][e] = sv[2 * y + e] * (mi.y * qscale[e]);
        if (rows < kSlice) {
#pragma unroll
          for (int y = 0; y < 2; ++y)
            if (ka + 8 * y >= rows) x[y][0] = x[y][1] = -INFINITY;
        }
        const float c0 = fmaxf(x[0][0], x[1][0]), c1 = fmaxf(x[0][1], x[1][1]), vs = mi.z;
        if (__any_sync(0xffffffffu, c0 > m_run[0] + kLazy || c1 > m_run[1] + kLazy ||
                                        vs * f[0] > kMost || vs * f[1] > kMost)) {
          float cm[2] = {c0, c1};
#pragma unroll
          for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1)
              cm[e] = fmaxf(cm[e], __shfl_xor_sync(0xffffffffu, cm[e], o));
            const float m = fmaxf(cm[e], m_run[e]);
            const float alpha = m_run[e] == m ? 1.f : ex2(m_run[e] - m);  // 0 at first
            // (a NaN is no maximum: it marks p, not w)
            w[e] = fmaxf(w[e] * alpha, cm[e] == -INFINITY ? 0.f : ex2(cm[e] - m) * vs);
            // f = 2^kUp over w's power of two, within 2^126, so that 1 / f is exact
            const int fe = min(254 + kUp - (int)(__float_as_uint(w[e]) >> 23), 253);
            const float fn = __uint_as_float((uint32_t)fe << 23);
            const float by = alpha * fn * __uint_as_float(0x7f000000u - __float_as_uint(f[e]));
            l_run[e] *= alpha;
            f[e] = fn;
#pragma unroll
            for (int i = 0; i < OT; ++i) {  // (by <= 2: w has not fallen below alpha times itself)
              oc[i][e] *= by;
              oc[i][e + 2] *= by;
            }
            m_run[e] = m;
          }
        }
        uint32_t hi[2], lo[2];
        {
          const float m0 = m_run[0] == -INFINITY ? 0.f : m_run[0];
          const float m1 = m_run[1] == -INFINITY ? 0.f : m_run[1];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float p0 = ex2(x[y][0] - m0), p1 = ex2(x[y][1] - m1);
            l_run[0] += p0;
            l_run[1] += p1;
            split_half2(p0 * vs * f[0], p1 * vs * f[1], hi[y], lo[y]);
            hi[y] = transpose8(hi[y]);
            lo[y] = transpose8(lo[y]);
          }
        }
        // O^T += V^T P^T
#pragma unroll
        for (int w = 0; w < D / 32; ++w)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // bytes (2 h, 2 h + 1) of the rows, paired by column
            const uint32_t sel = h ? 0x7362 : 0x5140;
            uint32_t a0, a1, a2, a3;
            q8_to_half4<F>(__byte_perm(r[0][w], r[1][w], sel), a0, a1);
            q8_to_half4<F>(__byte_perm(r[2][w], r[3][w], sel), a2, a3);
            mma16(oc[2 * w + h], a0, a1, a2, a3, hi[0], hi[1]);
            mma16(oc[2 * w + h], a0, a1, a2, a3, lo[0], lo[1]);
          }
      }
      st = st == stages - 1 ? 0 : st + 1;
      __syncwarp();  // the stage is read before it is filled again
    }

    // ---- the pair's end in this warp
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l_run[e] += __shfl_xor_sync(0xffffffffu, l_run[e], o);
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float by = __uint_as_float(0x7f000000u - __float_as_uint(f[e]));  // 1 / f
#pragma unroll
      for (int i = 0; i < OT; ++i) {
        oc[i][e] *= by;
        oc[i][e + 2] *= by;
      }
    }
    const int pair = b * Hkv + g;
    if (begins && ends) {
      // nobody else has a part of it; no key at all gives zeros
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (2 * tq + e < G) {
          const float inv = l_run[e] == 0.f ? 0.f : 1.f / l_run[e];
          T* op = O + ((int64_t)b * Hq + g * G + 2 * tq + e) * D + gr * (D / 8);
#pragma unroll
          for (int i = 0; i < OT; i += 2)
            store4(op + 2 * i, make_float4(oc[i][e], oc[i][e + 2], oc[i + 1][e], oc[i + 1][e + 2]),
                   inv);
        }
    } else {
      // a pair that began before the run, or one that goes on behind it (then the
      // warp's ring is free)
      const int last = begins ? 1 : 0;
      float* rec = last ? reinterpret_cast<float*>(ring) : rec0 + warp * REC;
      if (lane == 0) s_pair[warp][last] = pair;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int h = 2 * tq + e;
        if (gr == 0) {
          rec[h] = m_run[e];
          rec[8 + h] = l_run[e];
        }
#pragma unroll
        for (int i = 0; i < OT; i += 2)
          *reinterpret_cast<float4*>(rec + 16 + h * D + gr * (D / 8) + 2 * i) =
              make_float4(oc[i][e], oc[i][e + 2], oc[i + 1][e], oc[i + 1][e + 2]);
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (tmem && warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(s_tmem, 128);
  }

  // ---- join the warps' records, pair by pair.  Record 2 w is warp w's first, 2 w + 1
  // its last; those of a pair follow one another.
  if (warp == 0) {
    const int p = lane < 2 * kQW ? s_pair[lane >> 1][lane & 1] : -1;
    const uint32_t have = __ballot_sync(0xffffffffu, p >= 0);
    const uint32_t before = have & lanemask_lt();
    const int prev = __shfl_sync(0xffffffffu, p, before ? 31 - __clz(before) : 0);
    const bool first = p >= 0 && (before == 0 || prev != p);
    const uint32_t firsts = __ballot_sync(0xffffffffu, first);
    const int k = __popc(firsts & lanemask_lt());  // groups before this lane
    if (p >= 0) s_list[__popc(before)] = lane;
    if (first) {
      s_from[k] = __popc(before);
      s_gpair[k] = p;
    }
    if (lane == 0) {
      s_groups = __popc(firsts);
      s_from[__popc(firsts)] = __popc(have);
    }
  }
  __syncthreads();
  const int groups = s_groups;
  const size_t rec_g = (size_t)G * D + 16;  // o[G][D], m[8], l[8]
  // first slice of a pair, and its number of slices
  auto pair_first = [&](int p) {
    const int pb = p / Hkv;
    return (long long)off[pb] * Hkv + (long long)(p - pb * Hkv) * (off[pb + 1] - off[pb]);
  };
  auto pair_len = [&](int p) { return off[p / Hkv + 1] - off[p / Hkv]; };
  // Only the first and the last group can go on in other blocks.
  const long long cut = (long long)extra * (run + 1);
  auto block_of = [&](long long s) {
    return s < cut ? quotient(s, run + 1) : extra + quotient(s - cut, run);
  };
  if (warp == kQW - 1 && lane < 2) {
    const int p = groups > lane ? s_gpair[lane == 0 ? 0 : groups - 1] : -1;
    bool split = false;
    if (p >= 0 && !whole_pairs) {
      const long long f = pair_first(p), e = f + pair_len(p);
      split = f < s0 || e > s1;
      if (split) {
        s_first[lane] = block_of(f);
        s_parts[lane] = block_of(e - 1) - s_first[lane] + 1;
      }
    }
    s_split[lane] = split ? p : -1;
  }
  const int E = G * (D / 4);  // float4 of a record
  for (int e = t; e < groups * E; e += kQThreads) {
    const int k = e / E, r = e - k * E;
    const int h = r / (D / 4), d4 = (r - h * (D / 4)) * 4;
    const int from = s_from[k], to = s_from[k + 1], p = s_gpair[k];
    auto at = [&](int x) {
      const int rc = s_list[x];
      const unsigned char* own = q8_smem + (size_t)(rc >> 1) * stages * 2 * TILE;
      return rc & 1 ? reinterpret_cast<const float*>(own) : rec0 + (rc >> 1) * REC;
    };
    float M = -INFINITY;
#pragma unroll 4
    for (int x = from; x < to; ++x) M = fmaxf(M, at(x)[h]);
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.f;
#pragma unroll 4
    for (int x = from; x < to; ++x) {
      const float* rc = at(x);
      // a record without keys weighs 0; one whose logits were NaN keeps its NaN
      const float a = rc[h] == -INFINITY ? 0.f : ex2(rc[h] - M);
      const float4 o = *reinterpret_cast<const float4*>(rc + 16 + h * D + d4);
      num.x = fmaf(a, o.x, num.x);
      num.y = fmaf(a, o.y, num.y);
      num.z = fmaf(a, o.z, num.z);
      num.w = fmaf(a, o.w, num.w);
      den = fmaf(a, rc[8 + h], den);
    }
    const long long f = pair_first(p);
    if (f >= s0 && f + pair_len(p) <= s1) {
      store4(O + ((int64_t)(p / Hkv) * Hq + (p % Hkv) * G + h) * D + d4, num,
             den == 0.f ? 0.f : 1.f / den);
    } else {
      float* part = ws_part + ((size_t)blockIdx.x * 2 + (f < s0 ? 0 : 1)) * rec_g;
      *reinterpret_cast<float4*>(part + h * D + d4) = num;
      if (d4 == 0) {
        part[G * D + h] = M;
        part[G * D + 8 + h] = den;
      }
    }
  }
  // ---- pairs split between blocks: the last block to arrive joins the records
  if (whole_pairs) return;
  grid_wait();  // the counters are 0 (nothing is left to wait for where lists were)
  __syncthreads();
  if (t < 2) {
    const int p = s_split[t];
    // (the barrier has put the records before this)
    s_last[t] = p >= 0 && add_acq_rel(&ws_ctr[p], 1) == s_parts[t] - 1 ? p : -1;
  }
  __syncthreads();
  // One pair for the whole block, or one for each half of it.  This runs once a launch,
  // so its instructions come from L2: short loops, and the records by way of shared
  // memory, cost less than many loads a thread in unrolled code.
  const bool two = s_last[0] >= 0 && s_last[1] >= 0;
  const int half = two && t >= kQThreads / 2 ? 1 : 0;
  const int which = two ? half : s_last[0] >= 0 ? 0 : 1, p = s_last[which];
  if (p < 0) return;
  {
    const int nt = two ? kQThreads / 2 : kQThreads, tt = t - half * (kQThreads / 2);
    const int xf = s_first[which], parts = s_parts[which];
    // the pair is the last of its first block and the first of the others
    auto record = [&](int x) {
      return ws_part + ((size_t)(xf + x) * 2 + (x == 0 ? 1 : 0)) * rec_g;
    };
    // Sum e + E y: of the records y, y + PS, ... of float4 e.  (PS, and so the order of
    // the sums, does not depend on which pairs meet here.)
    const int PS = kQThreads / E, cap = kJoinStage / E / PS * PS;
    float* ml = reinterpret_cast<float*>(q8_smem) + half * (kJoinRoom / 2);  // the rings are free
    float* sums = ml + 16 * kQGridMax;                                       // [PS][E][8]
    float4* stage = reinterpret_cast<float4*>(sums + 8 * kQThreads);         // [cap][E]
    const uint32_t ml_s = (uint32_t)__cvta_generic_to_shared(ml);
    const uint32_t stage_s = (uint32_t)__cvta_generic_to_shared(stage);
    for (int i = tt; i < parts * 4; i += nt)
      cp16(ml_s + i * 16, record(i >> 2) + G * D + (i & 3) * 4);
    // (both halves make the same number of rounds, which have barriers)
    const int most = two ? max(s_parts[0], s_parts[1]) : parts;
    for (int x0 = 0; x0 < most; x0 += cap) {
      const int n = min(cap, parts - x0);  // 0 or less: nothing is left for this half
      for (int i = tt; i < n * E; i += nt) {
        const int x = i / E;
        cp16(stage_s + i * 16, record(x0 + x) + (i - x * E) * 4);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncthreads();
      for (int it = tt; it < E * PS; it += nt) {
        const int y = it / E, e = it - y * E, h = e / (D / 4);
        float M = -INFINITY;
#pragma unroll 4
        for (int x = 0; x < parts; ++x) M = fmaxf(M, ml[x * 16 + h]);
        float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
        float den = 0.f;
        float* sm = sums + it * 8;
        if (x0 > 0) {
          num = *reinterpret_cast<const float4*>(sm);
          den = sm[4];
        }
#pragma unroll 2
        for (int x = y; x < n; x += PS) {
          const float m = ml[(x0 + x) * 16 + h], a = m == -INFINITY ? 0.f : ex2(m - M);
          const float4 o = stage[x * E + e];
          num.x = fmaf(a, o.x, num.x);
          num.y = fmaf(a, o.y, num.y);
          num.z = fmaf(a, o.z, num.z);
          num.w = fmaf(a, o.w, num.w);
          den = fmaf(a, ml[(x0 + x) * 16 + 8 + h], den);
        }
        *reinterpret_cast<float4*>(sm) = num;
        sm[4] = den;
      }
      __syncthreads();
    }
    for (int e = tt; e < E; e += nt) {
      float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
      float den = 0.f;
#pragma unroll 1
      for (int y = 0; y < PS; ++y) {
        const float* sm = sums + (y * E + e) * 8;
        const float4 v = *reinterpret_cast<const float4*>(sm);
        num.x += v.x;
        num.y += v.y;
        num.z += v.z;
        num.w += v.w;
        den += sm[4];
      }
      store4(O + ((int64_t)(p / Hkv) * Hq + (p % Hkv) * G) * D + e * 4, num,
             den == 0.f ? 0.f : 1.f / den);
    }
  }
}

Q8Plan plan_q8(int batch, int Hq, int Hkv, int d, int B, int topk, int max_blocks) {
  Q8Plan p{};
  p.kk = topk < max_blocks ? topk : max_blocks;
  p.width = p.kk + 2;
  const size_t pairs = (size_t)batch * Hkv;
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  // lists are kept for rows that leave blocks out; with topk >= the candidates of
  // the longest row there are none
  p.lists = topk < max_blocks - 2;
  // Few pairs of few slices go to a block each (of 148 SMs) and need no split: without
  // lists in one launch and without scratch.  Split and whole, us: 1 row of 100 tokens
  // (8 / 2 heads) 10.3, 8.2; of 777 (4 / 1) 14.3, 12.3; 16 rows of 1500 (32 / 8) 21.5, 16.4;
  // 24 ragged rows, top-8 blocks of 128 (8 / 4) 25.6, 22.6; but 1 row of 3000 (8 pairs)
  // 16.4, 22.5 and 64 rows of 1500 (512 pairs) 46.6, 59.4.
  const int most = max_blocks < p.width ? max_blocks : p.width;  // blocks of a pair
  p.whole = pairs <= kWholePairs && (long long)most * (B / kSlice) <= kWholeSlices;
  if (p.whole && !p.lists) return p;  // bytes = 0
  p.off_off = up(p.lists ? pairs * p.width * sizeof(int32_t) : 0);
  p.off_ctr = up(p.off_off + ((size_t)batch + 1) * sizeof(int32_t));
  p.off_part = up(p.off_ctr + pairs * sizeof(int));
  p.bytes = up(p.off_part + (size_t)kQGridMax * 2 * ((size_t)(Hq / Hkv) * d + 16) * sizeof(float));
  return p;
}

template <typename T, int D, int F>
static cudaError_t launch_q8_t(const Q8Plan& p, const void* q, const void* Kp, const float* Ks,
                               const void* Vp, const float* Vs, const float* S,
                               const int32_t* table, int max_blocks, int num_pages,
                               const int32_t* seqlens, int batch, int Hq, int Hkv, int B,
                               float scale, void* O, int32_t* idx_out, void* ws,
                               cudaStream_t st) {
  char* w = static_cast<char*>(ws);
  int32_t* ws_idx = reinterpret_cast<int32_t*>(w);
  int32_t* ws_off = reinterpret_cast<int32_t*>(w + p.off_off);
  int* ws_ctr = reinterpret_cast<int*>(w + p.off_ctr);
  float* ws_part = reinterpret_cast<float*>(w + p.off_part);
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  constexpr int stages = q8_stages(D);
  const size_t smem2 = (size_t)kQW * 8 * (D + 2) * sizeof(float) +
                       (size_t)kQW * 8 * sizeof(float4) +
                       (size_t)kQW * stages * 2 * kSlice * D;
  e = cudaFuncSetAttribute(q8_split_kernel<T, D, F>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)smem2);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto split = [&](unsigned grid, bool whole) {
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kQThreads);
    cfg.dynamicSmemBytes = smem2;
    return cudaLaunchKernelEx(&cfg, q8_split_kernel<T, D, F>, (const T*)q, (const uint8_t*)Kp, Ks,
                              (const uint8_t*)Vp, Vs, table, seqlens, batch, Hq, Hkv, B,
                              max_blocks, num_pages, p.kk, p.width, p.lists ? 1 : 0,
                              whole ? 1 : 0, idx_out, (const int32_t*)ws_idx,
                              (const int32_t*)ws_off, ws_part, ws_ctr, (T*)O,
                              scale * 1.4426950408889634f);
  };
  if (p.whole && !p.lists) return split((unsigned)(batch * Hkv), true);

  // Few pairs of long rows: several blocks score a pair's summaries, as many as
  // the GPU takes at once (2 an SM) and as leave each warp two steps of 16.
  int CS = 1;
  while (CS < 8 && batch * (long long)Hkv * CS * 2 <= 2 * sms && max_blocks >= CS * 2 * 256) CS *= 2;
  constexpr size_t fixed = D + 512 + kListCap + kListCap / 2;
  const size_t smem1 = sizeof(float) * (fixed + (size_t)max_blocks);
  if (smem1 > 47 * 1024) {  // the static arrays count too
    // (the limit is the kernel's, for all host threads: always that of the longest table)
    e = cudaFuncSetAttribute(q8_route_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)(sizeof(float) * (fixed + kQ8MaxBlocks)));
    if (e != cudaSuccess) return e;
  }
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CS;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(batch * Hkv + 1) * CS);
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = smem1;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, q8_route_kernel<T, D>, (const T*)q, S, seqlens, batch, Hq, Hkv,
                         max_blocks * B, B, max_blocks, p.kk, p.width, CS, ws_idx, ws_ctr, ws_off,
                         (T*)O, idx_out, 1.0f / sqrtf((float)D));
  if (e != cudaSuccess) return e;
  cfg.numAttrs = 1;
  return p.whole ? split((unsigned)(batch * Hkv), true)
                 : split((unsigned)(sms < kQGridMax ? sms : kQGridMax), false);
}

cudaError_t launch_decode_q8(const Q8Plan& p, const void* q, const void* Kp, const float* Ks,
                             const void* Vp, const float* Vs, ssa_qformat fmt, ssa_dtype dt,
                             const float* S, const int32_t* table, int max_blocks, int num_pages,
                             const int32_t* seqlens, int batch, int Hq, int Hkv, int d, int B,
                             float scale, void* O, int32_t* idx_out, void* ws, cudaStream_t st) {
#define SSA_DECODE_Q8(T, D, F)                                                                    \
  return launch_q8_t<T, D, F>(p, q, Kp, Ks, Vp, Vs, S, table, max_blocks, num_pages, seqlens,     \
                              batch, Hq, Hkv, B, scale, O, idx_out, ws, st)
  if (dt == SSA_BF16) {
    if (d == 128) {
      if (fmt == SSA_E4M3) SSA_DECODE_Q8(__nv_bfloat16, 128, SSA_E4M3);
      SSA_DECODE_Q8(__nv_bfloat16, 128, SSA_I8);
    }
    if (fmt == SSA_E4M3) SSA_DECODE_Q8(__nv_bfloat16, 64, SSA_E4M3);
    SSA_DECODE_Q8(__nv_bfloat16, 64, SSA_I8);
  }
  if (d == 128) {
    if (fmt == SSA_E4M3) SSA_DECODE_Q8(float, 128, SSA_E4M3);
    SSA_DECODE_Q8(float, 128, SSA_I8);
  }
  if (fmt == SSA_E4M3) SSA_DECODE_Q8(float, 64, SSA_E4M3);
  SSA_DECODE_Q8(float, 64, SSA_I8);
#undef SSA_DECODE_Q8
}

}  // namespace ssa
