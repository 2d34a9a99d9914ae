// One decode step over a paged cache of 8-bit codes (ssa_decode_paged_q8).
//
// With k = Ks[page, g] * code, the scale of a block is a factor of its logits, and
// the scale of V a factor of the block's share of the output:
//   x_t = (scale ks) (q . kcode_t),   O = sum_blocks vs (sum_t p_t vcode_t) / l,
// so the codes go to the tensor cores as they are: both formats are exact in f16.
// HBM-bound; two launches:
//   1. route (one block per sequence and KV head, and one that sums the slices of
//      the batch): scores the summaries of rows that have more candidates than
//      are kept and writes their block lists; rows that keep every block are not
//      scored and need no list.
//   2. split attention.  The work is cut into slices of 16 keys; block x of the
//      grid takes an equal contiguous run of all slices, whatever the sequences'
//      lengths, and its warps take the run's slices in turn.  Each warp copies its
//      own slices into its own ring of shared memory (cp.async, 16 bytes a
//      thread), so nothing is waited for across warps but at the end of a
//      sequence and head, where the warps' states (m, l, O) are joined.  A
//      sequence and head that is split between blocks is finished by the last of
//      them, from the blocks' partial records in order.
//
// Fragments.  m16n8k16 tiles, f16 in and fp32 out: rows 0-7 are the group's query
// heads, rows 8-15 the same heads' low parts, so that q (fp32) and P are held as
// the sum of two f16, 22 bits, at no further cost.  A thread reads 16 bytes of
// a key row at a time: the tile's k index runs over the coordinates in an order of
// our choosing, the same for q.  The key order of a tile is pi(n), chosen with the
// chunk swizzle so that neither K nor V reads have bank conflicts.
#include "common.cuh"
#include "kernels.h"
#include "q8.cuh"
#include "select_block.cuh"

namespace ssa {

namespace {

constexpr int kQW = 12;                 // warps of the split kernel
constexpr int kQThreads = 32 * kQW;
constexpr int kSlice = 16;              // keys a slice
constexpr int kQGridMax = 512;

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

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                      uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// Key of a tile's column n.  Bits (n2 n1 n0) -> (n0 ^ n1, n2, n1).
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
template <typename T, int D>
__global__ void __launch_bounds__(256, 2) q8_route_kernel(
    const T* __restrict__ q, const float* __restrict__ S, const int32_t* __restrict__ seqlens,
    int batch, int Hq, int Hkv, int Lmax, int B, int nsum, int kk, int width,
    int32_t* __restrict__ ws_idx, int* __restrict__ ws_ctr, int32_t* __restrict__ ws_off,
    T* __restrict__ O, int32_t* __restrict__ idx_out, float inv_sqrt_d) {
  constexpr int SL = D / 32;
  extern __shared__ __align__(16) float smem[];
  __shared__ int sbuf[16];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int bg = blockIdx.x;
  if (bg == batch * Hkv) {
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
  if (t == 0) ws_ctr[bg] = 0;
  const int b = bg / Hkv, g = bg - (bg / Hkv) * Hkv, G = Hq / Hkv;
  const int L = seqlens[b];
  const bool valid = L >= 1 && L <= Lmax;
  const int last = valid ? (L - 1) / B : 0;
  const int n = valid ? max(last - 1, 0) : 0;  // candidates 1 .. last - 1
  if (!valid) {  // no slices: nothing else writes these rows
    for (int e = t; e < G * D; e += 256) store_out(O + ((int64_t)b * Hq + g * G) * D + e, 0.f);
  }
  if (n <= kk) {
    // every block: the list is 0 .. last, and the split pass knows it
    if (idx_out != nullptr) {
      const int c = valid ? last + 1 : 0;
      for (int p = t; p < width; p += 256) idx_out[(int64_t)bg * width + p] = p < c ? p : -1;
    }
    return;
  }
  float* qb = smem;                                      // [D]
  uint32_t* hist = reinterpret_cast<uint32_t*>(qb + D);  // [256]
  float* sc = reinterpret_cast<float*>(hist + 256);      // [nsum]
  if (t < D) {
    float s = 0.f;
    for (int h = 0; h < G; ++h) s += (float)q[((int64_t)b * Hq + g * G + h) * D + t];
    qb[t] = s / (float)G;
  }
  __syncthreads();
  float qs[SL];
#pragma unroll
  for (int e = 0; e < SL; ++e) qs[e] = qb[lane * SL + e];
  const float* Sg = S + ((int64_t)b * Hkv + g) * nsum * D + lane * SL;
  for (int j0 = 1 + warp * 32; j0 <= n; j0 += 32 * 8) {
    float v[32];
#pragma unroll
    for (int c = 0; c < 32; ++c) {
      const int j = min(j0 + c, n);
      float x[SL], a = 0.f;
      if constexpr (SL == 4) {
        const float4 y = __ldg(reinterpret_cast<const float4*>(Sg + (int64_t)j * D));
        x[0] = y.x; x[1] = y.y; x[2 % SL] = y.z; x[3 % SL] = y.w;
      } else {
        const float2 y = __ldg(reinterpret_cast<const float2*>(Sg + (int64_t)j * D));
        x[0] = y.x; x[1 % SL] = y.y;
      }
#pragma unroll
      for (int e = 0; e < SL; ++e) a = fmaf(x[e], qs[e], a);
      v[c] = a;
    }
    const float dot = reduce32_transpose(v);
    if (j0 + lane <= n) sc[j0 + lane - 1] = dot * inv_sqrt_d;
  }
  __syncthreads();
  int32_t* row = ws_idx + (int64_t)bg * width;
  block_select_topk(sc, n, kk, 1, row + 1, hist, sbuf);
  if (t == 0) {
    row[0] = 0;
    row[kk + 1] = last;
  }
  if (idx_out != nullptr) {
    __syncthreads();
    for (int p = t; p < width; p += 256) idx_out[(int64_t)bg * width + p] = row[p];
  }
}

// --------------------------------------------------------- 2. split attention
// Partial record: m[G], l[G], o[G][D] (log2 domain, o unnormalised); a block of the
// grid owns two, for the pair that begins before its run and for the one that goes
// on behind it.
template <typename T, int D, int F>
__global__ void __launch_bounds__(kQThreads, 1) q8_split_kernel(
    const T* __restrict__ q, const uint8_t* __restrict__ Kp, const float* __restrict__ Ks,
    const uint8_t* __restrict__ Vp, const float* __restrict__ Vs,
    const int32_t* __restrict__ table, const int32_t* __restrict__ seqlens, int batch, int Hq,
    int Hkv, int B, int max_blocks, int num_pages, int kk, int width, int stages, int min_slices,
    const int32_t* __restrict__ ws_idx, const int32_t* __restrict__ ws_off,
    float* __restrict__ ws_part, int* __restrict__ ws_ctr, T* __restrict__ O, float scale_log2) {
  constexpr int TILE = kSlice * D;       // bytes of K (or V) of a slice
  constexpr int KS = D / 16;             // k steps of S
  constexpr int ON = D / 8;              // column tiles of O
  constexpr int CPR = D / 16;            // 16-byte chunks of a row
  constexpr int NCP = kSlice * CPR / 32; // chunks a lane copies
  constexpr float kLazy = 8.0f;          // O is rescaled when the maximum grows by more
  extern __shared__ __align__(128) unsigned char q8_smem[];
  __shared__ int s_last, s_b;

  const int G = Hq / Hkv, Lmax = max_blocks * B, spb = B / kSlice;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const long long total = (long long)ws_off[batch] * Hkv;
  // no more blocks than leave each some slices
  const long long most = (total + min_slices - 1) / min_slices;
  const long long grid = most < gridDim.x ? most : gridDim.x;
  if (blockIdx.x >= grid) return;  // also when there is nothing at all
  const long long s0 = blockIdx.x * total / grid, s1 = (blockIdx.x + 1) * total / grid;
  const int ns = (int)(s1 - s0);

  uint4* qf = reinterpret_cast<uint4*>(q8_smem);                         // [KS][32]
  float* qx = reinterpret_cast<float*>(q8_smem + KS * 32 * 16);          // [8]
  float* mw = qx + 8;                                                    // [kQW][8]
  float* lw = mw + kQW * 8;                                              // [kQW][8]
  float* ow = lw + kQW * 8;                                              // [kQW][8][D]
  float4* meta = reinterpret_cast<float4*>(ow + kQW * 8 * D);            // [kQW][stages]
  unsigned char* ring0 = reinterpret_cast<unsigned char*>(meta + kQW * 8);
  unsigned char* ring = ring0 + (size_t)warp * stages * 2 * TILE;
  float4* minfo = meta + warp * 8;

  // the sequence of slice s: the last b with off[b] Hkv <= s
  if (t == 0) s_b = 0;
  __syncthreads();
  for (int b0 = 0; b0 < batch; b0 += kQThreads) {
    const int b = b0 + t;
    const bool in = b < batch && (long long)ws_off[b] * Hkv <= s0 &&
                    (long long)ws_off[b + 1] * Hkv > s0;
    if (in) s_b = b;
  }
  __syncthreads();
  const int b_first = s_b;

  // What a slice is: pair, page * Hkv + g (or -1), first row, rows.
  struct Slice {
    int pg, row, rows;
    float ks, vs;
  };
  auto resolve = [&](int i) -> Slice {
    Slice r{-1, 0, 0, 0.f, 0.f};
    if (i >= ns) return r;
    const long long s = s0 + i;
    int b = b_first;
    while ((long long)ws_off[b + 1] * Hkv <= s) ++b;
    const int L = seqlens[b];
    const int per = ws_off[b + 1] - ws_off[b];
    const int in = (int)(s - (long long)ws_off[b] * Hkv);
    const int g = in / per, k = in - g * per;
    const int e = k / spb, sub = k - e * spb;
    const int last = (L - 1) / B;
    const int j = last - 1 > kk ? ws_idx[((int64_t)b * Hkv + g) * width + e] : e;
    const int rows = min(kSlice, L - j * B - sub * kSlice);
    const int page = table[(int64_t)b * max_blocks + j];
    if (page < 0 || page >= num_pages || rows <= 0) return r;  // no page: no keys
    r.pg = page * Hkv + g;
    r.row = sub * kSlice;
    r.rows = rows;
    r.ks = Ks[r.pg];
    r.vs = Vs[r.pg];
    return r;
  };

  // Warp w takes slices w, w + kQW, ...; lane l resolves the warp's slice 32 c + l.
  Slice cur = resolve(warp + lane * kQW), nxt = resolve(warp + (32 + lane) * kQW);
  auto issue = [&](int n) {  // the warp's n-th slice into stage n % stages
    if (warp + n * kQW < ns) {
      const int src = n & 31;
      const int pg = __shfl_sync(0xffffffffu, cur.pg, src);
      const int row = __shfl_sync(0xffffffffu, cur.row, src);
      const int rows = __shfl_sync(0xffffffffu, cur.rows, src);
      const float ks = __shfl_sync(0xffffffffu, cur.ks, src);
      const float vs = __shfl_sync(0xffffffffu, cur.vs, src);
      const int st = n % stages;
      if (rows > 0) {
        const uint32_t dk = (uint32_t)__cvta_generic_to_shared(ring + (size_t)st * 2 * TILE);
        const int64_t base = ((int64_t)pg * B + row) * D;
#pragma unroll
        for (int i = 0; i < NCP; ++i) {
          const int c = lane + 32 * i, r = c / CPR, cc = c % CPR;
          // rows past the sequence read as zeros
          const int64_t src_at = base + (r < rows ? r : 0) * D + cc * 16;
          const int bytes = r < rows ? 16 : 0;
          cp16(dk + tile_at<D, false>(r, cc), Kp + src_at, bytes);
          cp16(dk + TILE + tile_at<D, true>(r, cc), Vp + src_at, bytes);
        }
      }
      if (lane == 0) minfo[st] = make_float4(__int_as_float(rows), ks, vs, 0.f);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if ((n & 31) == 31) {
      cur = nxt;
      nxt = resolve(warp + (n + 33 + lane) * kQW);
    }
  };
  for (int n = 0; n < stages - 1; ++n) issue(n);

  const int gr = lane >> 2, tq = lane & 3;
  const int key0 = key_of(gr);                 // K row of this lane (tile 0)
  const int va = key_of(2 * tq), vb = key_of(2 * tq + 1);
  float oc[ON][2];
  int n = 0;  // the warp's next slice

  int b = b_first;
  long long pos = s0;
  while (pos < s1) {
    // ---- the pair at slice pos
    while ((long long)ws_off[b + 1] * Hkv <= pos) ++b;
    const int per = ws_off[b + 1] - ws_off[b];
    const int g = (int)((pos - (long long)ws_off[b] * Hkv) / per);
    const long long pair0 = (long long)ws_off[b] * Hkv + (long long)g * per;
    const long long pair1 = pair0 + per;
    const long long end = pair1 < s1 ? pair1 : s1;
    // its queries: a power of two brings each head's largest coordinate into
    // [2^14, 2^15), and two f16 hold the rest
    __syncthreads();  // the last pair's q and merge buffers are free
    if (warp < 8) {
      float v[D / 32], m = 0.f;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) {
        v[e] = warp < G ? (float)q[((int64_t)b * Hq + g * G + warp) * D + lane + 32 * e] : 0.f;
        m = fmaxf(m, fabsf(v[e]));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      int ex = (int)(__float_as_uint(m) >> 23) - 127 - 14;
      ex = max(ex, -126);
      const float up = __uint_as_float((uint32_t)(127 - ex) << 23);
      if (lane == 0) qx[warp] = __uint_as_float((uint32_t)(127 + ex) << 23) * scale_log2;
      // coordinate dd = 64 c + 16 tq' + 4 s + i of head h: k step 4 c + s, lane
      // 4 h + tq', half i of the pair of words (a0, a2)
#pragma unroll
      for (int e = 0; e < D / 32; ++e) {
        const int dd = lane + 32 * e;
        const int ks = (dd >> 6) * 4 + ((dd >> 2) & 3), ln = warp * 4 + ((dd >> 4) & 3);
        const float y = v[e] * up;
        const __half hi = __float2half_rn(y);
        const __half lo = __float2half_rn(y - __half2float(hi));
        __half* w = reinterpret_cast<__half*>(qf + ks * 32 + ln);
        const int i = dd & 3;
        w[(i >> 1) * 4 + (i & 1)] = hi;       // a0 or a2
        w[(i >> 1) * 4 + 2 + (i & 1)] = lo;   // a1 or a3
      }
    }
    __syncthreads();
    const float qscale = qx[gr];
    float m_run = -INFINITY, l_run = 0.f;
#pragma unroll
    for (int i = 0; i < ON; ++i) oc[i][0] = oc[i][1] = 0.f;

    for (; s0 + warp + (long long)n * kQW < end; ++n) {
      issue(n + stages - 1);
      if (stages == 8) asm volatile("cp.async.wait_group 7;" ::: "memory");
      else if (stages == 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
      else asm volatile("cp.async.wait_group 2;" ::: "memory");
      __syncwarp();
      const int st = n % stages;
      const float4 mi = minfo[st];
      const int rows = __float_as_int(mi.x);
      const unsigned char* kt = ring + (size_t)st * 2 * TILE;
      const unsigned char* vt = kt + TILE;
      if (rows > 0) {
        // S = q . K^T of 16 keys
        float sc[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x) sc[x][0] = sc[x][1] = sc[x][2] = sc[x][3] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          uint4 w[2];
#pragma unroll
          for (int x = 0; x < 2; ++x)
            w[x] = *reinterpret_cast<const uint4*>(kt + tile_at<D, false>(key0 + 8 * x, 4 * c + tq));
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const uint4 a = qf[(4 * c + s) * 32 + lane];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint32_t b0, b1;
              q8_to_half4<F>(s == 0 ? w[x].x : s == 1 ? w[x].y : s == 2 ? w[x].z : w[x].w, b0, b1);
              mma16(sc[x], a.x, a.y, a.z, a.w, b0, b1);
            }
          }
        }
        // softmax over the row's keys, log2 domain
        const float f = mi.y * qscale;
        float cm = -INFINITY;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int key = 8 * x + (e == 0 ? va : vb);
            const float y = key < rows ? (sc[x][e] + sc[x][e + 2]) * f : -INFINITY;
            sc[x][e] = y;
            cm = fmaxf(cm, y);
          }
        cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, 1));
        cm = fmaxf(cm, __shfl_xor_sync(0xffffffffu, cm, 2));
        if (cm > m_run + kLazy) {
          const float alpha = ex2(m_run - cm);  // 0 on the first slice
          l_run *= alpha;
#pragma unroll
          for (int i = 0; i < ON; ++i) {
            oc[i][0] *= alpha;
            oc[i][1] *= alpha;
          }
          m_run = cm;
        }
        __syncwarp();
        const float mr = m_run == -INFINITY ? 0.f : m_run;
        float p[2][2];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            p[x][e] = ex2(sc[x][e] - mr);
            l_run += p[x][e];
          }
        uint32_t a0, a1, a2, a3;
        split_half2(p[0][0], p[0][1], a0, a1);
        split_half2(p[1][0], p[1][1], a2, a3);
        // O += vs (P . V): lane's columns are d = gr * (D / 8) + i
        const float vs = mi.z;
#pragma unroll
        for (int hw = 0; hw < D / 64; ++hw) {
          // d = 128: one 16-byte chunk a row, in two halves; d = 64: 8 bytes a row
          uint2 r0, r1, r2, r3;
          if constexpr (D == 128) {
            r0 = *reinterpret_cast<const uint2*>(vt + tile_at<D, true>(va, gr) + 8 * hw);
            r1 = *reinterpret_cast<const uint2*>(vt + tile_at<D, true>(vb, gr) + 8 * hw);
            r2 = *reinterpret_cast<const uint2*>(vt + tile_at<D, true>(va + 8, gr) + 8 * hw);
            r3 = *reinterpret_cast<const uint2*>(vt + tile_at<D, true>(vb + 8, gr) + 8 * hw);
          } else {
            r0 = *reinterpret_cast<const uint2*>(vt + tile_at<D, true>(va, gr >> 1) + 8 * (gr & 1));
            r1 = *reinterpret_cast<const uint2*>(vt + tile_at<D, true>(vb, gr >> 1) + 8 * (gr & 1));
            r2 = *reinterpret_cast<const uint2*>(vt + tile_at<D, true>(va + 8, gr >> 1) + 8 * (gr & 1));
            r3 = *reinterpret_cast<const uint2*>(vt + tile_at<D, true>(vb + 8, gr >> 1) + 8 * (gr & 1));
          }
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            const uint32_t x0 = w ? r0.y : r0.x, x1 = w ? r1.y : r1.x;
            const uint32_t x2 = w ? r2.y : r2.x, x3 = w ? r3.y : r3.x;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              // bytes (2 h, 2 h + 1) of the two rows, paired by column
              const uint32_t sel = h ? 0x7362 : 0x5140;
              uint32_t e0, e1, f0, f1;
              q8_to_half4<F>(__byte_perm(x0, x1, sel), e0, e1);
              q8_to_half4<F>(__byte_perm(x2, x3, sel), f0, f1);
              const int i = hw * 8 + w * 4 + h * 2;
              float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
              mma16(c0, a0, a1, a2, a3, e0, f0);
              mma16(c1, a0, a1, a2, a3, e1, f1);
              oc[i][0] = fmaf(c0[0] + c0[2], vs, oc[i][0]);
              oc[i][1] = fmaf(c0[1] + c0[3], vs, oc[i][1]);
              oc[i + 1][0] = fmaf(c1[0] + c1[2], vs, oc[i + 1][0]);
              oc[i + 1][1] = fmaf(c1[1] + c1[3], vs, oc[i + 1][1]);
            }
          }
        }
      }
      __syncwarp();  // the stage is read before it is filled again
    }

    // ---- end of the pair in this block: join the warps
    float l = l_run;
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (tq == 0) {
      mw[warp * 8 + gr] = m_run;
      lw[warp * 8 + gr] = l;
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < ON; i += 4)
        *reinterpret_cast<float4*>(ow + ((size_t)warp * 8 + gr) * D + (2 * tq + e) * ON + i) =
            make_float4(oc[i][e], oc[i + 1][e], oc[i + 2][e], oc[i + 3][e]);
    __syncthreads();
    const int64_t pr = (int64_t)b * Hkv + g;
    // blocks of the grid that hold slices of the pair
    auto block_of = [&](long long s) { return (int)(((s + 1) * grid + total - 1) / total - 1); };
    const int xf = block_of(pair0), xl = block_of(pair1 - 1);
    const bool whole = xf == xl;
    const size_t rec = (size_t)G * (D + 2);
    float* part = ws_part + ((size_t)blockIdx.x * 2 + (pair0 < s0 ? 0 : 1)) * rec;
    for (int e = t; e < G * D; e += kQThreads) {
      const int h = e / D, dd = e - h * D;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kQW; ++w) M = fmaxf(M, mw[w * 8 + h]);
      float num = 0.f, den = 0.f;
#pragma unroll
      for (int w = 0; w < kQW; ++w) {
        // a warp without keys weighs 0; one whose logits were NaN keeps its NaN
        const float a = mw[w * 8 + h] == -INFINITY ? 0.f : ex2(mw[w * 8 + h] - M);
        num = fmaf(a, ow[((size_t)w * 8 + h) * D + dd], num);
        den = fmaf(a, lw[w * 8 + h], den);
      }
      if (whole) {
        store_out(O + ((int64_t)b * Hq + g * G + h) * D + dd, den == 0.f ? 0.f : num / den);
      } else {
        part[2 * G + h * D + dd] = num;
        if (dd == 0) {
          part[h] = M;
          part[G + h] = den;
        }
      }
    }
    if (!whole) {
      __threadfence();
      __syncthreads();
      if (t == 0) s_last = atomicAdd(&ws_ctr[pr], 1) == xl - xf;
      __syncthreads();
      if (s_last) {
        __threadfence();
        for (int e = t; e < G * D; e += kQThreads) {
          const int h = e / D, dd = e - h * D;
          // the pair is the last of its first block and the first of the others
          auto record = [&](int x) { return ws_part + ((size_t)x * 2 + (x == xf ? 1 : 0)) * rec; };
          float M = -INFINITY;
          for (int x = xf; x <= xl; ++x) M = fmaxf(M, __ldcg(record(x) + h));
          float num = 0.f, den = 0.f;
          for (int x = xf; x <= xl; ++x) {
            const float* pp = record(x);
            const float mx = __ldcg(pp + h);
            const float a = mx == -INFINITY ? 0.f : ex2(mx - M);
            num = fmaf(a, __ldcg(pp + 2 * G + h * D + dd), num);
            den = fmaf(a, __ldcg(pp + G + h), den);
          }
          store_out(O + ((int64_t)b * Hq + g * G + h) * D + dd, den == 0.f ? 0.f : num / den);
        }
      }
    }
    pos = end;
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

Q8Plan plan_q8(int batch, int Hq, int Hkv, int d, int topk, int max_blocks) {
  Q8Plan p{};
  p.kk = topk < max_blocks ? topk : max_blocks;
  p.width = p.kk + 2;
  const size_t pairs = (size_t)batch * Hkv;
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  // lists are kept for rows that leave blocks out; with topk >= the candidates of
  // the longest row there are none
  const size_t lists = topk >= max_blocks - 2 ? 0 : pairs * p.width * sizeof(int32_t);
  p.off_off = up(lists);
  p.off_ctr = up(p.off_off + ((size_t)batch + 1) * sizeof(int32_t));
  p.off_part = up(p.off_ctr + pairs * sizeof(int));
  p.bytes = up(p.off_part + (size_t)kQGridMax * 2 * (Hq / Hkv) * (d + 2) * sizeof(float));
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
  const size_t smem1 = sizeof(float) * (D + 256 + (size_t)max_blocks);
  cudaError_t e = cudaFuncSetAttribute(q8_route_kernel<T, D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem1);
  if (e != cudaSuccess) return e;
  q8_route_kernel<T, D><<<batch * Hkv + 1, 256, smem1, st>>>(
      (const T*)q, S, seqlens, batch, Hq, Hkv, max_blocks * B, B, max_blocks, p.kk, p.width,
      ws_idx, ws_ctr, ws_off, (T*)O, idx_out, 1.0f / sqrtf((float)D));
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int stages = D == 128 ? 3 : 8;
  const size_t smem2 = (size_t)(D / 16) * 32 * 16 + 8 * sizeof(float) +
                       (size_t)kQW * 8 * (D + 2) * sizeof(float) +
                       (size_t)kQW * 8 * sizeof(float4) +
                       (size_t)kQW * stages * 2 * kSlice * D;
  int dev = 0, sms = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int grid = sms < kQGridMax ? sms : kQGridMax;
  e = cudaFuncSetAttribute(q8_split_kernel<T, D, F>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)smem2);
  if (e != cudaSuccess) return e;
  q8_split_kernel<T, D, F><<<grid, kQThreads, smem2, st>>>(
      (const T*)q, (const uint8_t*)Kp, Ks, (const uint8_t*)Vp, Vs, table, seqlens, batch, Hq, Hkv,
      B, max_blocks, num_pages, p.kk, p.width, stages, kQW, ws_idx, ws_off, ws_part, ws_ctr,
      (T*)O, scale * 1.4426950408889634f);
  return cudaGetLastError();
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
