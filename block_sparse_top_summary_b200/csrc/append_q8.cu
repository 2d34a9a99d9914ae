// New tokens of a ragged batch into pages of 8-bit codes.
//
// A unit is one block of one sequence that receives rows: rows [r0, r1) of its page
// are new.  A tile is a unit's rows of one KV head, of K or of V.  HBM-bound for
// prompts: every new element is read once, held in registers while the largest
// magnitude of the tile is formed, and written as a code.  What a part-filled block
// held before is read again only when the scale grows (its codes are then rounded
// again under the larger scale) or when the block is complete and its keys' mean
// is due.
//
// A block of threads takes a unit, K or V, and a group of heads.  It is as large as
// a tile of B rows with kChunks 8-element chunks a thread (bf16: 8, fp32: 4), and
// has the next two heads' rows under way while it works on the present one's.  Units
// of few rows (decode steps) are left to single warps, a head each, without a barrier.
// 52233 tokens of 8 heads, d = 128, B = 64 (bf16 to e4m3; 0.32 GB): 229 us with one block of
// 256 threads a tile and a bisection of dependent loads, 54 us (6.0 TB/s) this way, with
// the arithmetic at some 58% of the issue slots: 8 chunks a thread (4: 69 us) and
// mixed-precision FMAs on the bf16 elements (unpacked first: 76 us) cut that.  64 single
// tokens: 17 us before, 3.6 us (calls back to back in a CUDA graph).
//
// Units of sequence b start at floor(cu[b] / B) + 2 b: n new tokens touch at most
// floor(n / B) + 2 blocks, so the ranges do not meet, and a unit's sequence is found
// without another pass over the batch.
//
// The largest magnitude is a maximum over sign-less bits: a NaN or an infinity
// beats every finite value and marks the block by a NaN scale.
#include "common.cuh"
#include "kernels.h"
#include "q8.cuh"

namespace ssa {

namespace {

// Eight elements as they are read.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
};

template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i)
    r.v[i] = ldg16_stream(reinterpret_cast<const uint4*>(p) + i);
  return r;
}

// y = x f + c, rounded once to fp32.  bf16: mixed-precision FMAs take the elements as
// they are (f is a power of two, so exact in bf16).
__device__ __forceinline__ void fma8(const Raw8<float>& r, float f, float c, float* y) {
  float x[8];
  unpack16(r.v[0], x, x);
  unpack16(r.v[1], x + 4, x);
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = fmaf(x[e], f, c);
}
__device__ __forceinline__ void fma8(const Raw8<__nv_bfloat16>& r, float f, float c, float* y) {
  const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
  const uint16_t h = (uint16_t)(__float_as_uint(f) >> 16);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\t"
        "fma.rn.f32.bf16 %0, l, %3, %4;\n\tfma.rn.f32.bf16 %1, u, %3, %4;\n\t}"
        : "=f"(y[2 * i]), "=f"(y[2 * i + 1])
        : "r"(w[i]), "h"(h), "f"(c));
}

// sum += the eight e4m3 codes' values.
__device__ __forceinline__ void add8_e4m3(uint2 c, float* sum) {
  uint32_t h[4];
  q8_to_half4<SSA_E4M3>(c.x, h[0], h[1]);
  q8_to_half4<SSA_E4M3>(c.y, h[2], h[3]);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\t"
        "add.f32.f16 %0, l, %0;\n\tadd.f32.f16 %1, u, %1;\n\t}"
        : "+f"(sum[2 * i]), "+f"(sum[2 * i + 1])
        : "r"(h[i]));
}

// Largest magnitude so far; bf16: of even and odd elements, in the two halves.
__device__ __forceinline__ void max8(const Raw8<float>& r, uint32_t& m) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    m = max(m, max(r.v[i].x & 0x7fffffffu, r.v[i].y & 0x7fffffffu));
    m = max(m, max(r.v[i].z & 0x7fffffffu, r.v[i].w & 0x7fffffffu));
  }
}
__device__ __forceinline__ void max8(const Raw8<__nv_bfloat16>& r, uint32_t& m) {
  const uint4 v = r.v[0];
  m = __vmaxu2(m, __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                           __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu)));
}
// ... as fp32 bits
template <typename T>
__device__ __forceinline__ uint32_t max_bits(uint32_t m) {
  return sizeof(T) == 2 ? max(m << 16, m & 0xffff0000u) : m;
}

}  // namespace

template <typename T, int D, int F>
__global__ void __launch_bounds__(512) append_q8_kernel(
    uint8_t* __restrict__ Kp, float* __restrict__ Ks, uint8_t* __restrict__ Vp,
    float* __restrict__ Vs, float* __restrict__ S, const int32_t* __restrict__ slots,
    const int32_t* __restrict__ cu, const int32_t* __restrict__ seqlens, const T* __restrict__ kn,
    const T* __restrict__ vn, long long tok_stride, long long head_stride, int batch, int T_max,
    int Hkv, int heads, int B, int max_blocks, int num_pages) {
  constexpr int CPR = D / 8;        // 8-element chunks a row
  constexpr int RPW = 32 / CPR;     // rows a warp step
  constexpr int kChunks = sizeof(T) == 2 ? 8 : 4;
  __shared__ uint32_t s_max[2][16];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, warps = blockDim.x >> 5;
  const bool is_v = blockIdx.y & 1;
  const int g0 = (blockIdx.y >> 1) * heads, g1 = min(g0 + heads, Hkv);
  const int u = blockIdx.x;
  grid_wait();  // the kernels before

  // the sequence: the last b with floor(cu[b] / B) + 2 b <= u, 32 guesses a step
  int b = 0;
  for (int n = batch; n > 1;) {
    const int step = (n + 31) / 32, i = b + lane * step;
    const bool in = lane * step < n && cu[i] / B + 2 * i <= u;
    const int c = max(__popc(__ballot_sync(0xffffffffu, in)), 1) - 1;
    b += c * step;
    n = min(step, n - c * step);
  }
  const int c0 = cu[b], c1 = cu[b + 1];
  const int len = seqlens[b], p0 = len - (c1 - c0);
  if (c0 < 0 || c1 <= c0 || c1 > T_max || p0 < 0) return;
  const int j = p0 / B + (u - (c0 / B + 2 * b));
  if (j < 0 || j >= max_blocks || j * B >= len) return;
  const int r0 = max(p0 - j * B, 0), r1 = min(len - j * B, B);
  const int t0 = c0 + j * B + r0 - p0;  // token of row r0
  const int slot = slots[t0];
  if (slot < 0 || slot % B != r0 || slot / B >= num_pages) return;  // refused, or not this block's
  const int page = slot / B, nr = r1 - r0;
  const bool mean = !is_v && S != nullptr && r1 == B;

  const T* x = (is_v ? vn : kn) + (int64_t)t0 * tok_stride;
  uint8_t* P0 = (is_v ? Vp : Kp) + (int64_t)page * Hkv * B * D;
  float* Ps = (is_v ? Vs : Ks) + (int64_t)page * Hkv;

  // A tile by `rps` rows a step: this thread's chunks are column cc of the rows
  // rr, rr + rps, ...
  auto load = [&](int g, int rr, int cc, int rps, Raw8<T>(&raw)[kChunks]) {
    const T* p = x + (int64_t)g * head_stride + (int64_t)rr * tok_stride + cc * 8;
    const int64_t step = rps * tok_stride;
#pragma unroll
    for (int i = 0; i < kChunks; ++i, p += step)
      if (rr + i * rps < nr) raw[i] = load8(p);
  };
  auto largest = [&](int rr, int rps, const Raw8<T>(&raw)[kChunks]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
      if (rr + i * rps < nr) max8(raw[i], m);
    return __reduce_max_sync(0xffffffffu, max_bits<T>(m));
  };
  // codes of the tile; sum: of this thread's held values, where the mean is due
  auto write = [&](int g, int rr, int cc, int rps, const Raw8<T>(&raw)[kChunks], uint32_t m,
                   float old, float (&sum)[8]) -> float {
    const bool nan = m >= 0x7f800000u || old != old;
    const float scale = nan ? __uint_as_float(0x7fc00000u) : fmaxf(old, q8_scale<F>(m));
    // scales are powers of two, so the product with the reciprocal is x / scale
    const float inv = nan ? 0.f : 1.f / scale;
    uint8_t* P = P0 + (int64_t)g * B * D + cc * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = 0.f;
    // i8: y + 1.5 * 2^23 is rounded to a whole number, whose low byte is the code and
    // whose bits are 0x4b400000 + code
    constexpr float kRound = 12582912.f;
    uint32_t isum[8] = {0, 0, 0, 0, 0, 0, 0, 0}, cnt = 0;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
      const int r = rr + i * rps;
      if (r < nr) {
        float y[8];
        uint2 c;
        fma8(raw[i], inv, F == SSA_I8 ? kRound : -0.f, y);
        if constexpr (F == SSA_I8) {
          uint32_t w[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(y[e]);
          c.x = __byte_perm(__byte_perm(w[0], w[1], 0x0040), __byte_perm(w[2], w[3], 0x0040), 0x5410);
          c.y = __byte_perm(__byte_perm(w[4], w[5], 0x0040), __byte_perm(w[6], w[7], 0x0040), 0x5410);
          if (mean) {
            ++cnt;
#pragma unroll
            for (int e = 0; e < 8; ++e) isum[e] += w[e];
          }
        } else {
          c = q8_pack8<F>(y);
          if (mean) add8_e4m3(c, sum);
        }
        if (nan) c = make_uint2(0, 0);
        *reinterpret_cast<uint2*>(P + (r0 + r) * D) = c;
      }
    }
    if constexpr (F == SSA_I8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] = (float)(int)(isum[e] - cnt * 0x4b400000u);
    }
    // the rows that the block held before
    const bool grown = r0 > 0 && !nan && scale > old;
    if (grown || (mean && r0 > 0)) {
      const float ratio = grown ? old * inv : 1.f;
      for (int q = rr; q < r0; q += kChunks * rps) {
        // read together, ahead of the first write (each on its own: 64 us for the 52 K tokens)
        uint2 held[kChunks];
#pragma unroll
        for (int i = 0; i < kChunks; ++i)
          if (q + i * rps < r0) held[i] = *reinterpret_cast<const uint2*>(P + (q + i * rps) * D);
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const int r = q + i * rps;
          if (r < r0) {
            float y[8];
            uint2 c = held[i];
            if (grown) {
              q8_unpack8<F>(c, y);
#pragma unroll
              for (int e = 0; e < 8; ++e) y[e] *= ratio;
              c = q8_pack8<F>(y);
              *reinterpret_cast<uint2*>(P + r * D) = c;
            }
            if (mean) {
              q8_unpack8<F>(c, y);
#pragma unroll
              for (int e = 0; e < 8; ++e) sum[e] += y[e];
            }
          }
        }
      }
    }
    return scale;
  };
  float* Sj = S + ((int64_t)b * Hkv * max_blocks + j) * D;  // used only where the mean is due

  if (nr <= kChunks * RPW) {
    // a warp a head
    const int rr = lane / CPR, cc = lane % CPR;
    for (int g = g0 + warp; g < g1; g += warps) {
      Raw8<T> raw[kChunks];
      load(g, rr, cc, RPW, raw);
      const float old = r0 > 0 ? Ps[g] : 0.f;
      float sum[8];
      const float scale = write(g, rr, cc, RPW, raw, largest(rr, RPW, raw), old, sum);
      __syncwarp();  // every lane has the old scale
      if (lane == 0) Ps[g] = scale;
      if (mean) {  // the lanes of a column
#pragma unroll
        for (int o = CPR; o < 32; o <<= 1)
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[e] += __shfl_xor_sync(0xffffffffu, sum[e], o);
      }
      if (mean && lane < CPR) {
        float* d = Sj + (int64_t)g * max_blocks * D + cc * 8;
        const float f = scale / (float)B;
        *reinterpret_cast<float4*>(d) = make_float4(sum[0] * f, sum[1] * f, sum[2] * f, sum[3] * f);
        *reinterpret_cast<float4*>(d + 4) =
            make_float4(sum[4] * f, sum[5] * f, sum[6] * f, sum[7] * f);
      }
    }
    return;
  }
  // the block a head, the next ones on their way to shared memory: a thread copies its
  // own chunks and reads them back, so its own waits are enough
  const int rps = warps * RPW, rr = t / CPR, cc = t % CPR;
  constexpr int stages = 2;  // 3 and 4 were no faster
  constexpr int PIECES = kChunks * (int)sizeof(T) / 2;  // 16-byte pieces a thread and head
  extern __shared__ __align__(16) uint4 ring[];         // [stages][PIECES][threads]
  float* s_sum = reinterpret_cast<float*>(ring + stages * PIECES * blockDim.x);  // [rps][D]
  auto fetch = [&](int g, int stage) {
    if (g < g1) {
      const T* p = x + (int64_t)g * head_stride + (int64_t)rr * tok_stride + cc * 8;
      const int64_t step = rps * tok_stride;
      uint32_t to = (uint32_t)__cvta_generic_to_shared(ring + (stage * PIECES) * blockDim.x + t);
#pragma unroll
      for (int i = 0; i < kChunks; ++i, p += step)
#pragma unroll
        for (int k = 0; k < PIECES / kChunks; ++k, to += blockDim.x * 16)
          if (rr + i * rps < nr)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to),
                         "l"(reinterpret_cast<const uint4*>(p) + k)
                         : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  for (int i = 0; i < stages; ++i) fetch(g0 + i, i);
  float old = r0 > 0 ? Ps[g0] : 0.f, old_next = 0.f;
  int stage = 0;
  for (int g = g0; g < g1; ++g) {
    if (r0 > 0 && g + 1 < g1) old_next = Ps[g + 1];
    asm volatile("cp.async.wait_group %0;" ::"n"(stages - 1) : "memory");
    Raw8<T> raw[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i)
#pragma unroll
      for (int k = 0; k < PIECES / kChunks; ++k)
        raw[i].v[k] = ring[(stage * PIECES + i * (PIECES / kChunks) + k) * blockDim.x + t];
    uint32_t m = largest(rr, rps, raw);
    fetch(g + stages, stage);
    stage = stage == stages - 1 ? 0 : stage + 1;
    uint32_t* sm = s_max[(g - g0) & 1];  // the other one may still be read
    if (lane == 0) sm[warp] = m;
    __syncthreads();
    m = __reduce_max_sync(0xffffffffu, lane < warps ? sm[lane] : 0u);
    float sum[8];
    const float scale = write(g, rr, cc, rps, raw, m, old, sum);
    if (t == 0) Ps[g] = scale;  // the old one was read before the barrier
    if (mean) {
      float4* mine = reinterpret_cast<float4*>(s_sum + rr * D + cc * 8);
      mine[0] = make_float4(sum[0], sum[1], sum[2], sum[3]);
      mine[1] = make_float4(sum[4], sum[5], sum[6], sum[7]);
      __syncthreads();
      for (int c = t; c < D; c += blockDim.x) {
        float a = 0.f;
#pragma unroll 8
        for (int w = 0; w < rps; ++w) a += s_sum[w * D + c];
        Sj[(int64_t)g * max_blocks * D + c] = a * (scale / (float)B);
      }
      // s_sum is written again only behind the next head's barrier
    }
    old = old_next;
  }
}

template <typename T, int D, int F>
static cudaError_t launch_append_q8_t(void* Kp, float* Ks, void* Vp, float* Vs, float* S,
                                      const int32_t* slots, const int32_t* cu,
                                      const int32_t* seqlens, const void* kn, const void* vn,
                                      long long tok_stride, long long head_stride, int batch,
                                      int T_max, int Hkv, int B, int max_blocks, int num_pages,
                                      cudaStream_t st) {
  constexpr int chunks = sizeof(T) == 2 ? 8 : 4;
  const int threads = (B * (D / 8) / chunks + 31) / 32 * 32;  // 32 .. 512
  const long long units = T_max / B + 2LL * batch;
  // All heads of a unit in one block where the units alone fill the GPU (2 blocks for
  // each of 148 SMs), else fewer.
  int heads = Hkv;
  while (heads > 1 && units * 2 * ((Hkv + heads - 1) / heads) < 2 * 148) heads = (heads + 1) / 2;
  // Up to one and a half waves of blocks of all heads (512 threads an SM at 128 registers),
  // half of the heads a block, but 4 at least: the last wave's idle SMs cost more than a
  // second start of the pipeline.  All heads and half of 8 (bf16, d = 128, B = 64; 16 ragged
  // prompts), us: 12 K tokens 19.0, 15.7; 20 K 28.9, 25.9; 33 K 35.6, 36.6; 52 K 53.4, 54.8.
  // (Two heads of four: 65 K tokens 36.4, 38.9.)
  const long long blocks = 2 * (T_max / B + (long long)batch);
  if (heads == Hkv && Hkv >= 7 && 2 * blocks * threads < 3LL * 148 * 512) heads = (Hkv + 1) / 2;
  const dim3 grid((unsigned)units, (unsigned)(2 * ((Hkv + heads - 1) / heads)));
  // two heads' rows (16 KB each for 64 rows of 128 in bf16), and the threads' sums
  constexpr int each = 2 * chunks * 8 * (int)sizeof(T) + 8 * (int)sizeof(float);
  const int smem = threads * each;
  if (smem > 47 * 1024) {  // the static array counts too
    // (the limit is the kernel's, for all host threads: always that of B = 128)
    const cudaError_t e =
        cudaFuncSetAttribute(append_q8_kernel<T, D, F>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             128 * (D / 8) / chunks * each);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, append_q8_kernel<T, D, F>, (uint8_t*)Kp, Ks, (uint8_t*)Vp, Vs, S,
                            slots, cu, seqlens, (const T*)kn, (const T*)vn, tok_stride,
                            head_stride, batch, T_max, Hkv, heads, B, max_blocks, num_pages);
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
