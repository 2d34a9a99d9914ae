// Pages, slots and lengths of a batch of requests, on the GPU.
//
// Row b holds have[b] tokens and asks for want[b].  With hb = ceil(have / B) and
// wb = ceil(want / B), a growing row needs n = want - have token slots and
// need = max(wb - hb, 0) pages; a shrinking one gives back the blocks
// [max(wb, keep), hb).  Three prefix sums over the rows (tokens C, pages P,
// returned pages R) decide everything: which rows grow, which ring entry each new
// block takes and where each returned page goes.  All sums are 64 bits wide (a
// batch of long requests passes 2^31 tokens); what is kept in shared memory is
// clamped to 2^31 - 1, which no granted row reaches.
//
// One cluster of 1 or 8 blocks of 1024 threads.  Every block forms the prefix sums of
// the whole batch (a thread sums a run of rows, a block scan joins the runs) and
// keeps them in its shared memory; the blocks then share out the token slots, the
// new pages and the returned pages, each found in its prefix sum by bisection.
// The lengths and the pool's state are written behind a cluster barrier, by which
// all blocks have read them, so that both may be updated in place.
// Launch-bound up to a few thousand tokens; beyond, a block's work is the slots
// (4 bytes a token, one search for 8 tokens): 0.47 million slots take 637 us in
// one block with a search a token and 64-bit remainders, MEASURED us in 8.
#include "common.cuh"
#include "kernels.h"

namespace ssa {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kIntMax = 0x7fffffff;

struct PlanRow {
  long long n, need, back;
};

// Exclusive prefix sums of three values a thread; total: their sums.
__device__ __forceinline__ PlanRow plan_scan(PlanRow v, PlanRow* wsum, PlanRow* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  PlanRow in = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, in.n, o);
    const long long b = __shfl_up_sync(0xffffffffu, in.need, o);
    const long long c = __shfl_up_sync(0xffffffffu, in.back, o);
    if (lane >= o) {
      in.n += a;
      in.need += b;
      in.back += c;
    }
  }
  if (lane == 31) wsum[warp] = in;
  __syncthreads();
  if (warp == 0) {
    PlanRow w = wsum[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, w.n, o);
      const long long b = __shfl_up_sync(0xffffffffu, w.need, o);
      const long long c = __shfl_up_sync(0xffffffffu, w.back, o);
      if (lane >= o) {
        w.n += a;
        w.need += b;
        w.back += c;
      }
    }
    wsum[lane] = w;
  }
  __syncthreads();
  *total = wsum[kPlanThreads / 32 - 1];
  PlanRow out{in.n - v.n, in.need - v.need, in.back - v.back};
  if (warp > 0) {
    const PlanRow w = wsum[warp - 1];
    out.n += w.n;
    out.need += w.need;
    out.back += w.back;
  }
  return out;
}

// First row whose inclusive prefix sum lies above x (x below the last sum).
__device__ __forceinline__ int row_above(const int* incl, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (incl[mid] > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

__device__ __forceinline__ int clamp_int(long long v) { return v > kIntMax ? kIntMax : (int)v; }

}  // namespace

// V: tokens on end that a thread places at a time (1 or 8).
template <int V>
__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(
    const int32_t* have, const int32_t* want, const int32_t* keep, int batch, int B,
    int32_t* __restrict__ table, int max_blocks, int num_pages, int32_t* __restrict__ ring,
    const int32_t* pool, int32_t* pool_out, int32_t* got, int32_t* __restrict__ cu,
    int32_t* __restrict__ slots, int max_new) {
  extern __shared__ int plan_smem[];
  int* tok = plan_smem;       // [batch] inclusive sums of the rows' new tokens
  int* pag = tok + batch;     // [batch] ... of their new pages
  int* bak = pag + batch;     // [batch] ... of their returned pages
  int* row = bak + batch;     // [batch] tokens held, bit 31: the row grows
  int* from = row + batch;    // [batch] first block a shrinking row gives back
  int* len = from + batch;    // [batch] got
  __shared__ PlanRow wsum[32];
  __shared__ int s_taken;
  const int t = threadIdx.x;
  const int blocks = gridDim.x, rank = blockIdx.x;  // one cluster
  const int cap = max_blocks * B;
  // a pool state out of range is taken as an empty or a full ring
  const int head = min(max(pool[0], 0), num_pages - 1);
  const int count = min(max(pool[1], 0), num_pages);
  if (t == 0) s_taken = 0;

  const int per = (batch + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(t * per, batch), r1 = min(r0 + per, batch);
  struct Row {
    int h, w, lo;  // held, wanted (-1: refused), first block given back
    PlanRow v;
  };
  auto read = [&](int b) -> Row {
    Row r{have[b], want[b], 0, PlanRow{0, 0, 0}};
    const int kp = keep != nullptr ? keep[b] : 0;
    if (r.h < 0 || r.h > cap || r.w < 0 || r.w > cap) {
      r.w = -1;
      return r;
    }
    const int hb = (r.h + B - 1) / B, wb = (r.w + B - 1) / B;
    if (r.w >= r.h) {
      r.v.n = r.w - r.h;
      r.v.need = wb - hb;
    } else {
      r.lo = max(wb, min(max(kp, 0), hb));
      r.v.back = hb - r.lo;
    }
    return r;
  };
  PlanRow mine{0, 0, 0};
  Row one{};  // the thread's last row: its only one up to 1024 rows
  for (int b = r0; b < r1; ++b) {
    one = read(b);
    mine.n += one.v.n;
    mine.need += one.v.need;
    mine.back += one.v.back;
  }
  PlanRow total;
  PlanRow run = plan_scan(mine, wsum, &total);
  int taken = 0;
  for (int b = r0; b < r1; ++b) {
    const Row r = per == 1 ? one : read(b);
    run.n += r.v.n;
    run.need += r.v.need;
    run.back += r.v.back;
    const bool grows = r.v.n > 0 && run.n <= (long long)max_new &&
                       (r.v.need == 0 || run.need <= (long long)count);
    if (grows && r.v.need > 0) taken = (int)run.need;
    tok[b] = clamp_int(run.n);
    pag[b] = clamp_int(run.need);
    bak[b] = clamp_int(run.back);
    row[b] = r.w < 0 ? 0 : (r.h | (grows ? (int)0x80000000 : 0));
    from[b] = r.lo;
    len[b] = grows || (r.w >= 0 && r.w < r.h) ? r.w : r.h;
    if (rank == 0) cu[b + 1] = (int)min(run.n, (long long)max_new);
  }
  if (t == 0 && rank == 0) cu[0] = 0;
  if (taken > 0) atomicMax(&s_taken, taken);
  __syncthreads();
  taken = s_taken;  // the rows that take pages are a prefix of those that ask
  const int tokens = (int)min(total.n, (long long)max_new);
  const int given = (int)min(total.back, (long long)(num_pages - count));
  if (blocks > 1) cluster_arrive();  // this block has read the lengths and the pool's state

  // entry i behind the head; i <= num_pages
  auto ring_at = [&](int i) {
    const int x = head + i;
    return x >= num_pages ? x - num_pages : x;
  };
  for (int i0 = (rank * kPlanThreads + t) * V; i0 < max_new; i0 += blocks * kPlanThreads * V) {
    // first where each token's page stands, then the pages, all at once
    const int32_t* at[V];
    int r[V];
    int b = 0, end = 0, j = 0, hb = 0, place = 0;
    const int32_t* word = nullptr;
    auto enter = [&](int i) {  // token i of row b
      end = tok[b];
      const int x = row[b], h = x & kIntMax;
      const int pos = h + i - (b > 0 ? tok[b - 1] : 0);
      hb = x < 0 ? (h + B - 1) / B : -1;  // -1: a refused row
      j = pos / B;
      place = pos - j * B;
    };
    auto find = [&]() {  // block j of row b, of which the call may add some
      word = hb < 0    ? nullptr
             : j < hb ? table + (int64_t)b * max_blocks + j
                      : ring + ring_at((b > 0 ? pag[b - 1] : 0) + (j - hb));
    };
    if (i0 < tokens) {
      b = row_above(tok, batch, i0);
      enter(i0);
      find();
    }
#pragma unroll
    for (int u = 0; u < V; ++u) {
      if (u > 0 && i0 + u < tokens) {
        ++place;
        if (i0 + u >= end) {
          do ++b; while (tok[b] <= i0 + u);
          enter(i0 + u);
          find();
        } else if (place == B) {
          ++j;
          place = 0;
          find();
        }
      }
      at[u] = i0 + u < tokens ? word : nullptr;
      r[u] = place;
    }
    int out[V];
#pragma unroll
    for (int u = 0; u < V; ++u) out[u] = at[u] != nullptr ? *at[u] : -1;
#pragma unroll
    for (int u = 0; u < V; ++u)
      out[u] = out[u] >= 0 && out[u] < num_pages ? out[u] * B + r[u] : -1;
    if (V == 8 && i0 + V <= max_new) {
      *reinterpret_cast<int4*>(slots + i0) =
          make_int4(out[0], out[1 % V], out[2 % V], out[3 % V]);
      *reinterpret_cast<int4*>(slots + i0 + 4) =
          make_int4(out[4 % V], out[5 % V], out[6 % V], out[7 % V]);
    } else {
#pragma unroll
      for (int u = 0; u < V; ++u)
        if (i0 + u < max_new) slots[i0 + u] = out[u];
    }
  }
  // new blocks' pages
  for (int i = rank * kPlanThreads + t; i < taken; i += blocks * kPlanThreads) {
    const int page = ring[ring_at(i)];
    const int b = row_above(pag, batch, i);
    const int hb = ((row[b] & kIntMax) + B - 1) / B;
    table[(int64_t)b * max_blocks + hb + i - (b > 0 ? pag[b - 1] : 0)] = page;
  }
  // returned pages go behind the free ones; entries taken above are not reached,
  // as at most num_pages - count come back
  for (int i = rank * kPlanThreads + t; i < given; i += blocks * kPlanThreads) {
    const int b = row_above(bak, batch, i);
    ring[ring_at(count + i)] =
        table[(int64_t)b * max_blocks + from[b] + i - (b > 0 ? bak[b - 1] : 0)];
  }
  if (blocks > 1) cluster_wait();
  if (rank > 0) return;
  for (int b = r0; b < r1; ++b) got[b] = len[b];
  if (t == 0) {
    const int x = head + taken;
    pool_out[0] = x >= num_pages ? x - num_pages : x;
    pool_out[1] = count - taken + given;
  }
}

cudaError_t launch_page_plan(const int32_t* have, const int32_t* want, const int32_t* keep,
                             int batch, int B, int32_t* table, int max_blocks, int num_pages,
                             int32_t* ring, const int32_t* pool, int32_t* pool_out, int32_t* got,
                             int32_t* cu, int32_t* slots, int max_new, cudaStream_t st) {
  const size_t smem = (size_t)batch * 6 * sizeof(int);
  // Up to 8192 slots one block, a token a thread, so that the pages of one-token rows
  // are read at once; beyond, 8 tokens a thread in a cluster of 8 blocks.
  const bool one = max_new <= 8 * kPlanThreads;
  const auto kernel = one ? page_plan_kernel<1> : page_plan_kernel<8>;
  if (smem > 46 * 1024) {  // the static arrays count too
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 8;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(one ? 1 : 8);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = one ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, have, want, keep, batch, B, table, max_blocks, num_pages,
                            ring, pool, pool_out, got, cu, slots, max_new);
}

}  // namespace ssa
