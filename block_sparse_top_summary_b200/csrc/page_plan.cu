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
// One block of 1024 threads: each thread sums a run of rows, a block scan joins the
// runs, and then the threads walk the token slots, the new pages and the
// returned pages, each found in its prefix sum by bisection.
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
  __shared__ PlanRow wsum[32];
  __shared__ int s_taken;
  const int t = threadIdx.x;
  const int cap = max_blocks * B;
  // a pool state out of range is taken as an empty or a full ring
  const int head = min(max(pool[0], 0), num_pages - 1);
  const int count = min(max(pool[1], 0), num_pages);
  if (t == 0) s_taken = 0;

  const int per = (batch + kPlanThreads - 1) / kPlanThreads;
  const int r0 = min(t * per, batch), r1 = min(r0 + per, batch);
  auto read = [&](int b, int& h, int& w, int& lo) -> PlanRow {
    h = have[b];
    w = want[b];
    lo = 0;
    if (h < 0 || h > cap || w < 0 || w > cap) {
      w = -1;  // refused
      return PlanRow{0, 0, 0};
    }
    const int hb = (h + B - 1) / B, wb = (w + B - 1) / B;
    if (w >= h) return PlanRow{w - h, wb - hb, 0};
    const int kp = keep != nullptr ? min(max(keep[b], 0), hb) : 0;
    lo = max(wb, kp);
    return PlanRow{0, 0, hb - lo};
  };
  PlanRow mine{0, 0, 0};
  for (int b = r0; b < r1; ++b) {
    int h, w, lo;
    const PlanRow v = read(b, h, w, lo);
    mine.n += v.n;
    mine.need += v.need;
    mine.back += v.back;
  }
  PlanRow total;
  PlanRow run = plan_scan(mine, wsum, &total);
  int taken = 0;
  for (int b = r0; b < r1; ++b) {
    int h, w, lo;
    const PlanRow v = read(b, h, w, lo);
    run.n += v.n;
    run.need += v.need;
    run.back += v.back;
    const bool grows =
        v.n > 0 && run.n <= (long long)max_new && (v.need == 0 || run.need <= (long long)count);
    if (grows && v.need > 0) taken = (int)run.need;
    tok[b] = clamp_int(run.n);
    pag[b] = clamp_int(run.need);
    bak[b] = clamp_int(run.back);
    row[b] = w < 0 ? 0 : (h | (grows ? (int)0x80000000 : 0));
    from[b] = lo;
    // a thread writes the rows that it alone has read, so got may be have
    got[b] = grows || (w >= 0 && w < h) ? w : h;
    cu[b + 1] = (int)min(run.n, (long long)max_new);
  }
  if (t == 0) cu[0] = 0;
  if (taken > 0) atomicMax(&s_taken, taken);
  __syncthreads();
  taken = s_taken;  // the rows that take pages are a prefix of those that ask
  const int tokens = (int)min(total.n, (long long)max_new);
  const int given = (int)min(total.back, (long long)(num_pages - count));
  if (t == 0) {
    pool_out[0] = (int)(((long long)head + taken) % num_pages);
    pool_out[1] = count - taken + given;
  }

  auto ring_at = [&](long long i) { return (int)(((long long)head + i) % num_pages); };
  // the page of block j of row b, of which the call may add some
  auto page_of = [&](int b, int j, int hb) -> int {
    if (j < hb) return table[(int64_t)b * max_blocks + j];
    return ring[ring_at((b > 0 ? pag[b - 1] : 0) + (j - hb))];
  };
  for (int i = t; i < max_new; i += kPlanThreads) {
    int slot = -1;
    if (i < tokens) {
      const int b = row_above(tok, batch, i);
      if (row[b] < 0) {
        const int h = row[b] & kIntMax;
        const int pos = h + i - (b > 0 ? tok[b - 1] : 0);
        const int page = page_of(b, pos / B, (h + B - 1) / B);
        if (page >= 0 && page < num_pages) slot = page * B + pos % B;
      }
    }
    slots[i] = slot;
  }
  // new blocks' pages
  for (int i = t; i < taken; i += kPlanThreads) {
    const int b = row_above(pag, batch, i);
    const int hb = ((row[b] & kIntMax) + B - 1) / B;
    table[(int64_t)b * max_blocks + hb + i - (b > 0 ? pag[b - 1] : 0)] = ring[ring_at(i)];
  }
  // returned pages go behind the free ones; entries taken above are not reached,
  // as at most num_pages - count come back
  for (int i = t; i < given; i += kPlanThreads) {
    const int b = row_above(bak, batch, i);
    ring[ring_at((long long)count + i)] =
        table[(int64_t)b * max_blocks + from[b] + i - (b > 0 ? bak[b - 1] : 0)];
  }
}

cudaError_t launch_page_plan(const int32_t* have, const int32_t* want, const int32_t* keep,
                             int batch, int B, int32_t* table, int max_blocks, int num_pages,
                             int32_t* ring, const int32_t* pool, int32_t* pool_out, int32_t* got,
                             int32_t* cu, int32_t* slots, int max_new, cudaStream_t st) {
  const size_t smem = (size_t)batch * 5 * sizeof(int);
  cudaError_t e = cudaFuncSetAttribute(page_plan_kernel,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  page_plan_kernel<<<1, kPlanThreads, smem, st>>>(have, want, keep, batch, B, table, max_blocks,
                                                  num_pages, ring, pool, pool_out, got, cu, slots,
                                                  max_new);
  return cudaGetLastError();
}

}  // namespace ssa
