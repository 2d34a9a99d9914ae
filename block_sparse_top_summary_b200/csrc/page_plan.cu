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
// Blocks of 1024 threads form the prefix sums (a thread sums a run of rows, a block
// scan joins the runs) and keep them in shared memory; token slots, new pages and
// returned pages are then shared out, each found in its prefix sum by bisection.  The
// lengths and the pool's state are written last, when all blocks have read them, so
// that both may be updated in place.
//
// Bounds: up to a few thousand slots the launch and the chain of one block (lengths,
// scan, pages: 6 us for 256 one-token rows); beyond, the instructions that place a
// slot, which want the whole GPU.  So up to 8192 slots and 4096 rows one block does it all,
// and beyond a cluster of 8 does rows and pages (all of its blocks form the sums, and a
// cluster barrier stands before the last writes) and a second kernel the slots.
// Cluster and slots kernel against one block, us: 256 rows of 1 token 16.4, 6.1; 4000
// rows of 1 24.3, 14.3; 8 rows of 1000 8.2, 9.1; 64 rows of 250 10.2, 16.4; 4 rows of 8000
// 10.2, 24.6.  0.47 million slots of 1024 rows with 31 thousand pages: 18 us (16.4 with
// calls back to back, which overlap; 256 one-token rows then 4.1); with
// the slots in the cluster 31 us, in one block 637 us.
// Pages that come back are moved as well, and the host knows nothing of their number: rows of
// one token, of which some have finished, cluster and slots kernel against one block, us: 256
// rows, none 14.4, 4.2; 22 K pages back 14.9, 16.7; 1024 rows, 68 K back 27.2, 29.2; 4096
// rows, none 21.4, 15.9; 23 K back 28.8, 27.4; 246 K back 38.9, 85.7; 8192 rows, none 34.0,
// 34.5; 335 K back 51.2, 117.  One block keeps the quiet steps, up to where it gains nothing.
#include "common.cuh"
#include "kernels.h"

namespace ssa {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kIntMax = 0x7fffffff;
constexpr int kLongRow = 2048;  // most pages that a warp moves for one row

struct PlanRow {
  long long n, need, back;
};

// x / B for 0 <= x < 2^31, B = 16 d with d <= 8: with m = floor(2^32 / d) + 1 and
// n = x / 16 < 2^27, n m / 2^32 is at most n / 2^32 < 1 / 32 above n / d, so its whole
// part is that of n / d.
struct BlockDiv {
  int B;
  uint32_t m;
  __device__ explicit BlockDiv(int B_) : B(B_), m(B_ > 16 ? 0xffffffffu / (B_ / 16) + 1 : 0) {}
  __device__ int operator()(int x) const {
    const uint32_t n = (uint32_t)x >> 4;
    return m != 0 ? (int)__umulhi(n, m) : (int)n;
  }
  __device__ int up(int x) const {  // blocks of x tokens
    const int q = (*this)(x);
    return q + (q * B < x ? 1 : 0);
  }
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

// The same for one x by a whole warp, 32 guesses a step, among the n rows from lo on.
__device__ __forceinline__ int find_row(const int* incl, int lo, int n, int x) {
  const int lane = threadIdx.x & 31;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int i = lo + min((lane + 1) * step, n) - 1;
    const int k = __ffs(__ballot_sync(0xffffffffu, incl[i] > x)) - 1;
    lo += k * step;
    n = min(step, n - k * step);
  }
  return lo;
}

// row_above for an x of each lane, first <= x <= last.
__device__ __forceinline__ int row_above_warp(const int* incl, int n, int x, int first, int last) {
  const int lo = find_row(incl, 0, n, first);
  if (incl[lo] > last) return lo;
  const int hi = find_row(incl, lo, n - lo, last);
  return lo + row_above(incl + lo, hi - lo + 1, x);
}

__device__ __forceinline__ int clamp_int(long long v) { return v > kIntMax ? kIntMax : (int)v; }

}  // namespace

// kSlots: one block, which fills the slots; else a cluster, which writes the first
// slot of each row, and page_slots_kernel follows.
template <bool kSlots>
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
  __shared__ int s_taken, s_long;
  const int t = threadIdx.x;
  const int blocks = gridDim.x, rank = blockIdx.x;  // one cluster
  grid_wait();  // the kernels before
  if (!kSlots) grid_launch_next();
  const int cap = max_blocks * B;
  const BlockDiv div(B);
  // a pool state out of range is taken as an empty or a full ring
  const int head = min(max(pool[0], 0), num_pages - 1);
  const int count = min(max(pool[1], 0), num_pages);
  if (t == 0) s_taken = s_long = 0;

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
    const int hb = div.up(r.h), wb = div.up(r.w);
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
    if (r.v.need > kLongRow || r.v.back > kLongRow) s_long = 1;
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
  if (!kSlots) cluster_arrive();  // this block has read the lengths and the pool's state

  // entry i behind the head; i <= num_pages
  auto ring_at = [&](int i) {
    const int x = head + i;
    return x >= num_pages ? x - num_pages : x;
  };
  const int lane = t & 31;
  // slot of token i of row b, which holds x (bit 31: it grows); the call may add pages
  auto slot_at = [&](int b, int x, int i) {
    if (x >= 0) return -1;
    const int h = x & kIntMax;
    const int pos = h + i - (b > 0 ? tok[b - 1] : 0);
    const int j = div(pos), hb = div.up(h);
    const int page = j < hb ? table[(int64_t)b * max_blocks + j]
                            : ring[ring_at((b > 0 ? pag[b - 1] : 0) + (j - hb))];
    return page >= 0 && page < num_pages ? page * B + pos - j * B : -1;
  };
  if constexpr (kSlots) {
    for (int w0 = t - lane; w0 < max_new; w0 += kPlanThreads) {
      const int i = w0 + lane;
      int slot = -1;
      if (w0 < tokens) {
        const int last = min(w0 + 32, tokens) - 1;
        const int b = row_above_warp(tok, batch, min(i, last), w0, last);
        if (i < tokens) slot = slot_at(b, row[b], i);
      }
      if (i < max_new) slots[i] = slot;
    }
  } else {
    // the first of each row: whether it is granted, for page_slots_kernel
    for (int b = rank * kPlanThreads + t; b < batch; b += blocks * kPlanThreads) {
      const int i = b > 0 ? tok[b - 1] : 0;
      if (tok[b] > i && i < tokens) slots[i] = slot_at(b, row[b], i);
    }
  }
  // New blocks' pages, and returned pages behind the free ones (the entries taken above
  // are not reached, as at most num_pages - count come back): one or two pages of a row
  // by a thread, more by a warp, and more than kLongRow by all threads together.
  auto move = [&](int b, int first, int step) {
    const int p0 = b > 0 ? pag[b - 1] : 0, k0 = b > 0 ? bak[b - 1] : 0;
    int32_t* const mine = table + (int64_t)b * max_blocks;
    if (row[b] < 0) {
      int32_t* const to = mine + div.up(row[b] & kIntMax);
#pragma unroll 4
      for (int i = first; i < pag[b] - p0; i += step) to[i] = ring[ring_at(p0 + i)];
    }
    const int n = min(bak[b], given) - k0;
#pragma unroll 4
    for (int i = first; i < n; i += step) ring[ring_at(count + k0 + i)] = mine[from[b] + i];
  };
  const int warps = blocks * (kPlanThreads / 32), w = rank * (kPlanThreads / 32) + (t >> 5);
  // lane l of warp w takes the rows (k + l) warps + (w + l) % warps: no two lanes in a bank
  auto row_at = [&](int k, int l) { return (k + l) * warps + ((w + l) & (warps - 1)); };
  for (int k = 0; k * warps < batch; k += 32) {
    const int b = row_at(k, lane);
    const int n = b < batch ? max(pag[b] - (b > 0 ? pag[b - 1] : 0),
                                  bak[b] - (b > 0 ? bak[b - 1] : 0))
                            : 0;
    if (n > 0 && n <= 2) move(b, 0, 1);
    for (uint32_t m = __ballot_sync(0xffffffffu, n > 2 && n <= kLongRow); m != 0; m &= m - 1)
      move(row_at(k, __ffs(m) - 1), lane, 32);
  }
  for (int b0 = 0; s_long && b0 < batch; b0 += 32) {
    const int b = b0 + lane;
    const bool lng = b < batch && (pag[b] - (b > 0 ? pag[b - 1] : 0) > kLongRow ||
                                   bak[b] - (b > 0 ? bak[b - 1] : 0) > kLongRow);
    for (uint32_t m = __ballot_sync(0xffffffffu, lng); m != 0; m &= m - 1)
      move(b0 + __ffs(m) - 1, rank * kPlanThreads + t, blocks * kPlanThreads);
  }
  if (!kSlots) cluster_wait();
  if (rank > 0) return;
  for (int b = r0; b < r1; ++b) got[b] = len[b];
  if (t == 0) {
    const int x = head + taken;
    pool_out[0] = x >= num_pages ? x - num_pages : x;
    pool_out[1] = count - taken + given;
  }
}

// The slots of granted rows from what page_plan_kernel has written: lengths, prefix
// sums, page table and the first slot of each row (-1: refused).  Another warp may be
// writing that one again, with the same value.  A warp takes 256 slots on end; its
// time is a chain of dependent reads: prefix sums (two or three steps of 32 guesses,
// for its first and last token at once), rows, first slots, pages.
__global__ void __launch_bounds__(256) page_slots_kernel(const int32_t* __restrict__ got,
                                                         const int32_t* __restrict__ cu,
                                                         const int32_t* __restrict__ table,
                                                         int batch, int B, int max_blocks,
                                                         int num_pages, int32_t* slots,
                                                         int max_new) {
  const int lane = threadIdx.x & 31;
  const int w0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * 256;
  const BlockDiv div(B);
  grid_wait();
  if (w0 >= max_new) return;
  const int tokens = cu[batch];
  const int last = min(w0 + 256, tokens) - 1;
  // the first row whose sum lies above x, for x = w0 and x = last
  int at[2] = {0, 0}, len[2] = {batch, batch};
  while (w0 < tokens && max(len[0], len[1]) > 1) {
    int step[2], sum[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      step[e] = (len[e] + 31) / 32;
      sum[e] = cu[1 + at[e] + min((lane + 1) * step[e], len[e]) - 1];
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int k = __ffs(__ballot_sync(0xffffffffu, sum[e] > (e == 0 ? w0 : last))) - 1;
      at[e] += k * step[e];
      len[e] = min(step[e], len[e] - k * step[e]);
    }
  }
  const int lo = at[0], rows = at[1] - at[0] + 1;
  // lane r holds row lo + r: first token, end, position of the first token, granted or not
  int c = 0, end = 0, p0 = 0;
  bool granted = false;
  if (w0 < tokens && lane < rows) {
    c = cu[lo + lane];
    end = cu[lo + lane + 1];
    p0 = got[lo + lane] - (end - c);
    granted = end > c && slots[c] >= 0;
  }
  auto slot_of = [&](int page, int r) {
    return page >= 0 && page < num_pages ? page * B + r : -1;
  };
  if (rows == 1 && last == w0 + 255) {
    // one row: 8 slots on end a thread, in at most two blocks (B >= 16)
    c = __shfl_sync(0xffffffffu, c, 0);
    p0 = __shfl_sync(0xffffffffu, p0, 0);
    granted = __shfl_sync(0xffffffffu, granted, 0);
    const int i0 = w0 + lane * 8;
    int out[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) out[u] = -1;
    if (granted) {
      const int pos = p0 + i0 - c, j = div(pos), r = pos - j * B, left = B - r;
      const int32_t* w = table + (int64_t)lo * max_blocks + j;
      const int a = w[0], z = left < 8 ? w[1] : a;
#pragma unroll
      for (int u = 0; u < 8; ++u) out[u] = u < left ? slot_of(a, r + u) : slot_of(z, u - left);
    }
    *reinterpret_cast<int4*>(slots + i0) = make_int4(out[0], out[1], out[2], out[3]);
    *reinterpret_cast<int4*>(slots + i0 + 4) = make_int4(out[4], out[5], out[6], out[7]);
    return;
  }
  if (rows <= 32) {
    // row of token w0 + 32 u + lane: those that end before it are counted
    int k[8] = {0, 0, 0, 0, 0, 0, 0, 0}, out[8];
    for (int r = 0; r < rows - 1; ++r) {
      const int e = __shfl_sync(0xffffffffu, end, r);
#pragma unroll
      for (int u = 0; u < 8; ++u) k[u] += e <= w0 + 32 * u + lane;
    }
    int place[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = w0 + 32 * u + lane;
      const int first = __shfl_sync(0xffffffffu, c, k[u]), p = __shfl_sync(0xffffffffu, p0, k[u]);
      const bool ok = __shfl_sync(0xffffffffu, granted, k[u]) && i < tokens;
      const int pos = p + i - first, j = ok ? div(pos) : 0;
      place[u] = pos - j * B;
      out[u] = ok ? table[(int64_t)(lo + k[u]) * max_blocks + j] : -1;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = w0 + 32 * u + lane;
      if (i < max_new) slots[i] = slot_of(out[u], place[u]);
    }
    return;
  }
#pragma unroll 4
  for (int u = 0; u < 8; ++u) {
    const int i = w0 + 32 * u + lane;
    int slot = -1;
    if (i < tokens) {
      const int b = lo + row_above(cu + 1 + lo, rows, i);
      const int f = cu[b];
      if (slots[f] >= 0) {
        const int pos = got[b] - (cu[b + 1] - f) + i - f, j = div(pos);
        slot = slot_of(table[(int64_t)b * max_blocks + j], pos - j * B);
      }
    }
    if (i < max_new) slots[i] = slot;
  }
}

cudaError_t launch_page_plan(const int32_t* have, const int32_t* want, const int32_t* keep,
                             int batch, int B, int32_t* table, int max_blocks, int num_pages,
                             int32_t* ring, const int32_t* pool, int32_t* pool_out, int32_t* got,
                             int32_t* cu, int32_t* slots, int max_new, cudaStream_t st) {
  const size_t smem = (size_t)batch * 6 * sizeof(int);
  // (the rule's two sides are measured at the top)
  const bool one = max_new <= 8 * kPlanThreads && batch <= 4 * kPlanThreads;
  const auto kernel = one ? page_plan_kernel<true> : page_plan_kernel<false>;
  if (smem > 46 * 1024) {  // the static arrays count too
    // (the limit is the kernel's, for all host threads: always that of the largest batch)
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kPlanMaxBatch * 6 * (int)sizeof(int));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 8;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(one ? 1 : 8);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = one ? 1 : 2;
  const cudaError_t e =
      cudaLaunchKernelEx(&cfg, kernel, have, want, keep, batch, B, table, max_blocks, num_pages,
                         ring, pool, pool_out, got, cu, slots, max_new);
  if (e != cudaSuccess || one || max_new == 0) return e;
  cfg.gridDim = dim3((unsigned)((max_new + 2047) / 2048));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, page_slots_kernel, (const int32_t*)got, (const int32_t*)cu,
                            (const int32_t*)table, batch, B, max_blocks, num_pages, slots,
                            max_new);
}

}  // namespace ssa
