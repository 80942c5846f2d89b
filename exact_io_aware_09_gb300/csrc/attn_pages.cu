// Page lists of a paged cache, kept on the GPU: pages of a free list given to sequences that grow, and
// taken back from sequences that are cut short.  Nothing comes from or goes to the host, so a captured
// step can allocate its own pages.
//
// The free list is a stack, free_pages[0 .. n_free - 1].  With L_b cached and n_b new tokens and pages of
// P tokens, sequence b takes need_b = ceil((L_b + n_b) / P) - ceil(L_b / P) pages; numbered over the
// sequences in order, page k is free_pages[n_free - 1 - k].  Trimming gives them back in the same
// numbering, so that it undoes an extension exactly.  Which page a token gets depends on the numbers
// alone, not on the order in which threads run.
//
// One launch, but for whole prompts.  Every block of a cluster adds up the needs of all sequences by itself
// (a few loads a thread), so that all of them come to the same verdict; only when the last has read the
// lengths (the cluster's barrier) are they changed.  A call that cannot be met changes nothing.  Then the blocks share
// the tokens (or the pages that go back), each finding its sequence by a search of the offsets in shared
// memory.  Bound by latency: launch, two dependent reads and the barrier.
//
// Whole prompts' slots are more than a cluster's eight SMs write quickly (1.2 M tokens of 256 prompts: 40 us).
// From kPgManyRows rows on a first launch over all SMs writes the slots and the new entries, which nothing
// else reads, and a second of one block comes to the same verdict from what the first left unchanged, and
// changes the lengths and the list's: the same tokens in 15 us.
#include "internal.h"
#include "ptx.cuh"

namespace attn {

namespace {

constexpr int kPgThreads = 1024;
constexpr int kPgChunk = 2048;  // sequences whose offsets are in shared memory at a time
constexpr int kPgBlocks = 8;    // of a cluster
constexpr int kPgManyRows = 1 << 16, kPgManyBlocks = 152;

// What a launch does: everything (one cluster), the slots and entries, or the lengths and the list's.
enum { kPgAll, kPgSlots, kPgLengths };

struct PagesParams {
  int32_t* block_table;    // [B, max_pages]
  int32_t* seqlens;        // [B]
  const int32_t* lengths;  // extend: [B + 1] packed offsets of the new tokens; trim: [B] tokens kept
  int32_t* free_pages;     // [num_pages]
  int32_t* n_free;
  int32_t* slots;          // extend: [total]
  int* status;
  int num_pages, page_log2, max_pages, total, B;
};

struct PagesShared {
  int start[kPgChunk + 1];  // extend: first packed row of each sequence and the end; trim: pages kept
  int len[kPgChunk];        // extend: tokens before the new ones
  int off[kPgChunk + 1];    // number of each sequence's first page, less that of the chunk's first
  long long warp_sum[kPgThreads / 32];
  int bad;
};

__device__ __forceinline__ int pages_of(int tokens, int log2) {
  return static_cast<int>((static_cast<unsigned>(tokens) + ((1u << log2) - 1)) >> log2);
}

// Loads the chunk of sequences from b0 on; returns its pages (taken, or given back), with off[] their
// exclusive sums.  Marks s.bad for lengths that no call may have.
template <bool EXTEND>
__device__ __forceinline__ long long load_chunk(const PagesParams& p, PagesShared& s, int b0) {
  constexpr int kPer = kPgChunk / kPgThreads;
  const int n = min(kPgChunk, p.B - b0);
  const long long reach = static_cast<long long>(p.max_pages) << p.page_log2;
  __syncthreads();  // the last chunk's readers are done
  long long mine[kPer], sum = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int u = threadIdx.x * kPer + i;
    mine[i] = 0;
    if (u < n) {
      const int L = p.seqlens[b0 + u];
      if (EXTEND) {
        const int c0 = p.lengths[b0 + u], c1 = p.lengths[b0 + u + 1];
        const bool wrong = L < 0 || c0 < 0 || c1 < c0 || c1 > p.total ||
                           static_cast<long long>(L) + (c1 - c0) > reach;
        bad = bad || wrong;
        if (!wrong) mine[i] = pages_of(L + (c1 - c0), p.page_log2) - pages_of(L, p.page_log2);
        s.start[u] = c0;
        if (u == n - 1) s.start[n] = c1;
        s.len[u] = L;
      } else {
        const int keep = p.lengths[b0 + u];
        const bool wrong = keep < 0 || keep > L || L > reach;
        bad = bad || wrong;
        const int left = wrong ? 0 : pages_of(keep, p.page_log2);
        if (!wrong) mine[i] = pages_of(L, p.page_log2) - left;
        s.start[u] = left;
      }
    }
    sum += mine[i];
  }
  if (bad) s.bad = 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long incl = sum;
#pragma unroll
  for (int sh = 1; sh < 32; sh <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, incl, sh);
    if (lane >= sh) incl += up;
  }
  if (lane == 31) s.warp_sum[warp] = incl;
  __syncthreads();
  long long before = 0, all = 0;
  for (int w = 0; w < kPgThreads / 32; ++w) {
    const long long v = s.warp_sum[w];
    if (w < warp) before += v;
    all += v;
  }
  // (sums past 2^31 belong to calls that are refused)
  long long at = before + incl - sum;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int u = threadIdx.x * kPer + i;
    if (u < n) s.off[u] = static_cast<int>(at);
    at += mine[i];
  }
  if (threadIdx.x == 0) s.off[n] = static_cast<int>(all);
  __syncthreads();
  return all;
}

// The last of the ascending a[0 .. n - 1] that is at most x (a[0] is).
__device__ __forceinline__ int last_at_most(const int* a, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// The page of token t of the chunk's sequence u: one it has, or its new one, which goes into the table with
// its first token; -1 for an entry outside the pool, which is reported.
__device__ __forceinline__ int page_of_token(const PagesParams& p, const PagesShared& s, int b0, int u, int t,
                                             int base, int top) {
  const int j = t >> p.page_log2, have = pages_of(s.len[u], p.page_log2);
  int32_t* entry = p.block_table + static_cast<size_t>(b0 + u) * p.max_pages + j;
  const int page = j < have ? *entry : p.free_pages[top - (base + s.off[u] + j - have)];
  if (j >= have && (t & ((1 << p.page_log2) - 1)) == 0) *entry = page;
  if (page >= 0 && page < p.num_pages) return page;
  latch_status(p.status, kStatusBadLengths);
  return -1;
}

// Slots of the chunk's n sequences; `top`: the list's place of page 0, `base` the number of the chunk's first
// page.  A thread takes sixteen rows where there are many: they are mostly one sequence's, and lie in two
// pages at most.  (Rows go to 2^31 - 1: what steps past the last is unsigned.)
__device__ __forceinline__ void give_slots(const PagesParams& p, const PagesShared& s, int b0, int n, int base,
                                           int top, unsigned tid, unsigned step) {
  const int page_mask = (1 << p.page_log2) - 1;
  const unsigned lo = s.start[0], hi = s.start[n];
  const unsigned per = hi - lo <= step ? 1 : 16;
  if (lo >= hi) return;
  for (unsigned g = lo / per + tid; g <= (hi - 1) / per; g += step) {
    const int i0 = max(g * per, lo), i1 = min(g * per + per, hi);
    int u = last_at_most(s.start, n, i0);
    if (per == 16 && i1 - i0 == 16 && s.start[u + 1] >= i1) {
      const int t = s.len[u] + (i0 - s.start[u]), cut = page_mask + 1 - (t & page_mask);
      const int a = page_of_token(p, s, b0, u, t, base, top);
      const int b = cut < 16 ? page_of_token(p, s, b0, u, t + cut, base, top) : -1;
      const int at_a = (a << p.page_log2) + (t & page_mask), at_b = (b << p.page_log2) - cut;
      int slot[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) slot[e] = e < cut ? (a < 0 ? -1 : at_a + e) : b < 0 ? -1 : at_b + e;
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        *reinterpret_cast<int4*>(p.slots + i0 + e) = make_int4(slot[e], slot[e + 1], slot[e + 2], slot[e + 3]);
      continue;
    }
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
      while (i >= s.start[u + 1]) ++u;
      const int t = s.len[u] + (i - s.start[u]);
      const int page = page_of_token(p, s, b0, u, t, base, top);
      p.slots[i] = page < 0 ? -1 : (page << p.page_log2) + (t & page_mask);
    }
  }
}

template <bool EXTEND, int WHAT>
__global__ void __launch_bounds__(kPgThreads) attn_pages_kernel(const PagesParams p) {
  __shared__ PagesShared s;
  if (WHAT == kPgSlots) griddep_launch_dependents();
  if (WHAT == kPgLengths) griddep_wait();
  const int rank = blockIdx.x;
  const unsigned step = gridDim.x * kPgThreads;  // (kPgAll: the grid is one cluster)
  const unsigned tid = rank * kPgThreads + threadIdx.x;
  if (threadIdx.x == 0) s.bad = 0;
  const int n_free = *p.n_free;
  const int row0 = EXTEND ? p.lengths[0] : 0, row1 = EXTEND ? p.lengths[p.B] : 0;
  long long all = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPgChunk) all += load_chunk<EXTEND>(p, s, b0);
  int refuse = 0;
  if (s.bad || n_free < 0 || n_free > p.num_pages)
    refuse = kStatusBadLengths;
  else if (EXTEND && all > n_free)
    refuse = kStatusNoPages;
  else if (!EXTEND && n_free + all > p.num_pages)
    refuse = kStatusBadLengths;
  cluster_sync();  // every block has read the lengths and the list's, which change from here on
  if (refuse != 0) {
    if (tid == 0) latch_status(p.status, refuse);
    if (EXTEND && WHAT != kPgLengths)
      for (unsigned i = tid; i < static_cast<unsigned>(p.total); i += step) p.slots[i] = -1;
    return;
  }
  if (EXTEND && WHAT != kPgLengths) {  // rows of no sequence
    for (unsigned i = tid; i < static_cast<unsigned>(row0); i += step) p.slots[i] = -1;
    for (unsigned i = row1 + tid; i < static_cast<unsigned>(p.total); i += step) p.slots[i] = -1;
  }
  // the list's place of page 0
  const int top = EXTEND ? n_free - 1 : n_free + static_cast<int>(all) - 1;
  int base = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPgChunk) {
    const int n = min(kPgChunk, p.B - b0);
    if (p.B > kPgChunk) {
      load_chunk<EXTEND>(p, s, b0);
      cluster_sync();  // every block has this chunk's lengths
    }
    if (EXTEND) {
      if (WHAT != kPgLengths) give_slots(p, s, b0, n, base, top, tid, step);
    } else {
      for (int x = tid; x < s.off[n]; x += step) {  // (at most 2^27 pages)
        const int u = last_at_most(s.off, n, x);
        int32_t* entry = p.block_table + static_cast<size_t>(b0 + u) * p.max_pages + s.start[u] + (x - s.off[u]);
        const int page = *entry;  // (as it is, so that the numbering holds; one outside the pool is reported)
        if (page < 0 || page >= p.num_pages) latch_status(p.status, kStatusBadLengths);
        p.free_pages[top - (base + x)] = page;
        *entry = -1;
      }
    }
    if (WHAT != kPgSlots && rank == 0)
      for (int u = threadIdx.x; u < n; u += kPgThreads)
        p.seqlens[b0 + u] = EXTEND ? s.len[u] + (s.start[u + 1] - s.start[u]) : p.lengths[b0 + u];
    base += s.off[n];
  }
  if (WHAT != kPgSlots && tid == 0) *p.n_free = EXTEND ? n_free - static_cast<int>(all) : n_free + static_cast<int>(all);
}

}  // namespace

template <bool EXTEND>
static int launch_pages(const PagesArgs& a, cudaStream_t stream) {
  PagesParams p = {a.block_table, a.seqlens, a.lengths, a.free_pages, a.n_free, a.slots,
                   device_status_ptr(), a.num_pages, 0, a.max_pages, a.total, a.B};
  if (!p.status) return -5;
  while ((1 << p.page_log2) < a.page_size) ++p.page_log2;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kPgThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  cfg.attrs = attr;
  if (EXTEND && a.total >= kPgManyRows) {
    cfg.gridDim = dim3(kPgManyBlocks);
    if (cudaLaunchKernelEx(&cfg, attn_pages_kernel<true, kPgSlots>, p) != cudaSuccess) return -5;
    cfg.gridDim = dim3(1);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_pages_kernel<true, kPgLengths>, p) == cudaSuccess ? 0 : -5;
  }
  // one block where it has a few rows a thread at most
  const long long rows = EXTEND ? a.total : static_cast<long long>(a.B) * a.max_pages;
  const int blocks = rows > 4 * kPgThreads ? kPgBlocks : 1;
  cfg.gridDim = dim3(blocks);
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_pages_kernel<EXTEND, kPgAll>, p) == cudaSuccess ? 0 : -5;
}

int launch_pages_extend(const PagesArgs& a, cudaStream_t stream) { return launch_pages<true>(a, stream); }
int launch_pages_trim(const PagesArgs& a, cudaStream_t stream) { return launch_pages<false>(a, stream); }

}  // namespace attn
