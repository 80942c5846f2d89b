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
// One launch.  Every block of a cluster adds up the needs of all sequences by itself (a few loads a
// thread), so that all of them come to the same verdict; only when the last has read the lengths (the
// cluster's barrier) are they changed.  A call that cannot be met changes nothing.  Then the blocks share
// the tokens (or the pages that go back), each finding its sequence by a search of the offsets in shared
// memory.  Bound by latency: launch, two dependent reads and the barrier.
#include "internal.h"
#include "ptx.cuh"

namespace attn {

namespace {

constexpr int kPgThreads = 1024;
constexpr int kPgChunk = 2048;  // sequences whose offsets are in shared memory at a time
constexpr int kPgBlocks = 8;    // of a cluster

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

template <bool EXTEND>
__global__ void __launch_bounds__(kPgThreads) attn_pages_kernel(const PagesParams p) {
  __shared__ PagesShared s;
  const int rank = blockIdx.x, step = gridDim.x * kPgThreads;  // the grid is one cluster
  const int tid = rank * kPgThreads + threadIdx.x;
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
    if (EXTEND)
      for (int i = tid; i < p.total; i += step) p.slots[i] = -1;
    return;
  }
  if (EXTEND) {  // rows of no sequence
    for (int i = tid; i < row0; i += step) p.slots[i] = -1;
    for (int i = row1 + tid; i < p.total; i += step) p.slots[i] = -1;
  }
  const int page_mask = (1 << p.page_log2) - 1;
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
      // four packed rows a thread, which search once and share their pages' entries
      const int lo = s.start[0], hi = s.start[n];
      for (int g = (lo >> 2) + tid; g < (hi + 3) >> 2; g += step) {
        int slot[4];
        int u = last_at_most(s.start, n, max(g * 4, lo)), page = -1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int i = g * 4 + e;
          if (i < lo || i >= hi) continue;
          const int was = u;
          while (i >= s.start[u + 1]) ++u;
          const int t = s.len[u] + (i - s.start[u]), in_page = t & page_mask;
          if (page < 0 || u != was || in_page == 0) {
            const int j = t >> p.page_log2, have = pages_of(s.len[u], p.page_log2);
            int32_t* entry = p.block_table + static_cast<size_t>(b0 + u) * p.max_pages + j;
            page = j < have ? *entry : p.free_pages[top - (base + s.off[u] + j - have)];
            if (j >= have && in_page == 0) *entry = page;  // (by the page's first token)
            if (page < 0 || page >= p.num_pages) {
              latch_status(p.status, kStatusBadLengths);
              page = -1;
            }
          }
          slot[e] = page < 0 ? -1 : (page << p.page_log2) + in_page;
        }
        if (g * 4 >= lo && g * 4 + 4 <= hi) {
          *reinterpret_cast<int4*>(p.slots + g * 4) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (g * 4 + e >= lo && g * 4 + e < hi) p.slots[g * 4 + e] = slot[e];
        }
      }
    } else {
      for (int x = tid; x < s.off[n]; x += step) {
        const int u = last_at_most(s.off, n, x);
        int32_t* entry = p.block_table + static_cast<size_t>(b0 + u) * p.max_pages + s.start[u] + (x - s.off[u]);
        p.free_pages[top - (base + x)] = *entry;
        *entry = -1;
      }
    }
    if (rank == 0)
      for (int u = threadIdx.x; u < n; u += kPgThreads)
        p.seqlens[b0 + u] = EXTEND ? s.len[u] + (s.start[u + 1] - s.start[u]) : p.lengths[b0 + u];
    base += s.off[n];
  }
  if (tid == 0) *p.n_free = EXTEND ? n_free - static_cast<int>(all) : n_free + static_cast<int>(all);
}

}  // namespace

template <bool EXTEND>
static int launch_pages(const PagesArgs& a, cudaStream_t stream) {
  PagesParams p = {a.block_table, a.seqlens, a.lengths, a.free_pages, a.n_free, a.slots,
                   device_status_ptr(), a.num_pages, 0, a.max_pages, a.total, a.B};
  if (!p.status) return -5;
  while ((1 << p.page_log2) < a.page_size) ++p.page_log2;
  // one block where it has a few rows a thread at most
  const long long rows = EXTEND ? a.total : static_cast<long long>(a.B) * a.max_pages;
  const int blocks = rows > 4 * kPgThreads ? kPgBlocks : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kPgThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = blocks;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_pages_kernel<EXTEND>, p) == cudaSuccess ? 0 : -5;
}

int launch_pages_extend(const PagesArgs& a, cudaStream_t stream) { return launch_pages<true>(a, stream); }
int launch_pages_trim(const PagesArgs& a, cudaStream_t stream) { return launch_pages<false>(a, stream); }

}  // namespace attn
