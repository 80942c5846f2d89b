// A few new tokens of each sequence over a paged 16-bit cache: at most 16 (token, query head) rows per
// key/value head, so one token of any group the decode kernels take, or a few tokens of a small group.
//
// With so few rows a 128-row tile of the kernel for chunks (attn_fwd_paged.cu: two blocks on an SM, 64-key
// steps) spends its time on rows that do not exist: 0.9 us a step.  Here a block is a split of one
// (sequence, key/value head)'s visible keys, several blocks share an SM, and the two products run on
// warp-level tiles with the rows as columns (attn_rows.cuh).  The visible keys of the chunk are walked as
// 64-key stages: those that hold sinks, then those from the window's first key to the sequence's end.  A
// producer warp brings the stages page by page with TMA; the block-table entries of the whole split are
// read at its start.  At most eight splits merge inside a cluster; more go through the workspace and the
// paged merge kernel.
//
// Bound by HBM: 4 d bytes per visible cached token and head.  One token of 16 sequences (Hq=32 Hkv=8
// d=64, 16-token pages) under a 4,095-key window with 4 sinks, 134 MB: 26 us of kernel time (5.2 TB/s)
// against the tile kernel's 53; one of 64 sequences of 1k-32k tokens (Hq=64 Hkv=8 d=128 bf16, 64-token
// pages, 4.27 GB): 594 us back to back (7.2 TB/s; reads alone run faster than a copy).
#include "attn_decode.cuh"
#include "attn_rows.cuh"

namespace attn {

namespace {

constexpr int kFewRows = 16;
constexpr int kFewMaxStages = 2048 / kDecTok;  // of a split (row_split_tokens)

struct FewParams {
  const uint16_t* q;  // [total_q, Hq, D]
  const int32_t* block_table;
  const int32_t* cu_q;
  const int32_t* seqlens;
  int* status;
  int page_log2, max_pages, num_pages, total_q, max_q, max_k;
  int Hq, Hkv, G, window, sinks, split_stages;
  float sl2;
  float* ws_o;   // partial states, or null with a cluster
  float* ws_ml;
  uint16_t* out;
  float* lse;
  int n_splits, cluster;
};

template <int D>
struct FewLayout {
  static constexpr uint32_t kTensor = kDecTok * D * 2;  // K or V of one stage
  static constexpr uint32_t kStage = 2 * kTensor;
  static constexpr uint32_t kRing = kDecStages * kStage;
  static constexpr uint32_t kRed = kDecWarps * kFewRows * (D + 2) * 4;  // reuses the ring
  static constexpr uint32_t kFin = kRed;
  static_assert(kFin + kFewRows * (D + 2) * 4 <= kRing, "merge scratch must fit in the ring");
  static constexpr uint32_t kBar = kRing;
  static constexpr uint32_t kMisc = kBar + 2 * kDecStages * 8;
  static constexpr uint32_t kPages = kMisc + 16;  // first pool row of each page of the split, or -1
  static constexpr uint32_t kBytes = kPages + kFewMaxStages * 4 * 4 + 1024;
};

// Blocks that share an SM, by shared memory (97 KB at d = 128, 49 KB at d = 64) and registers.
template <int D>
constexpr int few_blocks_per_sm() {
  return D == 128 ? 2 : 4;
}

}  // namespace

template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(kDecThreads, few_blocks_per_sm<D>())
    attn_paged_few_kernel(const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const FewParams p) {
  using L = FewLayout<D>;
  const int split = blockIdx.x;
  const int hk = blockIdx.y;
  const int b = blockIdx.z;
  if (threadIdx.x == 0) griddep_launch_dependents();  // the merge may be scheduled (it waits)
  const int c0 = p.cu_q[b], n = p.cu_q[b + 1] - c0;
  const int len = p.seqlens[b];
  if (c0 < 0 || n < 0 || n > p.max_q || n > p.total_q - c0 || len < n || len > p.max_k ||
      ((len - 1) >> p.page_log2) >= p.max_pages) {
    if (split == 0 && hk == 0 && threadIdx.x == 0) latch_status(p.status, kStatusBadLengths);
    return;
  }
  if (n == 0) return;
  const int rows = n * p.G;
  const int pos0 = len - n;
  // 64-key stages of the visible keys: `sink_st` of them from key 0, then from stage w_begin on
  const int w_begin = p.window < 0 ? 0 : max(pos0 - p.window, 0) / kDecTok;
  const int sink_st = p.window < 0 ? 0 : min((min(p.sinks, len) + kDecTok - 1) / kDecTok, w_begin);
  const int all = sink_st + (len + kDecTok - 1) / kDecTok - w_begin;
  const int i0 = split * p.split_stages;
  const int n_stages = min(max(all - i0, 0), p.split_stages);
  auto stage_token = [&](int st) {
    const int i = i0 + st;
    return (i < sink_st ? i : w_begin + i - sink_st) * kDecTok;
  };
  auto out_row = [&](int row) {
    const int t = row / p.G;
    return static_cast<size_t>(c0 + t) * p.Hq + hk * p.G + (row - t * p.G);
  };
  if (n_stages == 0 && !p.cluster) {
    // no key of its own: the merge gives it no weight
    if (static_cast<int>(threadIdx.x) < rows)
      reinterpret_cast<float2*>(p.ws_ml)[out_row(threadIdx.x) * p.n_splits + split] =
          make_float2(-INFINITY, 0.0f);
    return;
  }

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  const uint32_t bars = base + L::kBar;
#define FULL(s) (bars + 8u * (s))
#define EMPTY(s) (bars + 8u * (kDecStages + (s)))
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::kMisc);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kDecStages; ++s) {
      mbar_init(FULL(s), 1);
      mbar_init(EMPTY(s), kDecWarps);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  const int box_log2 = min(p.page_log2, 6);  // rows of one TMA box: a page, or a stage's 64 of it

  if (warp == kDecWarps) {
    // ------------------------------------------------------------------ TMA producer
    int* page_row = reinterpret_cast<int*>(gbase + L::kPages);  // [stage][page of it]
    const int box = 1 << box_log2;
    const int pg_log2 = 6 - box_log2;  // log2 of the boxes of a stage
    const int32_t* tbl = p.block_table + static_cast<size_t>(b) * p.max_pages;
    for (int i = lane; i < n_stages << pg_log2; i += 32) {
      const int t = stage_token(i >> pg_log2) + (i & ((1 << pg_log2) - 1)) * box;
      int row = -1;
      if (t < len) {
        const int pg = tbl[t >> p.page_log2];
        if (pg >= 0 && pg < p.num_pages)
          row = (pg << p.page_log2) + (t & ((1 << p.page_log2) - 1));
        else
          latch_status(p.status, kStatusBadLengths);
      }
      page_row[i] = row;
    }
    __syncwarp();
    const uint64_t stream_policy = l2_policy_evict_first();
    const uint32_t box_bytes = static_cast<uint32_t>(box) * D * 2;
    int issued = 0;
    for (int st = 0; st < n_stages; ++st) {
      const int s = st % kDecStages;
      bool ok = true;
      if (lane == 0 && st >= kDecStages)
        ok = wait_bounded(EMPTY(s), ((st / kDecStages) - 1) & 1, abort_flag, p.status);
      if (!__shfl_sync(0xffffffffu, ok, 0)) break;
      const uint32_t kbuf = base + s * L::kStage;
      const int row = lane < (1 << pg_log2) ? page_row[(st << pg_log2) + lane] : -1;
      const uint32_t n_loads = __popc(__ballot_sync(0xffffffffu, row >= 0));
      if (lane == 0) mbar_arrive_expect_tx(FULL(s), n_loads * 2 * box_bytes);
      __syncwarp();
      if (row >= 0) {
        tma_load_4d_hint(kbuf + lane * box_bytes, &tm_k, FULL(s), 0, row, 0, hk, stream_policy);
        tma_load_4d_hint(kbuf + L::kTensor + lane * box_bytes, &tm_v, FULL(s), 0, row, 0, hk,
                         stream_policy);
      }
      issued = st + 1;
    }
    if (lane == 0)
      for (int st = (issued > kDecStages ? issued - kDecStages : 0); st < issued; ++st)
        wait_bounded(FULL(st % kDecStages), (st / kDecStages) & 1, nullptr, p.status, 100000000ull);
    return;  // the producer takes no part in the reduction below
  }

  // -------------------------------------------------------------------- compute warps
  const int g = lane >> 2, c = lane & 3;
  RowState<D, NT, BF16> rs;
  rs.init();
  uint32_t qf[NT][D / 16][2];
  int hi[NT][2], lo[NT][2];  // last and first key of the rows 2c, 2c + 1 of each column tile
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    const int row = u * 8 + g;
    const uint16_t* qr = p.q + out_row(row < rows ? row : 0) * D + 2 * c;
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks) {
      qf[u][ks][0] = row < rows ? *reinterpret_cast<const uint32_t*>(qr + ks * 16) : 0u;
      qf[u][ks][1] = row < rows ? *reinterpret_cast<const uint32_t*>(qr + ks * 16 + 8) : 0u;
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      hi[u][r] = pos0 + min((u * 8 + 2 * c + r) / p.G, n - 1);
      lo[u][r] = p.window < 0 ? 0 : hi[u][r] - p.window;
    }
  }
  // byte offset of (row, 64-channel half) in a stage laid out [box][half][box rows][128 B]
  auto stage_off = [&](int row, int half) -> uint32_t {
    return (static_cast<uint32_t>((row >> box_log2) * (D / 64) + half) << (box_log2 + 7)) +
           (static_cast<uint32_t>(row & ((1 << box_log2) - 1)) << 7);
  };
  // this lane's ldmatrix rows: matrix i = lane / 8 holds keys 8 (i % 2) .. of K (channels by i / 2)
  // and keys 8 (i / 2) .. of V (channels by i % 2)
  uint32_t k_row[D / 64], v_row[D / 64];
#pragma unroll
  for (int h = 0; h < D / 64; ++h) {
    k_row[h] = stage_off(warp * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), h);
    v_row[h] = stage_off(warp * 16 + (lane >> 4) * 8 + (lane & 7), h);
  }

  bool ok = true;
  for (int st = 0; st < n_stages; ++st) {
    const int s = st % kDecStages;
    if (!dec_warp_wait(FULL(s), (st / kDecStages) & 1, abort_flag, p.status)) {
      ok = false;
      break;
    }
    const uint32_t kbuf = base + s * L::kStage;
    const uint32_t vbuf = kbuf + L::kTensor;
    const int key0 = stage_token(st) + warp * 16;  // first key of this warp
    const int valid = len - key0;                  // keys of this warp the sequence has
    if (valid > 0) {
      if (valid < 16) {
        // Rows past the sequence: their weight is 0, and 0 times a NaN has to stay 0.
        for (int i = lane; i < (16 - valid) * (D / 8); i += 32) {
          const int rr = warp * 16 + valid + i / (D / 8);
          const int ch = i % (D / 8);
          *reinterpret_cast<uint4*>(gbase + (vbuf - base) + stage_off(rr, ch >> 3) +
                                    (((ch & 7) ^ (rr & 7)) << 4)) = make_uint4(0, 0, 0, 0);
        }
        __syncwarp();
      }
      float sc[NT][4] = {};
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const int chunk = ks * 2 + (lane >> 4);
        uint32_t a[4];
        ldmatrix_x4(kbuf + k_row[ks >> 2] + (((chunk & 7) ^ (lane & 7)) << 4), a[0], a[1], a[2], a[3]);
#pragma unroll
        for (int u = 0; u < NT; ++u) mma_m16n8k16<BF16>(sc[u], a, qf[u][ks][0], qf[u][ks][1]);
      }
      float x[NT][2][2];
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int key = key0 + g + 8 * k;
            const bool in = key <= hi[u][r] && (key >= lo[u][r] || key < p.sinks);
            x[u][k][r] = in ? sc[u][2 * k + r] * p.sl2 : -INFINITY;
          }
      uint32_t pb[NT][2];
      rs.step(x, pb);
#pragma unroll
      for (int t = 0; t < D / 16; ++t) {
        const int chunk = 2 * t + ((lane >> 3) & 1);
        uint32_t a[4];
        ldmatrix_x4_trans(vbuf + v_row[t >> 2] + (((chunk & 7) ^ (lane & 7)) << 4), a[0], a[1], a[2],
                          a[3]);
#pragma unroll
        for (int u = 0; u < NT; ++u) mma_m16n8k16<BF16>(rs.o[u][t], a, pb[u][0], pb[u][1]);
      }
      if (valid < 16) fence_proxy_async_smem();  // generic zeros before the next TMA write
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(EMPTY(s));
  }

  // ---------------------------------------------------- merge the four warps' states
  rs.finish();
  named_bar_sync(1, kDecWarps * 32);  // every warp is done with the ring
  ok = ok && (*abort_flag == 0);
  float* red = reinterpret_cast<float*>(gbase);  // [warp][row][D + 2]
  if (ok)
    rs.store(red + warp * kFewRows * (D + 2), rows, lane, [&](int t, int i) { return 16 * t + 8 * i + g; },
             [](int, int, float x) { return x; });
  named_bar_sync(1, kDecWarps * 32);
  const RowsOut w{p.ws_o, p.ws_ml, p.out, p.lse, p.n_splits, split, p.cluster != 0};
  merge_rows<D, BF16, kDecWarps, kFewRows, false>(red, reinterpret_cast<float*>(gbase + L::kFin), rows,
                                                  ok, n_stages > 0, w, out_row);
#undef FULL
#undef EMPTY
}

bool paged_few_rows(const PagedArgs& a) {
  return static_cast<long long>(a.max_q) * (a.Hq / a.Hkv) <= kFewRows && a.B <= 65535 &&
         a.Hkv <= 65535;
}

void paged_few_split(int B, int Hkv, int max_q, int max_k, int window, int sinks, int d,
                     int& n_splits, int& stages) {
  long long tokens = max_k;
  if (window >= 0) {
    // the window's keys with those of the stages its ends lie in, and the sinks' stages
    const long long near = static_cast<long long>(window) + max_q + 2 * kDecTok +
                           (static_cast<long long>(sinks) + kDecTok - 1) / kDecTok * kDecTok;
    if (near < tokens) tokens = near;
  }
  const int slots = 152 * (d == 128 ? few_blocks_per_sm<128>() : few_blocks_per_sm<64>());
  const int per = row_split_tokens(static_cast<long long>(B) * Hkv, tokens, slots);
  stages = per / kDecTok;
  const long long all = (tokens + kDecTok - 1) / kDecTok;
  n_splits = static_cast<int>((all + stages - 1) / stages);
}

template <int D, bool BF16>
static int launch_few_variant(const PagedArgs& a, cudaStream_t stream) {
  using L = FewLayout<D>;
  const uint64_t row = static_cast<uint64_t>(D) * 2;
  const uint64_t tokens = static_cast<uint64_t>(a.num_pages) * a.page_size;
  const uint32_t box_rows = static_cast<uint32_t>(a.page_size < kDecTok ? a.page_size : kDecTok);
  // {64 channels, token, channel half, head}: one box = box_rows tokens x both halves of d
  const uint64_t dims[4] = {64, tokens, D / 64, static_cast<uint64_t>(a.Hkv)};
  const uint64_t strides[3] = {row * a.Hkv, 128, row};
  const uint32_t box[4] = {64, box_rows, D / 64, 1};
  CUtensorMap tk, tv;
  if (!make_tmap_4d(&tk, a.k_pages, BF16, dims, strides, box) ||
      !make_tmap_4d(&tv, a.v_pages, BF16, dims, strides, box))
    return -5;
  FewParams p = {};
  p.q = static_cast<const uint16_t*>(a.q);
  p.block_table = a.block_table;
  p.cu_q = a.cu_q;
  p.seqlens = a.seqlens;
  p.status = device_status_ptr();
  if (!p.status) return -5;
  while ((1 << p.page_log2) < a.page_size) ++p.page_log2;
  p.max_pages = a.max_pages;
  p.num_pages = a.num_pages;
  p.total_q = a.total_q;
  p.max_q = a.max_q;
  p.max_k = a.max_k;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.G = a.Hq / a.Hkv;
  p.window = a.window;
  p.sinks = a.sinks;
  p.sl2 = a.scale * 1.4426950408889634f;
  p.out = static_cast<uint16_t*>(a.o);
  p.lse = a.lse;
  paged_few_split(a.B, a.Hkv, a.max_q, a.max_k, a.window, a.sinks, D, p.n_splits, p.split_stages);
  p.cluster = p.n_splits <= kMaxCluster;
  if (!p.cluster) paged_parts(a, D, p.n_splits, p.ws_o, p.ws_ml);
  auto kern = a.max_q * p.G <= 8 ? attn_paged_few_kernel<D, BF16, 1> : attn_paged_few_kernel<D, BF16, 2>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kBytes) !=
      cudaSuccess)
    return -5;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.n_splits, a.Hkv, a.B);
  cfg.blockDim = dim3(kDecThreads);
  cfg.dynamicSmemBytes = L::kBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.n_splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster ? 1 : 0;
  if (cudaLaunchKernelEx(&cfg, kern, tk, tv, p) != cudaSuccess) return -5;
  return p.cluster ? 0 : launch_paged_merge(a, p.n_splits, stream);
}

int launch_attn_paged_few(const PagedArgs& a, cudaStream_t stream) {
  if (a.d == 64)
    return a.bf16 ? launch_few_variant<64, true>(a, stream) : launch_few_variant<64, false>(a, stream);
  return a.bf16 ? launch_few_variant<128, true>(a, stream) : launch_few_variant<128, false>(a, stream);
}

}  // namespace attn
