// Moving tokens of the paged compressed cache: new tokens into pages, and the
// tokens that an eviction keeps into fresh pages.
//
// Both move, per (token, head), W code words (a plane each), a norm and a row
// of V; bound by memory. A block takes a tile of tokens of one head, looks up
// their places once, then copies plane by plane (lanes along tokens, so that
// a page's part of a plane is one contiguous access) and V in 16-byte pieces.
// Writing up to 2047 tokens of four sequences (8 heads, d = 128, b = 4; 22 MB)
// takes 9.4 us (1024 blocks, where 592 are resident: a wave and most of another),
// one token of 64 sequences 4.6 us; cutting 32 heads from 32768 to 8192 slots
// 65 us, 25 of them the choice.
//
// Which tokens an eviction keeps: per (sequence, head) a block finds the
// rank-th largest mass of the middle slots by three histogram passes over the
// ordered bits (11 + 11 + 10), then counts and writes the kept slots warp by
// warp in slot order, so the result does not depend on timing.

#include <cooperative_groups.h>

#include <algorithm>

#include "octo_paged.cuh"

namespace octo {
namespace paged {

constexpr int64_t kNone = -1;
constexpr int kBins = 2048 + 4;
constexpr int kHeld = 36000;  // slots of a block whose ordered bits fit into shared memory beside the bins

// Copies nt tokens of head h. s_src: token's offset in the source's plane 0
// and s_srow its row in the source gamma (kNone: a token without a source,
// written as zeros); s_dst: place in the destination pool as (page * heads +
// head) * page_size + offset (kNone: dropped), and s_page its page * heads +
// head.
struct MoveArgs {
  const uint32_t* src_packed;
  const float* src_gamma;
  const uint4* src_V;      // 16-byte pieces
  int64_t src_plane;       // words between planes of the source
  uint32_t* packed;
  float* gamma;
  uint4* V;
  int W, page_size, pieces;  // pieces: 16-byte pieces of a V row
};

template <int THREADS, int TILE>
__device__ __forceinline__ void move_tile(const MoveArgs& a, const int64_t* s_src, const int64_t* s_srow,
                                          const int64_t* s_vsrc, const int64_t* s_dst, const int64_t* s_page, int nt) {
  // batches of 8 loads, then their stores: the compiler may not move a load
  // past a store to memory that might be the same
  constexpr int N = 8;
  const int P = a.page_size;
  for (int k0 = threadIdx.x; k0 < a.W * TILE; k0 += N * THREADS) {
    uint32_t v[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int k = k0 + u * THREADS, w = k / TILE, t = k % TILE;
      const bool on = k < a.W * TILE && t < nt && s_src[t] >= 0;
      v[u] = on ? __ldg(a.src_packed + s_src[t] + w * a.src_plane) : 0u;
    }
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int k = k0 + u * THREADS, w = k / TILE, t = k % TILE;
      if (k >= a.W * TILE || t >= nt || s_dst[t] < 0) continue;
      const int64_t page = s_page[t];
      a.packed[page * a.W * P + static_cast<int64_t>(w) * P + (s_dst[t] - page * P)] = v[u];
    }
  }
  for (int t = threadIdx.x; t < nt; t += THREADS)
    if (s_dst[t] >= 0) a.gamma[s_dst[t]] = s_srow[t] < 0 ? 0.0f : __ldg(a.src_gamma + s_srow[t]);
  if (a.V) {
    for (int k0 = threadIdx.x; k0 < nt * a.pieces; k0 += N * THREADS) {
      uint4 v[N];
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const int k = k0 + u * THREADS, t = k / a.pieces, p = k - t * a.pieces;
        const bool on = k < nt * a.pieces && s_vsrc[t] >= 0;
        v[u] = on ? __ldg(a.src_V + s_vsrc[t] + p) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const int k = k0 + u * THREADS, t = k / a.pieces, p = k - t * a.pieces;
        if (k < nt * a.pieces && s_dst[t] >= 0) a.V[s_dst[t] * a.pieces + p] = v[u];
      }
    }
  }
}

// ---- new tokens into pages ----------------------------------------------------
struct WriteArgs {
  Table t;
  MoveArgs m;
  const int32_t* starts;
  const int32_t* cu;
  int64_t n_rows, v_row, v_head;  // V strides in 16-byte pieces
};

template <int TILE>
__global__ void __launch_bounds__(256) paged_write_kernel(const __grid_constant__ WriteArgs a) {
  __shared__ int64_t s_src[TILE], s_srow[TILE], s_vsrc[TILE], s_dst[TILE], s_page[TILE];
  const int h = blockIdx.y;
  const int64_t r0 = static_cast<int64_t>(blockIdx.x) * TILE;
  const int nt = static_cast<int>(min(static_cast<int64_t>(TILE), a.n_rows - r0));
  for (int t = threadIdx.x; t < nt; t += 256) {
    const int64_t r = r0 + t;
    // the sequence of row r: the last i with cu[i] <= r
    int lo = 0, hi = a.t.n_seqs;
    while (lo + 1 < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(a.cu + mid) <= r)
        lo = mid;
      else
        hi = mid;
    }
    const int64_t slot = static_cast<int64_t>(__ldg(a.starts + lo)) + (r - __ldg(a.cu + lo));
    int64_t to = kNone, page = 0;
    const bool held = r >= __ldg(a.cu + lo) && r < __ldg(a.cu + lo + 1);
    if (held && slot >= 0 && slot < static_cast<int64_t>(a.t.max_pages) * a.t.page_size) {
      const int pg = page_of(a.t, lo, static_cast<int>(slot));
      page = static_cast<int64_t>(pg) * a.t.n_heads + h;
      if (pg >= 0) to = page * a.t.page_size + page_offset(a.t, static_cast<int>(slot));
    } else if (r < __ldg(a.cu + a.t.n_seqs)) {  // (rows behind the last sequence are none of its tokens)
      report(a.t.status, OCTO_PAGED_BAD_LENGTH);
    }
    s_dst[t] = to;
    s_page[t] = page;
    s_src[t] = static_cast<int64_t>(h) * a.m.W * a.m.src_plane + r;
    s_srow[t] = static_cast<int64_t>(h) * a.m.src_plane + r;
    s_vsrc[t] = r * a.v_row + h * a.v_head;
  }
  __syncthreads();
  move_tile<256, TILE>(a.m, s_src, s_srow, s_vsrc, s_dst, s_page, nt);
}

// ---- eviction: which slots stay -----------------------------------------------
struct SelectArgs {
  const int32_t* seq_lens;
  const float* mass;
  int64_t mass_stride;
  int n_heads, cap, keep, sink, recent;
  int32_t* kept;
  float* new_mass;
  int32_t* status;
};

// Order of masses as unsigned numbers: larger first means larger here; NaN
// below every number, -0 as 0.
__device__ __forceinline__ uint32_t order_bits(float v) {
  if (!(v == v)) return 0u;
  const uint32_t u = __float_as_uint(v + 0.0f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// C blocks (a cluster) share a (sequence, head): its passes are bound by one
// SM's instructions, and few heads would leave the other SMs idle. A warp owns a contiguous run of slots, lanes along
// it. HELD: the slots' ordered bits are kept in shared memory; else every pass
// reads the masses again.
template <bool HELD, int C>
__global__ void __launch_bounds__(1024) paged_select_kernel(const __grid_constant__ SelectArgs a) {
  namespace cg = cooperative_groups;
  // eight copies of each bin, a lane uses copy lane mod 8: lanes of a warp that count one value (a fifth of the slots
  // may hold 0) would queue for its bin
  extern __shared__ uint32_t hist[];  // [8][kBins]; 4 words of stagger: the copies of a bin in different banks
  uint32_t* total = hist + 8 * kBins;            // [2][2048] this block's bins, of even and odd passes
  uint32_t* bits_of = total + 2 * 2048;          // HELD
  __shared__ uint32_t s_part[32], s_eq[32], s_mine[2];
  __shared__ uint32_t s_bin, s_rank;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank_in = C > 1 ? static_cast<int>(cg::this_cluster().block_rank()) : 0;
  auto all_sync = [] {
    if constexpr (C > 1)
      cg::this_cluster().sync();
    else
      __syncthreads();
  };
  auto of_block = [](uint32_t* p, int r) -> const uint32_t* {
    if constexpr (C > 1)
      return cg::this_cluster().map_shared_rank(p, r);
    else
      return p;
  };
  const int row = blockIdx.x / C, i = row / a.n_heads, h = row % a.n_heads;
  const int told = a.seq_lens[i];
  const int n = min(max(told, 0), a.cap);
  if (tid == 0 && h == 0 && rank_in == 0 && n != told) report(a.status, OCTO_PAGED_BAD_LENGTH);
  const float* mass = a.mass + static_cast<int64_t>(row) * a.mass_stride;
  int32_t* kept = a.kept + static_cast<int64_t>(row) * a.keep;
  float* out = a.new_mass ? a.new_mass + static_cast<int64_t>(row) * a.keep : nullptr;
  if (n <= a.keep) {
    for (int j = rank_in * 1024 + tid; j < a.keep; j += 1024 * C) {
      kept[j] = j < n ? j : -1;
      if (out) out[j] = j < n ? mass[j] : 0.0f;
    }
    return;
  }
  const int lo = a.sink, hi = n - a.recent;            // the middle: [lo, hi)
  const uint32_t want = a.keep - a.sink - a.recent;    // of it stay (0 .. hi - lo - 1)
  const int run = (n + 1024 * C - 1) / (1024 * C) * 32;  // slots of a warp
  const int b0 = rank_in * 32 * run;                   // first slot of the block
  const int j0 = min(n, b0 + warp * run), j1 = min(n, j0 + run);
  if constexpr (HELD) {
#pragma unroll 4
    for (int j = b0 + tid; j < min(n, b0 + 32 * run); j += 1024) bits_of[j - b0] = order_bits(mass[j]);
    __syncthreads();
  }
  // f(slot, ordered bits) for this thread's slots, in order (warp-uniform calls)
  auto each = [&](auto&& f) {
#pragma unroll 4
    for (int j = j0 + lane; j - lane < j1; j += 32) f(j, j < j1 ? (HELD ? bits_of[j - b0] : order_bits(mass[j])) : 0u);
  };
  // the want-th largest: its bits, digit by digit, and how many of its equals stay
  uint32_t prefix = 0, rank = want;
  if (want > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int sh = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      const uint32_t above = pass == 0 ? 0u : 0xffffffffu << (sh + bits);
      for (int b = tid; b < kBins * 8; b += 1024) hist[b] = 0u;
      __syncthreads();
      each([&](int j, uint32_t u) {
        if (j >= lo && j < min(hi, j1) && (u & above) == prefix)
          atomicAdd(&hist[(lane & 7) * kBins + ((u >> sh) & ((1u << bits) - 1u))], 1u);
      });
      __syncthreads();
      // (the other buffer may still be read by the cluster's blocks: they are at most a pass behind)
      uint32_t* mine = total + (pass & 1) * 2048;
      for (int b = tid; b < 2048; b += 1024) {
        uint32_t x = 0;
#pragma unroll
        for (int c = 0; c < 8; ++c) x += hist[c * kBins + b];
        mine[b] = x;
      }
      all_sync();
      // the digit: bins from the top until they hold `rank`; thread t sums bins 2047 - 2t and 2046 - 2t
      uint32_t x = 0, y = 0;
#pragma unroll
      for (int r = 0; r < C; ++r) {
        const uint32_t* t = of_block(mine, r);
        x += t[2047 - 2 * tid];
        y += t[2046 - 2 * tid];
      }
      uint32_t sum = x + y;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += u;
      }
      if (lane == 31) s_part[warp] = sum;
      __syncthreads();
      if (warp == 0) {
        uint32_t w = s_part[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t u = __shfl_up_sync(0xffffffffu, w, o);
          if (lane >= o) w += u;
        }
        s_part[lane] = w;
      }
      __syncthreads();
      const uint32_t end = sum + (warp ? s_part[warp - 1] : 0u), begin = end - x - y;
      if (begin < rank && rank <= end) {  // one thread
        const bool second = rank > begin + x;
        s_bin = second ? 2046 - 2 * tid : 2047 - 2 * tid;
        s_rank = rank - begin - (second ? x : 0u);
      }
      __syncthreads();
      prefix |= s_bin << sh;
      rank = s_rank;
      __syncthreads();
    }
  }
  // count what each warp and block keeps, then write in order
  uint32_t sure = 0, eq = 0;
  each([&](int j, uint32_t u) {
    const bool in = j < j1, mid = j >= lo && j < hi;
    sure += in && (!mid || (want > 0 && u > prefix));
    eq += in && mid && want > 0 && u == prefix;
  });
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sure += __shfl_xor_sync(0xffffffffu, sure, o);
    eq += __shfl_xor_sync(0xffffffffu, eq, o);
  }
  if (lane == 0) {
    s_part[warp] = sure;
    s_eq[warp] = eq;
  }
  __syncthreads();
  if (tid == 0) {
    uint32_t x = 0, y = 0;
    for (int k = 0; k < 32; ++k) {
      x += s_part[k];
      y += s_eq[k];
    }
    s_mine[0] = x;
    s_mine[1] = y;
  }
  all_sync();
  uint32_t at = 0, ties = 0;  // kept and equal slots of the blocks and warps before
  for (int r = 0; r < rank_in; ++r) {
    const uint32_t* t = of_block(s_mine, r);
    at += t[0];
    ties += t[1];
  }
  for (int k = 0; k < warp; ++k) {
    at += s_part[k];
    ties += s_eq[k];
  }
  if constexpr (C > 1) all_sync();  // no block leaves while others read its counts
  at += min(ties, rank);
  each([&](int j, uint32_t u) {
    const bool in = j < j1, mid = j >= lo && j < hi;
    const bool same = in && mid && want > 0 && u == prefix;
    const uint32_t eqs = __ballot_sync(0xffffffffu, same);
    const uint32_t below = (1u << lane) - 1u;
    const bool stays = in && (!mid || (want > 0 && u > prefix) || (same && ties + __popc(eqs & below) < rank));
    const uint32_t all = __ballot_sync(0xffffffffu, stays);
    if (stays) {
      const uint32_t o = at + __popc(all & below);
      kept[o] = j;
      if (out) out[o] = mass[j];
    }
    at += __popc(all);
    ties += __popc(eqs);
  });
}

template <bool HELD, int C>
static cudaError_t launch_select(const SelectArgs& s, int64_t rows, cudaStream_t st) {
  static LaunchCache cache;
  constexpr size_t fixed = (kBins * 8 + 2 * 2048) * sizeof(uint32_t);
  int resident = 0;
  cudaError_t e = launch_setup(paged_select_kernel<HELD, C>, cache, 1024, fixed + (HELD ? kHeld * sizeof(uint32_t) : 0), resident);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(rows) * C);
  cfg.blockDim = dim3(1024);
  cfg.dynamicSmemBytes = fixed + (HELD ? std::min<size_t>(kHeld, s.cap / C + 1024) * sizeof(uint32_t) : 0);
  cfg.stream = st;
  cudaLaunchAttribute cluster{};
  cluster.id = cudaLaunchAttributeClusterDimension;
  cluster.val.clusterDim.x = C;
  cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
  cfg.attrs = &cluster;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_select_kernel<HELD, C>, s);
}

// ---- eviction: the tokens that stay move --------------------------------------
struct GatherArgs {
  Table src, dst;
  MoveArgs m;
  const int32_t* kept;
  int keep, cap;
  const int32_t* seq_lens;
  int32_t* new_lens;  // may be seq_lens: written here, when the choice has read all lengths
};

template <int TILE>
__global__ void __launch_bounds__(256) paged_gather_kernel(const __grid_constant__ GatherArgs a) {
  __shared__ int64_t s_src[TILE], s_srow[TILE], s_vsrc[TILE], s_dst[TILE], s_page[TILE];
  const int i = blockIdx.y / a.src.n_heads, h = blockIdx.y % a.src.n_heads, P = a.src.page_size;
  const int k0 = blockIdx.x * TILE, nt = min(TILE, a.keep - k0);
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0)
    // (a plain load: new_lens may be seq_lens, and the read-only path is for memory that the kernel does not write)
    a.new_lens[i] = min(min(max(*const_cast<const volatile int32_t*>(a.seq_lens + i), 0), a.cap), a.keep);
  for (int t = threadIdx.x; t < nt; t += 256) {
    const int slot = __ldg(a.kept + static_cast<int64_t>(blockIdx.y) * a.keep + k0 + t);
    int64_t from = kNone, to = kNone, row = kNone, page = 0;
    if (slot >= 0) {
      const int pg = page_of(a.src, i, slot), z = page_of(a.dst, i, k0 + t);
      if (pg >= 0) {
        row = (static_cast<int64_t>(pg) * a.src.n_heads + h) * P + page_offset(a.src, slot);
        from = (static_cast<int64_t>(pg) * a.src.n_heads + h) * a.m.W * P + page_offset(a.src, slot);
      }
      page = static_cast<int64_t>(z) * a.src.n_heads + h;
      if (z >= 0) to = page * P + page_offset(a.dst, k0 + t);
    }
    s_src[t] = from;
    s_srow[t] = row;
    s_vsrc[t] = row < 0 ? kNone : row * a.m.pieces;
    s_dst[t] = to;
    s_page[t] = page;
  }
  __syncthreads();
  move_tile<256, TILE>(a.m, s_src, s_srow, s_vsrc, s_dst, s_page, nt);
}

}  // namespace paged
}  // namespace octo

extern "C" int octo_paged_write(const octo_layout* L, const octo_pages* pages, const octo_page_table* table,
                                const uint32_t* packed, const float* gamma, int64_t staged_cap, const void* V,
                                int64_t v_row_stride, int64_t v_head_stride, int64_t n_rows, const int32_t* starts,
                                const int32_t* cu, octo_stream_t stream) {
  using namespace octo::paged;
  int c = check_layout(L);
  if (c != OCTO_OK) return c;
  if ((c = check_pages(pages)) != OCTO_OK) return c;
  if ((c = check_table(table, pages->page_size)) != OCTO_OK) return c;
  if (n_rows < 0 || staged_cap < n_rows || v_row_stride < 0 || v_head_stride < 0) return OCTO_EINVAL;
  if (n_rows > INT32_MAX) return OCTO_EUNSUPPORTED;
  if (pages->n_heads > 65535) return OCTO_EUNSUPPORTED;  // grid.y limit
  if (n_rows == 0 || table->n_seqs == 0) return OCTO_OK;
  if ((V == nullptr) != (pages->V == nullptr)) return OCTO_EINVAL;
  if (!packed || !gamma || !starts || !cu) return OCTO_EINVAL;
  if (reinterpret_cast<uintptr_t>(V) % 16 != 0 || (V && (v_row_stride % 8 != 0 || v_head_stride % 8 != 0)))
    return OCTO_EINVAL;
  WriteArgs a{};
  a.t = make_table(pages, table);
  a.m = MoveArgs{packed,          gamma,        static_cast<const uint4*>(V), staged_cap, pages->packed,
                 pages->gamma,    static_cast<uint4*>(pages->V), L->words,    pages->page_size, L->d / 8};
  a.starts = starts;
  a.cu = cu;
  a.n_rows = n_rows;
  a.v_row = v_row_stride / 8;
  a.v_head = v_head_stride / 8;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  constexpr int TILE = 32;
  paged_write_kernel<TILE><<<dim3(static_cast<unsigned>((n_rows + TILE - 1) / TILE), pages->n_heads), 256, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? OCTO_OK : OCTO_ECUDA;
}

extern "C" int octo_paged_evict(const octo_layout* L, const octo_pages* src, const octo_page_table* src_table,
                                const int32_t* seq_lens, const float* mass, int64_t mass_stride, int32_t keep,
                                int32_t sink, int32_t recent, const octo_pages* dst, const octo_page_table* dst_table,
                                int32_t* kept, int32_t* new_lens, float* new_mass, octo_stream_t stream) {
  using namespace octo::paged;
  int c = check_layout(L);
  if (c != OCTO_OK) return c;
  if ((c = check_pages(src)) != OCTO_OK || (c = check_pages(dst)) != OCTO_OK) return c;
  if (src->n_heads != dst->n_heads || src->page_size != dst->page_size || (src->V == nullptr) != (dst->V == nullptr))
    return OCTO_EINVAL;
  if ((c = check_table(src_table, src->page_size)) != OCTO_OK || (c = check_table(dst_table, dst->page_size)) != OCTO_OK)
    return c;
  if (src_table->n_seqs != dst_table->n_seqs || keep < 1 || sink < 0 || recent < 0 || mass_stride < 0 ||
      static_cast<int64_t>(sink) + recent > keep)
    return OCTO_EINVAL;
  if (static_cast<int64_t>(dst_table->max_pages) * dst->page_size < keep) return OCTO_EINVAL;
  const int64_t rows = static_cast<int64_t>(src_table->n_seqs) * src->n_heads;
  if (rows > 65535) return OCTO_EUNSUPPORTED;  // grid.y limit
  if (rows == 0) return OCTO_OK;
  if (!seq_lens || !mass || !kept || !new_lens) return OCTO_EINVAL;
  const uintptr_t l0 = reinterpret_cast<uintptr_t>(seq_lens), n0 = reinterpret_cast<uintptr_t>(new_lens);
  const uintptr_t lens_bytes = static_cast<uintptr_t>(src_table->n_seqs) * 4;
  if (l0 != n0 && l0 < n0 + lens_bytes && n0 < l0 + lens_bytes) return OCTO_EINVAL;  // in place, or apart
  if (new_mass) {  // the choice writes it while it reads mass
    const uintptr_t m0 = reinterpret_cast<uintptr_t>(mass), o0 = reinterpret_cast<uintptr_t>(new_mass);
    if (o0 < m0 + static_cast<uintptr_t>(rows) * mass_stride * 4 && m0 < o0 + static_cast<uintptr_t>(rows) * keep * 4)
      return OCTO_EINVAL;
  }
  SelectArgs s{};
  s.seq_lens = seq_lens;
  s.mass = mass;
  s.mass_stride = mass_stride;
  s.n_heads = src->n_heads;
  s.cap = static_cast<int>(std::min<int64_t>(static_cast<int64_t>(src_table->max_pages) * src->page_size, mass_stride));
  s.keep = keep;
  s.sink = sink;
  s.recent = recent;
  s.kept = kept;
  s.new_mass = new_mass;
  s.status = src->status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // One block or a cluster of four per (sequence, head). Four share the slots but meet eight times, and every block fills
  // an SM: they pay for long rows, and only while all clusters run at once. One / four, both launches of a call in us:
  // 32 rows of 4096 slots 13.0 / 21.3, of 16384 19.9 / 23.5, of 32768 29.2 / 25.5; 256 rows of 32768 54.9 / 166. Beyond
  // what one block can hold (34976 slots) four hold them, and beyond 139904 the masses are read in every pass.
  const bool four = s.cap > kHeld - 1024 || (s.cap > 24576 && rows <= 32);
  if ((!four ? launch_select<true, 1>(s, rows, st)
       : s.cap <= 4 * (kHeld - 1024) ? launch_select<true, 4>(s, rows, st) : launch_select<false, 4>(s, rows, st)) != cudaSuccess)
    return OCTO_ECUDA;
  GatherArgs g{};
  g.src = make_table(src, src_table);
  g.dst = make_table(dst, dst_table);
  g.m = MoveArgs{src->packed, src->gamma, static_cast<const uint4*>(src->V), src->page_size, dst->packed,
                 dst->gamma,  static_cast<uint4*>(dst->V), L->words, src->page_size, L->d / 8};
  g.kept = kept;
  g.keep = keep;
  g.cap = s.cap;
  g.seq_lens = seq_lens;
  g.new_lens = new_lens;
  constexpr int TILE = 128;
  paged_gather_kernel<TILE><<<dim3((keep + TILE - 1) / TILE, static_cast<unsigned>(rows)), 256, 0, st>>>(g);
  return cudaGetLastError() == cudaSuccess ? OCTO_OK : OCTO_ECUDA;
}
