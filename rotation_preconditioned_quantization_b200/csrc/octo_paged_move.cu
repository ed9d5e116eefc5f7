// Moving tokens of the paged compressed cache: new tokens into pages, and the
// tokens that an eviction keeps into fresh pages.
//
// Both move, per (token, head), W code words (a plane each), a norm and a row
// of V; bound by memory. A block takes a tile of tokens of one head, looks up
// their places once, then copies plane by plane (lanes along tokens, so that
// a page's part of a plane is one contiguous access) and V in 16-byte pieces.
//
// Which tokens an eviction keeps: per (sequence, head) a block finds the
// rank-th largest mass of the middle slots by three histogram passes over the
// ordered bits (11 + 11 + 10), then counts and writes the kept slots warp by
// warp in slot order, so the result does not depend on timing.

#include <algorithm>

#include "octo_paged.cuh"

namespace octo {
namespace paged {

constexpr int64_t kNone = -1;

// Copies nt tokens of head h. s_src: token's offset in the source's plane 0
// and s_srow its row in the source gamma (kNone: a token without a source,
// written as zeros); s_dst: place in the destination pool as (page * heads +
// head) * page_size + offset (kNone: dropped).
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
                                          const int64_t* s_vsrc, const int64_t* s_dst, int nt) {
  const int P = a.page_size;
#pragma unroll 4
  for (int k = threadIdx.x; k < a.W * TILE; k += THREADS) {
    const int w = k / TILE, t = k % TILE;
    if (t >= nt) continue;
    const int64_t to = s_dst[t], from = s_src[t];
    if (to < 0) continue;
    const int64_t page = to / P;
    a.packed[page * a.W * P + static_cast<int64_t>(w) * P + (to - page * P)] =
        from < 0 ? 0u : a.src_packed[from + w * a.src_plane];
  }
  for (int t = threadIdx.x; t < nt; t += THREADS)
    if (s_dst[t] >= 0) a.gamma[s_dst[t]] = s_srow[t] < 0 ? 0.0f : a.src_gamma[s_srow[t]];
  if (a.V) {
#pragma unroll 4
    for (int k = threadIdx.x; k < nt * a.pieces; k += THREADS) {
      const int t = k / a.pieces, p = k - t * a.pieces;
      const int64_t to = s_dst[t], from = s_vsrc[t];
      if (to < 0) continue;
      a.V[to * a.pieces + p] = from < 0 ? make_uint4(0u, 0u, 0u, 0u) : __ldg(a.src_V + from + p);
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
  __shared__ int64_t s_src[TILE], s_vsrc[TILE], s_dst[TILE];
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
    int64_t to = kNone;
    const bool held = r >= __ldg(a.cu + lo) && r < __ldg(a.cu + lo + 1);
    if (held && slot >= 0 && slot < static_cast<int64_t>(a.t.max_pages) * a.t.page_size) {
      const int pg = page_of(a.t, lo, static_cast<int>(slot));
      if (pg >= 0) to = (static_cast<int64_t>(pg) * a.t.n_heads + h) * a.t.page_size + page_offset(a.t, static_cast<int>(slot));
    } else {
      report(a.t.status, OCTO_PAGED_BAD_LENGTH);
    }
    s_dst[t] = to;
    s_src[t] = static_cast<int64_t>(h) * a.m.W * a.m.src_plane + r;
    s_vsrc[t] = r * a.v_row + h * a.v_head;
  }
  __syncthreads();
  // gamma rows of the staging cache: head h, row r
  __shared__ int64_t s_srow[TILE];
  for (int t = threadIdx.x; t < nt; t += 256) s_srow[t] = static_cast<int64_t>(h) * a.m.src_plane + r0 + t;
  __syncthreads();
  move_tile<256, TILE>(a.m, s_src, s_srow, s_vsrc, s_dst, nt);
}

// ---- eviction: which slots stay -----------------------------------------------
struct SelectArgs {
  const int32_t* seq_lens;
  const float* mass;
  int64_t mass_stride;
  int n_heads, cap, keep, sink, recent;
  int32_t* kept;
  int32_t* new_lens;
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

__global__ void __launch_bounds__(1024) paged_select_kernel(const __grid_constant__ SelectArgs a) {
  __shared__ uint32_t hist[2048];
  __shared__ uint32_t s_part[32], s_eq[32];
  __shared__ uint32_t s_bin, s_rank;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int i = blockIdx.x / a.n_heads, h = blockIdx.x % a.n_heads;
  const int told = a.seq_lens[i];
  const int n = min(max(told, 0), a.cap);
  if (tid == 0 && h == 0) {
    a.new_lens[i] = min(n, a.keep);
    if (n != told) report(a.status, OCTO_PAGED_BAD_LENGTH);
  }
  const float* mass = a.mass + static_cast<int64_t>(blockIdx.x) * a.mass_stride;
  int32_t* kept = a.kept + static_cast<int64_t>(blockIdx.x) * a.keep;
  float* out = a.new_mass ? a.new_mass + static_cast<int64_t>(blockIdx.x) * a.keep : nullptr;
  if (n <= a.keep) {
    for (int j = tid; j < a.keep; j += 1024) {
      kept[j] = j < n ? j : -1;
      if (out) out[j] = j < n ? mass[j] : 0.0f;
    }
    return;
  }
  const int lo = a.sink, hi = n - a.recent;            // the middle: [lo, hi)
  const uint32_t want = a.keep - a.sink - a.recent;    // of it stay (0 .. hi - lo - 1)
  // the want-th largest: its bits, digit by digit, and how many of its equals stay
  uint32_t prefix = 0, rank = want;
  if (want > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int sh = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      const uint32_t above = pass == 0 ? 0u : 0xffffffffu << (sh + bits);
      for (int b = tid; b < 2048; b += 1024) hist[b] = 0u;
      __syncthreads();
#pragma unroll 4
      for (int j = lo + tid; j < hi; j += 1024) {
        const uint32_t u = order_bits(mass[j]);
        if ((u & above) == prefix) atomicAdd(&hist[(u >> sh) & ((1u << bits) - 1u)], 1u);
      }
      __syncthreads();
      // the digit: bins from the top until they hold `rank`; thread t sums bins 2047 - 2t and 2046 - 2t
      const uint32_t x = hist[2047 - 2 * tid], y = hist[2046 - 2 * tid];
      uint32_t run = x + y;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += v;
      }
      if (lane == 31) s_part[warp] = run;
      __syncthreads();
      if (warp == 0) {
        uint32_t v = s_part[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
          if (lane >= o) v += u;
        }
        s_part[lane] = v;
      }
      __syncthreads();
      const uint32_t end = run + (warp ? s_part[warp - 1] : 0u), begin = end - x - y;
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
  // warps take contiguous runs of slots; count what each keeps, then write in order
  const int run = (n + 1023) / 1024 * 32, j0 = min(n, warp * run), j1 = min(n, j0 + run);
  uint32_t sure = 0, eq = 0;
#pragma unroll 4
  for (int j = j0 + lane; j < j1; j += 32) {
    const bool mid = j >= lo && j < hi;
    const uint32_t u = order_bits(mass[j]);
    sure += !mid || (want > 0 && u > prefix);
    eq += mid && want > 0 && u == prefix;
  }
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
  uint32_t at = 0, ties = 0;  // kept and equal slots of the warps before
  for (int k = 0; k < warp; ++k) {
    at += s_part[k];
    ties += s_eq[k];
  }
  at += min(ties, rank);
  for (int jj = j0; jj < j1; jj += 32) {
    const int j = jj + lane;
    const bool in = j < j1, mid = j >= lo && j < hi;
    const float v = in ? mass[j] : 0.0f;
    const uint32_t u = order_bits(v);
    const bool same = in && mid && want > 0 && u == prefix;
    const uint32_t eqs = __ballot_sync(0xffffffffu, same);
    const uint32_t below = (1u << lane) - 1u;
    const bool stays = in && (!mid || (want > 0 && u > prefix) || (same && ties + __popc(eqs & below) < rank));
    const uint32_t all = __ballot_sync(0xffffffffu, stays);
    if (stays) {
      const uint32_t o = at + __popc(all & below);
      kept[o] = j;
      if (out) out[o] = v;
    }
    at += __popc(all);
    ties += __popc(eqs);
  }
}

// ---- eviction: the tokens that stay move --------------------------------------
struct GatherArgs {
  Table src, dst;
  MoveArgs m;
  const int32_t* kept;
  int keep;
};

template <int TILE>
__global__ void __launch_bounds__(256) paged_gather_kernel(const __grid_constant__ GatherArgs a) {
  __shared__ int64_t s_src[TILE], s_srow[TILE], s_vsrc[TILE], s_dst[TILE];
  const int i = blockIdx.y / a.src.n_heads, h = blockIdx.y % a.src.n_heads, P = a.src.page_size;
  const int k0 = blockIdx.x * TILE, nt = min(TILE, a.keep - k0);
  for (int t = threadIdx.x; t < nt; t += 256) {
    const int slot = __ldg(a.kept + static_cast<int64_t>(blockIdx.y) * a.keep + k0 + t);
    int64_t from = kNone, to = kNone, row = kNone;
    if (slot >= 0) {
      const int pg = page_of(a.src, i, slot), z = page_of(a.dst, i, k0 + t);
      if (pg >= 0) {
        row = (static_cast<int64_t>(pg) * a.src.n_heads + h) * P + page_offset(a.src, slot);
        from = (static_cast<int64_t>(pg) * a.src.n_heads + h) * a.m.W * P + page_offset(a.src, slot);
      }
      if (z >= 0) to = (static_cast<int64_t>(z) * a.src.n_heads + h) * P + page_offset(a.dst, k0 + t);
    }
    s_src[t] = from;
    s_srow[t] = row;
    s_vsrc[t] = row < 0 ? kNone : row * a.m.pieces;
    s_dst[t] = to;
  }
  __syncthreads();
  move_tile<256, TILE>(a.m, s_src, s_srow, s_vsrc, s_dst, nt);
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
  if ((V == nullptr) != (pages->V == nullptr)) return OCTO_EINVAL;
  if (n_rows == 0 || table->n_seqs == 0) return OCTO_OK;
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
  s.new_lens = new_lens;
  s.new_mass = new_mass;
  s.status = src->status;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  paged_select_kernel<<<static_cast<unsigned>(rows), 1024, 0, st>>>(s);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return OCTO_ECUDA;
  GatherArgs g{};
  g.src = make_table(src, src_table);
  g.dst = make_table(dst, dst_table);
  g.m = MoveArgs{src->packed, src->gamma, static_cast<const uint4*>(src->V), src->page_size, dst->packed,
                 dst->gamma,  static_cast<uint4*>(dst->V), L->words, src->page_size, L->d / 8};
  g.kept = kept;
  g.keep = keep;
  constexpr int TILE = 64;
  paged_gather_kernel<TILE><<<dim3((keep + TILE - 1) / TILE, static_cast<unsigned>(rows)), 256, 0, st>>>(g);
  return cudaGetLastError() == cudaSuccess ? OCTO_OK : OCTO_ECUDA;
}
