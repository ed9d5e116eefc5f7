// Attention of a chunk of new tokens over the paged compressed cache.
//
// Per sequence and KV head the rows are the chunk's (token, query head of the
// group) pairs; row r's logits over slot n are
//   s_rn = scale * gamma_n * <R q_r, u_hat_n>,
// and its output softmax(s_r) V, by one pass over the slots with a running
// reference m_r and sum l_r (base 2): o_r accumulates 2^(s - m) v, and is
// rescaled when a logit passes the reference by more than 16 (base 2).
//
// Matrix work on tcgen05: S = Q K^T with 128-row query tiles (fp16, scaled by
// a power of two per row so that every |q| <= 1) and 128-slot key tiles, whose
// rows are the decoded unit directions in fp16 (gamma is applied to S in
// fp32, so a key's norm costs no precision); O += P V with P in bf16 in
// tensor memory, in place of its S, and V (bf16) as TMA brings it. A CTA
// holds two query tiles (256 rows), so each key tile is decoded once per 256
// rows. Tensor memory: S0, S1 (128 columns each), O0, O1 (D columns each).
//
// Warps (16): 0-3 and 4-7 the softmax of query tile 0 and 1 (a thread owns a
// row: no shuffles), and before it the rotation of their queries; 8-11 decode
// key tiles, a thread per slot, one ahead of the products; 12 issues the
// products; 13 copies V.
//
// Schedule: the (sequence, head, 256-row tile) items' key tiles form one
// list, cut into equal contiguous pieces, one per CTA, whatever the lengths.
// An item that several CTAs share leaves fp32 partials (m, l, O) in the
// workspace: at most the first and the last item of a CTA's piece, so two
// slots per CTA; a second kernel joins them.

#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>
#include <cstring>

#include "octo_paged.cuh"

namespace octo {
namespace paged {

constexpr int kRows = 256;   // query rows of an item
constexpr int kKeys = 128;   // slots of a key tile
constexpr int kPanel = 128 * 128;  // bytes of a 128-row panel of 64 halves
constexpr float kRaise = 16.0f;    // log2 excess over the reference that raises it: weights stay below 2^16

struct AttnArgs {
  Table t;
  const uint32_t* packed;
  const float* gamma;
  const float* dir_c;
  const float* rho_c;
  const float* signs;
  int64_t table_heads;
  const int32_t* seq_lens;
  const int32_t* cu;
  const void* q;
  int64_t q_row, q_head, n_rows;
  int q_bf16, Hq, g, causal, box;  // box: V rows per copy
  float scale;
  void* out;
  int out_bf16;
  float* lse;
  float* part_o;   // [slots][slot_rows][D]
  float2* part_ml; // [slots][slot_rows]
  int slot_rows;
};

// An item's place: sequence, head, 256-row tile, and its key tiles.
__device__ __forceinline__ int row_tiles(const Seq& s, int g) { return (s.fresh * g + kRows - 1) / kRows; }
// slots that the last row of row tile m sees
__device__ __forceinline__ int item_limit(const Seq& s, int g, int causal, int m) {
  if (!causal) return s.len;
  const int last = (min(s.fresh * g, (m + 1) * kRows) - 1) / g;
  return max(0, s.len - s.fresh + last + 1);
}
__device__ __forceinline__ int item_tiles(const Seq& s, int g, int causal, int m) {
  return max(1, (item_limit(s, g, causal, m) + kKeys - 1) / kKeys);
}
// key tiles of one head of a sequence
__device__ __forceinline__ int64_t head_tiles(const Seq& s, int g, int causal) {
  const int mt = row_tiles(s, g);
  if (!causal) return static_cast<int64_t>(mt) * max(1, (s.len + kKeys - 1) / kKeys);
  int64_t n = 0;
  for (int m = 0; m < mt; ++m) n += item_tiles(s, g, causal, m);
  return n;
}

// Where a CTA's piece of the list starts (warp-wide, all lanes the same).
struct Place {
  int64_t count;  // key tiles of the piece
  int i, h, m, tile;
};
__device__ __forceinline__ int64_t warp_scan(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
__device__ int64_t total_tiles(const AttnArgs& a, int lane, bool tell) {
  int64_t n = 0;
  for (int i = lane; i < a.t.n_seqs; i += 32)
    n += head_tiles(seq_of(a.t, a.seq_lens, a.cu, a.n_rows, i, tell), a.g, a.causal) * a.t.n_heads;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
  return n;
}
__device__ Place find_place(const AttnArgs& a, int lane, int64_t total) {
  // no more pieces than tiles: an empty piece would leave no partial where the join looks for one
  const int64_t ctas = min(static_cast<int64_t>(gridDim.x), total);
  Place p{0, 0, 0, 0, 0};
  if (blockIdx.x >= ctas) return p;
  const int64_t at = blockIdx.x * total / ctas;
  p.count = (blockIdx.x + 1) * total / ctas - at;
  int64_t before = 0;
  for (int base = 0; base < a.t.n_seqs; base += 32) {
    const int i = base + lane;
    Seq s{0, 0, 0};
    if (i < a.t.n_seqs) s = seq_of(a.t, a.seq_lens, a.cu, a.n_rows, i);
    const int64_t th = i < a.t.n_seqs ? head_tiles(s, a.g, a.causal) : 0;
    const int64_t n = th * a.t.n_heads;
    const int64_t end = before + warp_scan(n, lane);
    const uint32_t past = __ballot_sync(0xffffffffu, end > at);
    if (past) {
      const int who = __ffs(past) - 1;
      if (lane == who) {
        int64_t rest = at - (end - n);
        p.i = i;
        p.h = static_cast<int>(rest / th);
        rest -= p.h * th;
        int m = 0, k;
        while (rest >= (k = item_tiles(s, a.g, a.causal, m))) {
          rest -= k;
          ++m;
        }
        p.m = m;
        p.tile = static_cast<int>(rest);
      }
      p.i = __shfl_sync(0xffffffffu, p.i, who);
      p.h = __shfl_sync(0xffffffffu, p.h, who);
      p.m = __shfl_sync(0xffffffffu, p.m, who);
      p.tile = __shfl_sync(0xffffffffu, p.tile, who);
      return p;
    }
    before = __shfl_sync(0xffffffffu, end, 31);
  }
  p.count = 0;
  return p;
}

// Walks a piece item by item: tiles [t0, t1) of item (i, h, m), which has
// `tiles` in all and whose last row sees `limit` slots.
struct Walk {
  const AttnArgs& a;
  int64_t left;
  int i, h, m, t0, t1, tiles, limit;
  Seq s;
  __device__ Walk(const AttnArgs& a_, const Place& p) : a(a_), left(p.count), i(p.i), h(p.h), m(p.m), t0(p.tile) {
    if (left > 0) {
      s = seq_of(a.t, a.seq_lens, a.cu, a.n_rows, i);
      open();
    }
  }
  __device__ void open() {
    limit = item_limit(s, a.g, a.causal, m);
    tiles = item_tiles(s, a.g, a.causal, m);
    t1 = static_cast<int>(min(static_cast<int64_t>(tiles), t0 + left));
  }
  __device__ bool on() const { return left > 0; }
  // tiles that hold slots: none for an item whose rows see nothing
  __device__ int work() const { return limit > 0 ? t1 - t0 : 0; }
  __device__ int rows() const { return min(kRows, s.fresh * a.g - m * kRows); }
  __device__ void next() {
    left -= t1 - t0;
    if (left <= 0) return;
    t0 = 0;
    if (++m >= row_tiles(s, a.g)) {
      m = 0;
      if (++h >= a.t.n_heads) {
        h = 0;
        do {
          ++i;
          s = seq_of(a.t, a.seq_lens, a.cu, a.n_rows, i);
        } while (s.fresh <= 0);
      }
    }
    open();
  }
};

template <int D, int B>
struct AttnCfg {
  using K = Code<D, B>;
  static constexpr int NP = D / 64;                    // 64-half panels of a row
  static constexpr int TILE = NP * kPanel;             // bytes of a 128 x D tile of halves
  // Table entries of 8 bytes {x, y | z, z} (fp16), replicated so that the
  // lanes of a half-warp meet few bank conflicts: every signed code for
  // b <= 3, the directions alone for b = 4 (8192 codes would fill 64 KB
  // without a replica), times the norm level from a second table.
  static constexpr bool SPLIT = B == 4;
  static constexpr int NE = SPLIT ? K::NDIR : 1 << K::C;
  static constexpr int REP = NE <= 128 ? 16 : 4;
  static constexpr int SH = 3 + (REP == 16 ? 4 : 2);   // log2 bytes of an entry with its replicas
  static constexpr int GS = 3;                         // gamma rows in flight
  static constexpr int Q = 0, KT = 2 * TILE, V = 4 * TILE, TAB = 6 * TILE, RHO = TAB + (NE << SH);
  static constexpr int GAM = RHO + (SPLIT ? 8 * 16 * 4 : 0), BARS = GAM + GS * kKeys * 4;
  static constexpr int PLACE = BARS + 144, TMEM = PLACE + 40, DIR = PLACE + 64, RHOF = DIR + 128, SMEM = RHOF + 32;
  static_assert(SMEM <= 232448, "shared memory of an SM");
  static constexpr int THREADS = 512;
};

// barriers
enum { kQF = 0, kSF = 2, kPR = 4, kKF = 6, kKE = 8, kVF = 10, kVE = 12, kVZ = 14, kEND = 16, kBars = 17 };

// ---- decode warps: key tiles ------------------------------------------------
template <int D, int B>
__device__ __forceinline__ bool decode_role(const AttnArgs& a, const Place& place, unsigned char* sm, uint32_t base,
                                            uint32_t bars) {
  using Cfg = AttnCfg<D, B>;
  using K = Code<D, B>;
  constexpr int W = K::W, T = K::T;
  const int n = threadIdx.x & 127, lane = threadIdx.x & 31;
  const uint32_t tab = base + Cfg::TAB + (lane & (Cfg::REP - 1)) * 8;
  const uint32_t rho = base + Cfg::RHO + (lane & 15) * 4;
  uint32_t w[W];
  float gm = 0.0f;
  // words and gamma of this thread's slot of a tile (0 behind the sequence)
  auto fetch = [&](const Walk& it, int tile) {
    const int slot = tile * kKeys + n;
#pragma unroll
    for (int k = 0; k < W; ++k) w[k] = 0u;
    gm = 0.0f;
    if (slot < it.s.len) {
      const int pg = max(0, page_of(a.t, it.i, slot));
      const int64_t row = static_cast<int64_t>(pg) * a.t.n_heads + it.h;
      const int off = slot % a.t.page_size;
      const uint32_t* p = a.packed + row * W * a.t.page_size + off;
#pragma unroll
      for (int k = 0; k < W; ++k) w[k] = __ldg(p + static_cast<int64_t>(k) * a.t.page_size);
      gm = __ldg(a.gamma + row * a.t.page_size + off);
    }
  };
  int c = 0;
  Walk it(a, place);
  while (it.on() && it.work() == 0) it.next();
  if (it.on()) fetch(it, it.t0);
  while (it.on()) {
    for (int tile = it.t0; tile < it.t1; ++tile, ++c) {
      const int st = c & 1;
      if (!bar_wait(bars + 8 * (kKE + st), ((c >> 1) & 1) ^ 1)) return false;
      reinterpret_cast<float*>(sm + Cfg::GAM)[(c % Cfg::GS) * kKeys + n] = gm;
      unsigned char* kt = sm + Cfg::KT + st * Cfg::TILE;
      // groups of 8 triplets: 24 halves, three 16-byte chunks of the row
#pragma unroll
      for (int g0 = 0; g0 < T; g0 += 8) {
        uint32_t o[12];
#pragma unroll
        for (int pr = 0; pr < 4; ++pr) {
          uint2 e[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int i = g0 + 2 * pr + u;
            e[u] = make_uint2(0u, 0u);
            if (i < T) {
              if constexpr (Cfg::SPLIT) {
                const uint32_t code = code_at<K::C, 0>(w, i);
                const uint32_t at = (code & (K::NDIR - 1)) << Cfg::SH;
                asm("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(e[u].x), "=r"(e[u].y) : "r"(tab + at));
                uint32_t r;
                asm("ld.shared.b32 %0, [%1];" : "=r"(r) : "r"(rho + (code >> K::DIR) * 64));
                const __half2 r2 = *reinterpret_cast<const __half2*>(&r);
                const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&e[u].x), r2);
                const __half2 z = __hmul2(*reinterpret_cast<const __half2*>(&e[u].y), r2);
                e[u].x = *reinterpret_cast<const uint32_t*>(&x);
                e[u].y = *reinterpret_cast<const uint32_t*>(&z);
              } else {
                asm("ld.shared.v2.b32 {%0, %1}, [%2];"
                    : "=r"(e[u].x), "=r"(e[u].y)
                    : "r"(tab + code_at<K::C, Cfg::SH>(w, i)));
              }
            }
          }
          o[3 * pr] = e[0].x;
          o[3 * pr + 1] = lolo(e[0].y, e[1].x);
          o[3 * pr + 2] = hilo(e[1].x, e[1].y);
        }
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          const int chunk = g0 / 8 * 3 + q;
          if (chunk < D / 8)
            *reinterpret_cast<uint4*>(kt + sw128(n, chunk, kPanel)) =
                make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        }
      }
      fence_async_shared();
      bar_arrive(bars + 8 * (kKF + st));
      // V rows behind the sequence's end hold whatever the page held: zero
      // them once the copy is in (0 * NaN would reach the output)
      const int valid = it.s.len - tile * kKeys;
      if (valid < kKeys) {
        if (!bar_wait(bars + 8 * (kVF + st), (c >> 1) & 1)) return false;
        unsigned char* vt = sm + Cfg::V + st * Cfg::TILE;
        if (n >= valid) {
#pragma unroll
          for (int q = 0; q < D / 8; ++q)
            *reinterpret_cast<uint4*>(vt + (q >> 3) * kPanel + n * 128 + (q & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_async_shared();
        bar_arrive(bars + 8 * (kVZ + st));
      }
      // next tile's words
      if (tile + 1 < it.t1) fetch(it, tile + 1);
    }
    do it.next();
    while (it.on() && it.work() == 0);
    if (it.on()) fetch(it, it.t0);
  }
  return true;
}

// ---- V copies ---------------------------------------------------------------
template <int D, int B>
__device__ __forceinline__ bool v_role(const AttnArgs& a, const Place& place, const CUtensorMap* map, uint32_t base,
                                       uint32_t bars, int& issued) {
  using Cfg = AttnCfg<D, B>;
  const int lane = threadIdx.x & 31;
  int c = 0;
  for (Walk it(a, place); it.on(); it.next()) {
    if (it.work() == 0) continue;
    for (int tile = it.t0; tile < it.t1; ++tile, ++c) {
      const int st = c & 1;
      if (!bar_wait(bars + 8 * (kVE + st), ((c >> 1) & 1) ^ 1)) return false;
      // boxes of a.box rows, each inside one page; none behind the last slot
      const int valid = min(kKeys, it.s.len - tile * kKeys);
      const int boxes = (valid + a.box - 1) / a.box;
      if (lane == 0) bar_expect(bars + 8 * (kVF + st), boxes * a.box * D * 2);
      __syncwarp();
      issued = c + 1;
      for (int b = lane; b < boxes; b += 32) {
        const int slot = tile * kKeys + b * a.box;
        const int pg = max(0, page_of(a.t, it.i, slot));
#pragma unroll
        for (int p = 0; p < Cfg::NP; ++p)
          tma_3d(base + Cfg::V + st * Cfg::TILE + p * kPanel + b * a.box * 128, map, p * 64, slot % a.t.page_size,
                 pg * a.t.n_heads + it.h, bars + 8 * (kVF + st));
      }
      __syncwarp();
    }
  }
  return true;
}

// ---- products ---------------------------------------------------------------
template <int D, int B>
__device__ __forceinline__ bool mma_role(const AttnArgs& a, const Place& place, uint32_t base, uint32_t bars,
                                         uint32_t tmem) {
  using Cfg = AttnCfg<D, B>;
  constexpr uint32_t kQK = instr_desc(128, kKeys, false, false), kPV = instr_desc(128, D, true, true);
  const bool one = (threadIdx.x & 31) == 0;
  auto qk = [&](int qt, int st) {
#pragma unroll
    for (int k = 0; k < D / 16; ++k) {
      const uint32_t off = (k >> 2) * kPanel + (k & 3) * 32;
      mma_ss(tmem + qt * kKeys, smem_desc(base + Cfg::Q + qt * Cfg::TILE + off, 16),
             smem_desc(base + Cfg::KT + st * Cfg::TILE + off, 16), kQK, k > 0);
    }
  };
  auto pv = [&](int qt, int st, bool acc) {
#pragma unroll
    for (int k = 0; k < kKeys / 16; ++k)
      mma_ts(tmem + 2 * kKeys + qt * D, tmem + qt * kKeys + k * 8,
             smem_desc(base + Cfg::V + st * Cfg::TILE + k * 16 * 128, kPanel), kPV, acc || k > 0);
  };
  // phases: query tile 0 takes part in every item, tile 1 in those of more than 128 rows; V tails are per stage
  int c = 0, nq = 0, np[2] = {0, 0};
  uint32_t nz = 0;
  for (Walk it(a, place); it.on(); it.next()) {
    const int nt = it.work();
    if (nt == 0) continue;
    const int tiles2 = it.rows() > 128 ? 2 : 1;
    for (int qt = 0; qt < tiles2; ++qt)
      if (!bar_wait(bars + 8 * (kQF + qt), (qt == 0 ? nq : np[1]) & 1)) return false;
    ++nq;
    if (tiles2 == 2) ++np[1];
    if (!bar_wait(bars + 8 * (kKF + (c & 1)), (c >> 1) & 1)) return false;
    tc_after();
    if (one) {
      for (int qt = 0; qt < tiles2; ++qt) {
        qk(qt, c & 1);
        tc_commit(bars + 8 * (kSF + qt));
      }
      tc_commit(bars + 8 * (kKE + (c & 1)));
    }
    __syncwarp();
    for (int j = 0; j < nt; ++j, ++c) {
      const int st = c & 1, sn = st ^ 1;
      const bool more = j + 1 < nt;
      if (more && !bar_wait(bars + 8 * (kKF + sn), ((c + 1) >> 1) & 1)) return false;
      if (!bar_wait(bars + 8 * (kVF + st), (c >> 1) & 1)) return false;
      if ((it.t0 + j + 1) * kKeys > it.s.len) {
        if (!bar_wait(bars + 8 * (kVZ + st), (nz >> st) & 1)) return false;
        nz ^= 1u << st;
      }
      for (int qt = 0; qt < tiles2; ++qt) {
        if (!bar_wait(bars + 8 * (kPR + qt), (qt == 0 ? c : np[0]) & 1)) return false;
        tc_after();
        if (one) {
          pv(qt, st, j > 0);
          if (more) qk(qt, sn);
          tc_commit(bars + 8 * (kSF + qt));  // S of the next tile, or O after the last
        }
        __syncwarp();
      }
      if (tiles2 == 2) ++np[0];
      if (one) {
        tc_commit(bars + 8 * (kVE + st));
        if (more) tc_commit(bars + 8 * (kKE + sn));
      }
      __syncwarp();
    }
  }
  return true;
}

// ---- softmax warps ----------------------------------------------------------
// Rotates the queries of this query tile into its shared tile (fp16, scaled
// by 2^-e per row), a warp per row at a time; lane r of the warp keeps row
// r's logit factor 2^e * |scale| * log2 e.
template <int D, int B>
__device__ __forceinline__ float rotate_queries(const AttnArgs& a, const Walk& it, unsigned char* qtile, int row0,
                                                int rows, int lane) {
  constexpr int E = D / 32;
  const float* sg = a.signs + (it.h % a.table_heads) * D + lane * E;
  float sign[E];
  const float pre = a.scale == 0.0f ? 0.0f : copysignf(1.0f / sqrtf(static_cast<float>(D)), a.scale);
#pragma unroll
  for (int e = 0; e < E; ++e) sign[e] = sg[e] * pre;
  float factor = 1.0f;
#pragma unroll 4
  for (int r = 0; r < rows; ++r) {
    const int rr = it.m * kRows + row0 + r;  // row of the item's (token, group head) list
    const int tok = rr / a.g, hq = it.h * a.g + rr % a.g;
    const int64_t off = (it.s.row0 + tok) * a.q_row + hq * a.q_head + lane * E;
    float v[E];
#pragma unroll
    for (int e = 0; e < E; ++e)
      v[e] = sign[e] * (a.q_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[off + e])
                                 : static_cast<const float*>(a.q)[off + e]);
    fwht_warp<E>(v, lane);
    float mx = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) mx = fmaxf(mx, fabsf(v[e]));
    mx = warp_max(mx);
    // 2^ex > mx (within 2^-125 .. 2^126, so that 2^-ex is a normal number)
    const int ex = min(max(static_cast<int>(__float_as_uint(mx) >> 23) - 126, -125), 126);
    const float down = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
    uint32_t h[E / 2];
#pragma unroll
    for (int e = 0; e < E; e += 2) h[e / 2] = half2_bits(v[e] * down, v[e + 1] * down);
    const int row = row0 % 128 + r;
    unsigned char* p = qtile + sw128(row, lane * E / 8, kPanel) + (lane * E % 8) * 2;
    if constexpr (E == 4)
      *reinterpret_cast<uint2*>(p) = make_uint2(h[0], h[1]);
    else
      *reinterpret_cast<uint32_t*>(p) = h[0];
    if (lane == r) {
      const float sc = a.scale == 0.0f ? 1.0f : fabsf(a.scale);
      factor = ldexpf(sc * 1.4426950408889634f, ex);
    }
  }
  return factor;
}

template <int D, int B>
__device__ __forceinline__ bool softmax_role(const AttnArgs& a, const Place& place, unsigned char* sm, uint32_t bars,
                                             uint32_t tmem, int qt) {
  using Cfg = AttnCfg<D, B>;
  const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
  const uint32_t S = tmem + lanes + qt * kKeys, O = tmem + lanes + 2 * kKeys + qt * D;
  int c = 0, ns = 0;
  for (Walk it(a, place); it.on(); it.next()) {
    const int nt = it.work(), rows = it.rows();
    const bool mine = qt == 0 || rows > 128;  // this query tile takes part in the item
    if (!mine) {
      c += nt;
      continue;
    }
    const int r0 = qt * 128 + warp * 32;                     // first row of the warp
    const int wr = min(32, max(0, rows - r0));               // its rows
    const int rr = it.m * kRows + r0 + lane;
    const bool there = lane < wr;
    int limit = 0;
    if (there) limit = a.causal ? max(0, it.s.len - it.s.fresh + rr / a.g + 1) : it.s.len;
    float ref = -INFINITY, sum = 0.0f;
    if (nt > 0) {
      const float factor = rotate_queries<D, B>(a, it, sm + Cfg::Q + qt * Cfg::TILE, r0, wr, lane);
      fence_async_shared();
      bar_arrive(bars + 8 * (kQF + qt));
      for (int j = 0; j < nt; ++j, ++c) {
        if (!bar_wait(bars + 8 * (kSF + qt), ns & 1)) return false;
        ++ns;
        tc_after();
        if (wr > 0) {  // a warp without rows leaves its part of P as it is: those rows go nowhere
          const float* gm = reinterpret_cast<const float*>(sm + Cfg::GAM) + (c % Cfg::GS) * kKeys;
          const int left = limit - (it.t0 + j) * kKeys;  // slots of the tile that the row sees
          const bool masked = __any_sync(0xffffffffu, there && left < kKeys);
          // two halves of 64 slots, so that a row's logits stay in registers from the maximum to the weights
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            uint32_t s[2][32];
            tmem_ld32(s[0], S + half * 64);
            tmem_ld32(s[1], S + half * 64 + 32);
            tc_wait_ld();
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
              for (int x = 0; x < 32; x += 4) {
                const float4 g4 = *reinterpret_cast<const float4*>(gm + half * 64 + k * 32 + x);
                const float2 lo = mul_f32x2(make_float2(__uint_as_float(s[k][x]), __uint_as_float(s[k][x + 1])),
                                            make_float2(g4.x, g4.y));
                const float2 hi = mul_f32x2(make_float2(__uint_as_float(s[k][x + 2]), __uint_as_float(s[k][x + 3])),
                                            make_float2(g4.z, g4.w));
                s[k][x] = __float_as_uint(lo.x);
                s[k][x + 1] = __float_as_uint(lo.y);
                s[k][x + 2] = __float_as_uint(hi.x);
                s[k][x + 3] = __float_as_uint(hi.y);
              }
            }
            if (masked) {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int x = 0; x < 32; ++x)
                  if (half * 64 + k * 32 + x >= left) s[k][x] = 0xff800000u;  // -inf
              }
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
              for (int x = 0; x < 32; x += 2)
                top[k] = fmaxf(top[k], fmaxf(__uint_as_float(s[k][x]), __uint_as_float(s[k][x + 1])));
            }
            const float high = fmaxf(top[0], top[1]) * factor;  // factor > 0
            const bool raise = high > ref + kRaise || (ref == -INFINITY && high > -INFINITY);
            if (__any_sync(0xffffffffu, raise)) {
              const float keep = raise ? ex2(ref - high) : 1.0f;
              if (raise) ref = high;
              sum *= keep;
              if (j > 0) {
#pragma unroll 1
                for (int k = 0; k < D; k += 16) {
                  uint32_t o[16];
                  tmem_ld16(o, O + k);
                  tc_wait_ld();
#pragma unroll
                  for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * keep);
                  tmem_st16(O + k, o);
                }
              }
              if (half == 1) {  // the first half's weights follow
#pragma unroll 1
                for (int k = 0; k < 32; k += 16) {
                  uint32_t o[16];
                  tmem_ld16(o, S + k);
                  tc_wait_ld();
#pragma unroll
                  for (int x = 0; x < 16; ++x) {
                    const __nv_bfloat162 b2 = __floats2bfloat162_rn(bf16_lo(o[x]) * keep, bf16_hi(o[x]) * keep);
                    o[x] = *reinterpret_cast<const uint32_t*>(&b2);
                  }
                  tmem_st16(S + k, o);
                }
              }
            }
            const float shift = ref == -INFINITY ? 0.0f : -ref;
            float2 part = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              uint32_t p[16];
#pragma unroll
              for (int x = 0; x < 32; x += 2) {
                const float2 y = fma_f32x2(make_float2(__uint_as_float(s[k][x]), __uint_as_float(s[k][x + 1])),
                                           make_float2(factor, factor), make_float2(shift, shift));
                const float2 e = make_float2(ex2(y.x), ex2(y.y));
                part = add_f32x2(part, e);
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(e.x, e.y);
                p[x / 2] = *reinterpret_cast<const uint32_t*>(&b2);
              }
              tmem_st16(S + half * 32 + k * 16, p);
            }
            sum += part.x + part.y;
          }
          tc_wait_st();
        }
        tc_before();
        bar_arrive(bars + 8 * (kPR + qt));
      }
      if (!bar_wait(bars + 8 * (kSF + qt), ns & 1)) return false;  // O is complete
      ++ns;
      tc_after();
    }
    // ---- results of the item (or of this piece of it)
    const bool whole = it.t0 == 0 && it.t1 == it.tiles;
    const int64_t slot = 2 * blockIdx.x + (it.t0 > 0 ? 0 : 1);
    const int64_t prow = slot * a.slot_rows + r0 + lane;
    const int tok = rr / a.g, hq = it.h * a.g + rr % a.g;
    const int64_t orow = static_cast<int64_t>(it.s.row0 + tok) * a.Hq + hq;
    if (wr > 0) {
      const float inv = whole ? (sum == 0.0f ? 0.0f : 1.0f / sum) : 1.0f;
      if (there) {
        if (!whole)
          a.part_ml[prow] = make_float2(ref, sum);
        else if (a.lse)
          a.lse[orow] = sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
      }
#pragma unroll 1
      for (int k = 0; k < D; k += 32) {
        uint32_t o[32];
        if (nt > 0) {
          tmem_ld32(o, O + k);
          tc_wait_ld();
        }
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          const float v = nt > 0 ? __uint_as_float(o[x]) * inv : 0.0f;
          o[x] = __float_as_uint(sum == 0.0f ? 0.0f : v);  // a row that saw nothing: its P rows were all 0 or never written
        }
        if (there) {
          if (whole && a.out_bf16) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + orow * D + k);
#pragma unroll
            for (int x = 0; x < 32; x += 8) {
              uint32_t w[4];
#pragma unroll
              for (int y = 0; y < 4; ++y) {
                const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(o[x + 2 * y]), __uint_as_float(o[x + 2 * y + 1]));
                w[y] = *reinterpret_cast<const uint32_t*>(&b2);
              }
              dst[x / 8] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
            float* dst = whole ? static_cast<float*>(a.out) + orow * D + k : a.part_o + prow * D + k;
#pragma unroll
            for (int x = 0; x < 32; x += 4)
              *reinterpret_cast<uint4*>(dst + x) = make_uint4(o[x], o[x + 1], o[x + 2], o[x + 3]);
          }
        }
      }
    }
    tc_before();
  }
  return true;
}

template <int D, int B>
__global__ void __launch_bounds__(512, 1) paged_attn_kernel(const __grid_constant__ AttnArgs a,
                                                            const __grid_constant__ CUtensorMap vmap) {
  using Cfg = AttnCfg<D, B>;
  using K = Code<D, B>;
  extern __shared__ __align__(1024) unsigned char sm[];
  const uint32_t base = s32(sm), bars = base + Cfg::BARS;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // everything in the dynamic block, so that it starts on a swizzle atom
  Place& s_place = *reinterpret_cast<Place*>(sm + Cfg::PLACE);
  uint32_t& s_tmem = *reinterpret_cast<uint32_t*>(sm + Cfg::TMEM);
  float* s_dir = reinterpret_cast<float*>(sm + Cfg::DIR);
  float* s_rho = reinterpret_cast<float*>(sm + Cfg::RHOF);
  if (tid < (1 << (B + 1))) s_dir[tid] = a.dir_c[tid];
  if (tid < K::NRHO) s_rho[tid] = a.rho_c[tid];
  if (warp == 15) {
    const int64_t total = total_tiles(a, lane, blockIdx.x == 0);
    const Place p = find_place(a, lane, total);
    if (lane == 0) s_place = p;
  }
  if (tid == 0) {
    for (int q = 0; q < 2; ++q) {
      bar_init(bars + 8 * (kQF + q), 128);
      bar_init(bars + 8 * (kSF + q), 1);
      bar_init(bars + 8 * (kPR + q), 128);
      bar_init(bars + 8 * (kKF + q), 128);
      bar_init(bars + 8 * (kKE + q), 1);
      bar_init(bars + 8 * (kVF + q), 1);
      bar_init(bars + 8 * (kVE + q), 1);
      bar_init(bars + 8 * (kVZ + q), 128);
    }
    bar_init(bars + 8 * kEND, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 12) tmem_alloc(s32(&s_tmem), 512);
  __syncthreads();
  const Place place = s_place;
  if (place.count > 0) {
    // decoded codes (b = 4: directions) in fp16, Cfg::REP copies of each
    for (int e = tid; e < Cfg::NE; e += Cfg::THREADS) {
      const float3 d = field_direction<B>(e & (K::NDIR - 1), s_dir);
      const float r = Cfg::SPLIT ? 1.0f : s_rho[e >> K::DIR];
      const uint2 v = make_uint2(half2_bits(d.x * r, d.y * r), half2_bits(d.z * r, d.z * r));
#pragma unroll
      for (int k = 0; k < Cfg::REP; ++k)
        *reinterpret_cast<uint2*>(sm + Cfg::TAB + (e << Cfg::SH) + k * 8) = v;
    }
    if (Cfg::SPLIT && tid < 128)
      *reinterpret_cast<uint32_t*>(sm + Cfg::RHO + tid * 4) = half2_bits(s_rho[tid >> 4], s_rho[tid >> 4]);
  }
  tc_before();
  __syncthreads();
  tc_after();
  const uint32_t tmem = s_tmem;
  bool ok = true;
  if (place.count > 0) {
    if (warp < 8) {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
      ok = softmax_role<D, B>(a, place, sm, bars, tmem, warp >> 2);
    } else if (warp < 12) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 112;");
      ok = decode_role<D, B>(a, place, sm, base, bars);
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
      if (warp == 12) {
        ok = mma_role<D, B>(a, place, base, bars, tmem);
        // products in flight end before tensor memory is given back
        if (!ok) {
          if (lane == 0) tc_commit(bars + 8 * kEND);
          __syncwarp();
          bar_wait(bars + 8 * kEND, 0);
        }
      } else if (warp == 13) {
        int issued = 0;
        ok = v_role<D, B>(a, place, &vmap, base, bars, issued);
        // copies in flight end before the CTA does
        for (int c = max(0, issued - 2); c < issued; ++c) bar_wait(bars + 8 * (kVF + (c & 1)), (c >> 1) & 1);
      }
    }
  }
  if (!ok && lane == 0) report(a.t.status, OCTO_PAGED_TIMEOUT);
  tc_before();
  __syncthreads();
  if (warp == 12) tmem_free(tmem, 512);
}

// ---- joining the pieces of shared items --------------------------------------
// One block per (256-row tile of any sequence, head, 32 rows of the tile); it
// finds the item's place in the list as the CTAs of the first kernel did.
template <int D>
__global__ void __launch_bounds__(256) paged_attn_join(const __grid_constant__ AttnArgs a, int grid_ctas) {
  const int h = blockIdx.y, tid = threadIdx.x, lane = tid & 31, r0 = blockIdx.z * 32;
  __shared__ int64_t s_at, s_total;
  __shared__ int s_i, s_m;
  if (tid < 32) {
    int64_t items = 0, before = 0;  // row tiles of the sequences so far; their key tiles
    int who = -1, mine = 0;
    int64_t at = 0;
    for (int base = 0; base < a.t.n_seqs; base += 32) {
      const int i = base + lane;
      Seq s{0, 0, 0};
      if (i < a.t.n_seqs) s = seq_of(a.t, a.seq_lens, a.cu, a.n_rows, i);
      const int64_t mt = row_tiles(s, a.g), n = mt ? head_tiles(s, a.g, a.causal) * a.t.n_heads : 0;
      const int64_t mend = items + warp_scan(mt, lane), nend = before + warp_scan(n, lane);
      const bool hit = static_cast<int64_t>(blockIdx.x) < mend && static_cast<int64_t>(blockIdx.x) >= mend - mt;
      if (hit) {
        who = i;
        mine = static_cast<int>(blockIdx.x - (mend - mt));
        at = nend - n + h * (n / a.t.n_heads);
        for (int k = 0; k < mine; ++k) at += item_tiles(s, a.g, a.causal, k);
        s_i = who;
        s_m = mine;
        s_at = at;
      }
      items = __shfl_sync(0xffffffffu, mend, 31);
      before = __shfl_sync(0xffffffffu, nend, 31);
    }
    if (!__any_sync(0xffffffffu, who >= 0) && lane == 0) s_i = -1;
    if (lane == 0) s_total = before;
  }
  __syncthreads();
  const int i = s_i, m = s_m;
  if (i < 0) return;
  const Seq s = seq_of(a.t, a.seq_lens, a.cu, a.n_rows, i);
  const int rows = min(kRows, s.fresh * a.g - m * kRows);
  if (r0 >= rows) return;
  const int64_t total = s_total;
  const int ctas = static_cast<int>(min(static_cast<int64_t>(grid_ctas), total));
  const int64_t at = s_at, end = at + item_tiles(s, a.g, a.causal, m);
  // the CTA that holds list position p is the last whose piece starts at or before it
  auto owner = [&](int64_t p) { return static_cast<int>(((p + 1) * ctas + total - 1) / total - 1); };
  const int c0 = owner(at), c1 = owner(end - 1);
  if (c0 == c1) return;  // written whole
  auto part_row = [&](int c, int r) {
    return (2 * static_cast<int64_t>(c) + (at < c * total / ctas ? 0 : 1)) * a.slot_rows + r;
  };
  constexpr int TPR = D / 4, RPB = 256 / TPR;  // threads per row, rows at a time
  for (int r = r0 + tid / TPR; r < min(rows, r0 + 32); r += RPB) {
    const int x = (tid % TPR) * 4;
    float ref = -INFINITY;
    for (int c = c0; c <= c1; ++c) ref = fmaxf(ref, a.part_ml[part_row(c, r)].x);
    const float base = ref == -INFINITY ? 0.0f : ref;
    float sum = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int c = c0; c <= c1; ++c) {
      const int64_t pr = part_row(c, r);
      const float2 ml = a.part_ml[pr];
      const float4 v = *reinterpret_cast<const float4*>(a.part_o + pr * D + x);
      const float w = ex2(ml.x - base);
      sum = fmaf(w, ml.y, sum);
      o.x = fmaf(w, v.x, o.x);
      o.y = fmaf(w, v.y, o.y);
      o.z = fmaf(w, v.z, o.z);
      o.w = fmaf(w, v.w, o.w);
    }
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    const int rr = m * kRows + r, hq = h * a.g + rr % a.g;
    const int64_t orow = static_cast<int64_t>(s.row0 + rr / a.g) * a.Hq + hq;
    if (a.out_bf16) {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv), hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + orow * D + x) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    } else {
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + orow * D + x) =
          make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    }
    if (a.lse && x == 0) a.lse[orow] = sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
  }
}

// ---- host -------------------------------------------------------------------
static int sm_count() {
  static std::atomic<int> known[kLaunchCacheDevices];
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  const bool cached = dev >= 0 && dev < kLaunchCacheDevices;
  if (cached && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
  if (cached) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

static bool encode_v_map(CUtensorMap* m, const octo_pages* p, int D, int box) {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  }();
  if (!fn) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(p->page_size),
                              static_cast<cuuint64_t>(p->n_pages) * p->n_heads};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(D) * 2, static_cast<cuuint64_t>(D) * 2 * p->page_size};
  const cuuint32_t bx[3] = {64, static_cast<cuuint32_t>(box), 1}, elem[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p->V, dims, strides, bx, elem, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// rows of a partial's slot: no item has more
static int slot_rows(int64_t n_rows, int g) {
  return static_cast<int>(std::min<int64_t>(kRows, (n_rows * g + 31) / 32 * 32));
}

template <int D, int B>
static cudaError_t launch_attn(const AttnArgs& a, const CUtensorMap& map, int ctas, cudaStream_t st) {
  static LaunchCache cache;
  int resident = 0;
  cudaError_t e = launch_setup(paged_attn_kernel<D, B>, cache, 512, AttnCfg<D, B>::SMEM, resident);
  if (e != cudaSuccess) return e;
  paged_attn_kernel<D, B><<<ctas, 512, AttnCfg<D, B>::SMEM, st>>>(a, map);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const int64_t rows = a.n_rows * a.g;
  const dim3 grid(static_cast<unsigned>(rows / kRows + a.t.n_seqs), a.t.n_heads,
                  static_cast<unsigned>((std::min<int64_t>(rows, kRows) + 31) / 32));
  paged_attn_join<D><<<grid, 256, 0, st>>>(a, ctas);
  return cudaGetLastError();
}

}  // namespace paged
}  // namespace octo

extern "C" size_t octo_paged_attn_workspace(const octo_layout* L, int64_t n_rows, int n_seqs, int Hq, int Hkv) {
  using namespace octo::paged;
  if (check_layout(L) != OCTO_OK || L->d > 128 || n_rows < 0 || n_seqs < 0 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0)
    return 0;
  const size_t rows = static_cast<size_t>(2) * sm_count() * slot_rows(n_rows, Hq / Hkv);
  return 256 + rows * (static_cast<size_t>(L->d) * sizeof(float) + sizeof(float2));
}

extern "C" int octo_paged_attn(const octo_layout* L, const octo_tables* tab, const octo_pages* pages,
                               const octo_page_table* table, const int32_t* seq_lens, const void* q, int q_dtype,
                               int64_t q_row_stride, int64_t q_head_stride, int64_t n_rows, int Hq,
                               const int32_t* cu_q, int causal, float scale, void* out, int out_dtype, float* lse,
                               void* workspace, size_t ws_bytes, octo_stream_t stream) {
  using namespace octo::paged;
  int c = check_layout(L);
  if (c != OCTO_OK) return c;
  if (L->d > 128) return OCTO_EUNSUPPORTED;
  if ((c = check_pages(pages)) != OCTO_OK) return c;
  if ((c = check_table(table, pages->page_size)) != OCTO_OK) return c;
  if (!tab || !tab->dir_c || !tab->rho_c || !tab->signs || tab->n_heads < 1 || !pages->V) return OCTO_EINVAL;
  if (q_dtype != OCTO_F32 && q_dtype != OCTO_BF16) return OCTO_EINVAL;
  if (out_dtype != OCTO_F32 && out_dtype != OCTO_BF16) return OCTO_EINVAL;
  if (n_rows < 0 || q_row_stride < 0 || q_head_stride < 0 || Hq < pages->n_heads || Hq % pages->n_heads != 0)
    return OCTO_EINVAL;
  if (!(scale - scale == 0.0f)) return OCTO_EINVAL;  // NaN or infinite
  const int g = Hq / pages->n_heads;
  if (g > 256) return OCTO_EUNSUPPORTED;
  if (n_rows * g > INT32_MAX - 1024) return OCTO_EUNSUPPORTED;
  if (pages->n_heads > 65535) return OCTO_EUNSUPPORTED;  // grid.y limit
  if (n_rows == 0 || table->n_seqs == 0) return OCTO_OK;
  if (!q || !out || !seq_lens || !cu_q) return OCTO_EINVAL;
  if (reinterpret_cast<uintptr_t>(out) % 16 != 0) return OCTO_EINVAL;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return OCTO_EINVAL;
  if (ws_bytes < octo_paged_attn_workspace(L, n_rows, table->n_seqs, Hq, pages->n_heads)) return OCTO_EWORKSPACE;
  AttnArgs a{};
  a.t = make_table(pages, table);
  a.packed = pages->packed;
  a.gamma = pages->gamma;
  a.dir_c = tab->dir_c;
  a.rho_c = tab->rho_c;
  a.signs = tab->signs;
  a.table_heads = tab->n_heads;
  a.seq_lens = seq_lens;
  a.cu = cu_q;
  a.q = q;
  a.q_row = q_row_stride;
  a.q_head = q_head_stride;
  a.n_rows = n_rows;
  a.q_bf16 = q_dtype == OCTO_BF16;
  a.Hq = Hq;
  a.g = g;
  a.causal = causal != 0;
  a.scale = scale;
  a.out = out;
  a.out_bf16 = out_dtype == OCTO_BF16;
  a.lse = lse;
  const int ctas = sm_count();
  a.slot_rows = slot_rows(n_rows, g);
  a.part_ml = reinterpret_cast<float2*>(workspace);
  const size_t ml = (static_cast<size_t>(2) * ctas * a.slot_rows * sizeof(float2) + 255) / 256 * 256;
  a.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + ml);
  // V comes in boxes that lie inside one page: the largest power of two (8-row swizzle groups) that divides it
  a.box = 16;
  while (a.box < kKeys && pages->page_size % (2 * a.box) == 0) a.box *= 2;
  CUtensorMap map;
  if (!encode_v_map(&map, pages, L->d, a.box)) return OCTO_ECUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (L->d == 64)
    e = L->b == 2 ? launch_attn<64, 2>(a, map, ctas, st) : L->b == 3 ? launch_attn<64, 3>(a, map, ctas, st) : launch_attn<64, 4>(a, map, ctas, st);
  else
    e = L->b == 2 ? launch_attn<128, 2>(a, map, ctas, st) : L->b == 3 ? launch_attn<128, 3>(a, map, ctas, st) : launch_attn<128, 4>(a, map, ctas, st);
  return e == cudaSuccess ? OCTO_OK : OCTO_ECUDA;
}
