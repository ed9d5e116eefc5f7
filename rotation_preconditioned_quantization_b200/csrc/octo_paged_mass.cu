// The attention weight that cached tokens gather from a chunk of new ones:
// per slot n the sum over the chunk's rows r (token, query head of the group)
// of exp(s_rn - lse_r), added to a decayed running mass.
//
// The lse of each row is known, so nothing runs along the slots: with the key
// tile as the M side of the product (S^T = K Q^T, a slot per tensor-memory
// lane) the sum over rows is a thread's own, in a fixed order, and each key
// is decoded once however many rows there are.
//
// The result is an fp32 statistic, so logits need more than the 11 bits of
// fp16, and more than sums on the tensor cores give: those are cut, not
// rounded, at every step, which biased each weight by 3e-6. So keys and rotated
// queries (times scale * log2 e, over a power of two per row) are held as fp16
// pairs whose high parts lie on fixed grids, 2^-12 and 2^-11: the products of
// high parts and their sums below 2 are whole multiples of 2^-23, exact in
// fp32 whatever their order, and have accumulators of their own. K_lo Q_hi +
// K_hi Q_lo, 2^-10 of that, go to a second one (K_lo Q_lo is below 2^-25 per
// term), and the two are added in fp32. Three products bound long chunks.
//
// A first kernel rotates and splits the queries into the tiles the second
// one's bulk copies bring: 64 rows, hi then lo, already swizzled.
//
// Second kernel, per CTA a contiguous run of units of 256 slots of one
// (sequence, head); cuts follow the units' cost. Warps (18): 0-3 and 4-7 sum
// the weights of the unit's first and second 128 slots, 8-11 and 12-15 decode
// them, 16 issues the products, 17 copies query tiles. Both halves use a
// query tile while it is in shared memory, which halves what the copies move.
// 512 tokens of 32/8 heads over 16384 slots (d = 128, b = 3) take 286 us, 130
// of them the products at full rate; single tokens of four sequences of up to
// 32767 slots, bound by the decode, 63 us.

#include <algorithm>

#include "octo_paged.cuh"

namespace octo {
namespace paged {

constexpr int kQRows = 64;    // rows of a query tile
constexpr int kUnit = 256;    // slots of a unit
constexpr float kQGrid = 2048.0f, kKGrid = 4096.0f;  // high parts are multiples of 1 / grid
constexpr int kQPanel = kQRows * 128, kKPanel = 128 * 128;

struct MassArgs {
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
  int q_bf16, Hq, g, causal;
  float scale, decay;
  const float* lse;
  const float* mass_in;
  float* mass_out;
  int64_t mass_stride, n_tiles;  // n_tiles: row tiles that the workspace holds per head
  unsigned char* tiles;  // [row tile][head][hi, lo] images
  float* rows;           // [row tile][head][4][64]: 2^e, -lse * log2 e, its rounding's factor, slots seen (as int)
};

// x as fp16 pair (hi on the grid, lo), low halves of the results
__device__ __forceinline__ void split2(float x, float y, float grid, uint32_t& hi, uint32_t& lo) {
  const __half2 h = __floats2half2_rn(rintf(x * grid) / grid, rintf(y * grid) / grid);
  const float2 b = __half22float2(h);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = half2_bits(x - b.x, y - b.y);
}

__device__ __forceinline__ int query_tiles(const Seq& s, int g) { return (s.fresh * g + kQRows - 1) / kQRows; }

// ---- queries: rotate, scale, split ---------------------------------------------
template <int D>
__global__ void __launch_bounds__(256) paged_mass_prep(const __grid_constant__ MassArgs a) {
  constexpr int E = D / 32, NP = D / 64;
  const int h = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ int s_i, s_m;
  if (warp == 0) {
    int64_t before = 0;
    bool found = false;
    for (int base = 0; base < a.t.n_seqs; base += 32) {
      const int i = base + lane;
      const int mt = i < a.t.n_seqs ? query_tiles(seq_of(a.t, a.seq_lens, a.cu, a.n_rows, i, blockIdx.x == 0 && h == 0), a.g) : 0;
      const int64_t end = before + warp_scan(mt, lane);
      if (static_cast<int64_t>(blockIdx.x) < end && static_cast<int64_t>(blockIdx.x) >= end - mt) {
        s_i = i;
        s_m = static_cast<int>(blockIdx.x - (end - mt));
        found = true;
      }
      before = __shfl_sync(0xffffffffu, end, 31);
    }
    if (!__any_sync(0xffffffffu, found) && lane == 0) s_i = -1;
  }
  __syncthreads();
  const int i = s_i, m = s_m;
  if (i < 0) return;
  const Seq s = seq_of(a.t, a.seq_lens, a.cu, a.n_rows, i);
  const int rows = min(kQRows, s.fresh * a.g - m * kQRows), padded = (rows + 15) / 16 * 16;
  const int64_t tile = static_cast<int64_t>(blockIdx.x) * a.t.n_heads + h;
  unsigned char* hi = a.tiles + tile * (2 * NP * kQPanel);
  unsigned char* lo = hi + NP * kQPanel;
  float* info = a.rows + tile * kQRows * 4;
  const float* sg = a.signs + (h % a.table_heads) * D + lane * E;
  // 1 / sqrt(d) of the rotation, the softmax scale and log2 e in one factor
  const float pre = static_cast<float>(static_cast<double>(a.scale) * 1.4426950408889634 / sqrt(static_cast<double>(D)));
  for (int r = warp; r < padded; r += 8) {
    const bool there = r < rows;
    const int rr = m * kQRows + r, tok = rr / a.g, hq = h * a.g + rr % a.g;
    float v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = 0.0f;
    if (there) {
      const int64_t off = (s.row0 + tok) * a.q_row + hq * a.q_head + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e)
        v[e] = sg[e] * (a.q_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[off + e])
                                 : static_cast<const float*>(a.q)[off + e]);
    }
    fwht_warp<E>(v, lane);
    float mx = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      v[e] *= pre;
      mx = fmaxf(mx, fabsf(v[e]));
    }
    mx = warp_max(mx);
    const int ex = min(max(static_cast<int>(__float_as_uint(mx) >> 23) - 126, -120), 120);  // 2^ex > mx
    const float down = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
    unsigned char *ph = hi + sw128(r, lane * E / 8, kQPanel) + (lane * E % 8) * 2, *pl = ph + (lo - hi);
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      uint32_t h, l;
      split2(v[e] * down, v[e + 1] * down, kQGrid, h, l);
      *reinterpret_cast<uint32_t*>(ph + 2 * e) = h;
      *reinterpret_cast<uint32_t*>(pl + 2 * e) = l;
    }
    if (lane == 0) {
      // a row that is not there, or saw nothing, gives nothing: 2^(x - inf) = 0
      float up = 0.0f, l2 = -INFINITY, z = 0.0f;
      int seen = 0;
      if (there) {
        const float l = a.lse[static_cast<int64_t>(s.row0 + tok) * a.Hq + hq];
        up = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
        if (l != -INFINITY) {
          const double exact = -static_cast<double>(l) * 1.4426950408889634;
          l2 = static_cast<float>(exact);
          z = fabsf(l) < INFINITY ? exp2f(static_cast<float>(exact - static_cast<double>(l2))) : 1.0f;  // (+inf: weight 0; NaN stays)
          seen = a.causal ? max(0, s.len - s.fresh + tok + 1) : s.len;
        }
      }
      info[r] = up;
      info[kQRows + r] = l2;
      info[2 * kQRows + r] = z;
      info[3 * kQRows + r] = __int_as_float(seen);
    }
  }
}

// ---- units ----------------------------------------------------------------------
__device__ __forceinline__ int64_t unit_cost(const Seq& s, int g) { return 4 + 6 * static_cast<int64_t>(query_tiles(s, g)); }
__device__ __forceinline__ int units_of(const Seq& s) { return (s.len + kUnit - 1) / kUnit; }

struct UnitPlace {
  int64_t count;  // units of this CTA
  int64_t tile0;  // query tiles of the sequences before i
  int i, h, u;
};

// Walks a CTA's units.
struct Units {
  const MassArgs& a;
  int64_t left, tile0;
  int i, h, u, first, tiles;  // query tiles [first, tiles) see a slot of the unit
  Seq s;
  __device__ Units(const MassArgs& a_, const UnitPlace& p) : a(a_), left(p.count), tile0(p.tile0), i(p.i), h(p.h), u(p.u) {
    if (left > 0) {
      s = seq_of(a.t, a.seq_lens, a.cu, a.n_rows, i);
      open();
    }
  }
  __device__ void open() {
    tiles = static_cast<int>(min(static_cast<int64_t>(query_tiles(s, a.g)), max(static_cast<int64_t>(0), a.n_tiles - tile0)));
    first = 0;
    // rows before token u*256 - (len - fresh) see no slot of the unit
    if (a.causal) first = static_cast<int>(min(static_cast<int64_t>(tiles), static_cast<int64_t>(max(0, u * kUnit - s.len + s.fresh)) * a.g / kQRows));
  }
  __device__ bool on() const { return left > 0; }
  __device__ int cols(int m) const { return min(kQRows, (s.fresh * a.g - m * kQRows + 15) / 16 * 16); }
  __device__ void next() {
    if (--left <= 0) return;
    if (++u >= units_of(s)) {
      u = 0;
      if (++h >= a.t.n_heads) {
        h = 0;
        do {
          tile0 += query_tiles(s, a.g);
          ++i;
          s = seq_of(a.t, a.seq_lens, a.cu, a.n_rows, i);
        } while (s.len <= 0);
      }
    }
    open();
  }
};

// CTA b takes the units whose cost prefix falls into [b, b + 1) / ctas of the
// whole cost; warp-wide.
__device__ UnitPlace find_units(const MassArgs& a, int lane) {
  int64_t total = 0;
  for (int i = lane; i < a.t.n_seqs; i += 32) {
    const Seq s = seq_of(a.t, a.seq_lens, a.cu, a.n_rows, i);
    total += unit_cost(s, a.g) * units_of(s) * a.t.n_heads;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  const int64_t w0 = blockIdx.x * total / gridDim.x, w1 = (blockIdx.x + 1) * total / gridDim.x;
  UnitPlace p{0, 0, -1, 0, 0};
  int64_t before = 0, tiles = 0;
  for (int base = 0; base < a.t.n_seqs; base += 32) {
    const int i = base + lane;
    Seq s{0, 0, 0};
    if (i < a.t.n_seqs) s = seq_of(a.t, a.seq_lens, a.cu, a.n_rows, i);
    const int64_t n = static_cast<int64_t>(units_of(s)) * a.t.n_heads, c = unit_cost(s, a.g), w = n * c;
    const int64_t end = before + warp_scan(w, lane), start = end - w;
    const int64_t tend = tiles + warp_scan(query_tiles(s, a.g), lane);
    // units k of this sequence with start + k * c in [w0, w1)
    const int64_t k0 = min(n, max(static_cast<int64_t>(0), (w0 - start + c - 1) / c)),
                  k1 = min(n, max(static_cast<int64_t>(0), (w1 - start + c - 1) / c));
    int64_t mine = (start >= w1 || end <= w0) ? 0 : k1 - (w0 <= start ? 0 : k0);
    mine = max(mine, static_cast<int64_t>(0));
    const uint32_t has = __ballot_sync(0xffffffffu, mine > 0);
    if (has && p.i < 0) {
      const int who = __ffs(has) - 1;
      const int64_t k = w0 <= start ? 0 : k0;
      const int uo = units_of(s);
      p.i = __shfl_sync(0xffffffffu, i, who);
      p.h = __shfl_sync(0xffffffffu, uo ? static_cast<int>(k / uo) : 0, who);
      p.u = __shfl_sync(0xffffffffu, uo ? static_cast<int>(k % uo) : 0, who);
      p.tile0 = __shfl_sync(0xffffffffu, tend - query_tiles(s, a.g), who);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
    p.count += mine;
    before = __shfl_sync(0xffffffffu, end, 31);
    tiles = __shfl_sync(0xffffffffu, tend, 31);
  }
  return p;
}

template <int D, int B>
struct MassCfg {
  using K = Code<D, B>;
  static constexpr int NP = D / 64;
  static constexpr int KT = NP * kKPanel;          // one part (hi or lo) of a 128-slot key tile
  static constexpr int QT = NP * kQPanel;          // one part of a query tile
  // Entries of 16 bytes, 8 copies of each: the lanes of a quarter-warp read
  // distinct banks (one copy of every signed code at b = 3 met 2.5 a bank, and
  // the lookups bound single tokens). b = 2 every signed code, b = 3 those of
  // the positive quadrant, as {x, y hi | z hi | x, y lo | z lo} (fp16 pairs);
  // b = 4 the quadrant's unit directions in fp32, times the norm level in
  // registers. A code's signs flip sign bits (the codebook and the inverse map
  // are odd in x and in y).
  static constexpr bool SPLIT = B == 4, QUAD = B > 2;
  static constexpr int NE = B == 2 ? 128 : 256, REP = 8, SH = 4 + 3;
  static constexpr int KB = 0, QB = 4 * KT, TAB = QB + 4 * QT, RHO = TAB + (NE << SH), ROWS = RHO + 32;
  static constexpr int BARS = ROWS + 2 * kQRows * 16, PLACE = BARS + 16 * 8, TMEM = PLACE + 40, DIR = PLACE + 48,
                       SMEM = DIR + 128;
  static constexpr int THREADS = 576;
  static_assert(SMEM <= 232448, "shared memory of an SM");
};

enum { mKF = 0, mKE = 2, mQF = 4, mQE = 6, mDF = 8, mDE = 12 };  // D barriers: [half][buffer]; the sixteen fill 128 bytes

template <int D, int B>
__device__ __forceinline__ bool mass_decode(const MassArgs& a, const UnitPlace& place, unsigned char* sm, uint32_t bars,
                                            int half) {
  using Cfg = MassCfg<D, B>;
  using K = Code<D, B>;
  constexpr int W = K::W;
  const int n = threadIdx.x & 127;
  const uint32_t copy = (threadIdx.x & (Cfg::REP - 1)) * 16;  // this lane's copy of the table
  // words are fetched a unit ahead, page ids a unit before that
  uint32_t w[W], wn[W];
  Units it(a, place);
  int slot = 0, id = 0;
  bool held = false, more = false;
  auto look = [&] {
    slot = it.u * kUnit + half * 128 + n;
    held = it.on() && slot < it.s.len;
    if (held) id = static_cast<int>(load_now(page_entry(a.t, it.i, slot)));
  };
  auto fetch = [&] {
#pragma unroll
    for (int k = 0; k < W; ++k) wn[k] = 0u;
    more = it.on();
    if (!more) return;
    if (held) {
      const uint32_t* p = a.packed + (static_cast<int64_t>(max(0, page_checked(a.t, id))) * a.t.n_heads + it.h) * W * a.t.page_size +
                          page_offset(a.t, slot);
#pragma unroll
      for (int k = 0; k < W; ++k) wn[k] = load_now(p + static_cast<int64_t>(k) * a.t.page_size);
    }
    do it.next();
    while (it.on() && it.first >= it.tiles);
    look();
  };
  while (it.on() && it.first >= it.tiles) it.next();
  look();
  for (int c = -1; c < 0 || more; ++c) {  // the first turn only fetches
#pragma unroll
    for (int k = 0; k < W; ++k) w[k] = wn[k];
    const bool now = c >= 0;
    fetch();
    if (!now) continue;
    if (!bar_wait(bars + 8 * (mKE + half), (c & 1) ^ 1)) return false;
    unsigned char* hi = sm + Cfg::KB + half * 2 * Cfg::KT;
    unsigned char* lo = hi + Cfg::KT;
    constexpr int GROUPS = (D + 23) / 24;
#pragma unroll 1
    for (int grp = 0; grp < GROUPS; ++grp) {
      uint32_t oh[12], ol[12];
#pragma unroll
      for (int pr = 0; pr < 4; ++pr) {
        uint4 e[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int i = 2 * pr + u;  // (codes behind the key's last are zeros of the stream, and their halves go nowhere)
          const uint32_t code = code_at<K::C, Cfg::SH>(w, i);
          constexpr int sx = 2 * B + Cfg::SH, sy = sx + 1;  // sign bits in code
          uint32_t at = code;
          if constexpr (Cfg::QUAD) at = code & ((1u << sx) - (1u << Cfg::SH));
          if constexpr (B == 3) at |= (code >> 2) & (3u << sx);  // the norm level's two bits behind
          e[u] = *reinterpret_cast<const uint4*>(sm + Cfg::TAB + (at | copy));
          if constexpr (Cfg::SPLIT) {
            const float r = *reinterpret_cast<const float*>(sm + Cfg::RHO + (code >> (K::DIR + Cfg::SH)) * 4);
            const float x = __uint_as_float(e[u].x ^ ((code << (31 - sx)) & 0x80000000u)) * r;
            const float y = __uint_as_float(e[u].y ^ ((code << (31 - sy)) & 0x80000000u)) * r;
            const float z = __uint_as_float(e[u].z) * r;
            split2(x, y, kKGrid, e[u].x, e[u].z);
            split2(z, 0.0f, kKGrid, e[u].y, e[u].w);
          } else if constexpr (Cfg::QUAD) {  // s_xi to bit 15, s_eta to bit 31
            const uint32_t flip = ((code << (15 - sx)) & 0x8000u) | ((code << (31 - sy)) & 0x80000000u);
            e[u].x ^= flip;
            e[u].z ^= flip;
          }
        }
        oh[3 * pr] = e[0].x;
        oh[3 * pr + 1] = lolo(e[0].y, e[1].x);
        oh[3 * pr + 2] = hilo(e[1].x, e[1].y);
        ol[3 * pr] = e[0].z;
        ol[3 * pr + 1] = lolo(e[0].w, e[1].z);
        ol[3 * pr + 2] = hilo(e[1].z, e[1].w);
      }
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        const int chunk = grp * 3 + q;
        if (chunk < D / 8) {
          const uint32_t at = sw128(n, chunk, kKPanel);
          *reinterpret_cast<uint4*>(hi + at) = make_uint4(oh[4 * q], oh[4 * q + 1], oh[4 * q + 2], oh[4 * q + 3]);
          *reinterpret_cast<uint4*>(lo + at) = make_uint4(ol[4 * q], ol[4 * q + 1], ol[4 * q + 2], ol[4 * q + 3]);
        }
      }
      next_codes<K::C>(w);
    }
    fence_async_shared();
    bar_arrive(bars + 8 * (mKF + half));
    if (!more) break;
  }
  return true;
}

template <int D, int B>
__device__ __forceinline__ bool mass_copies(const MassArgs& a, const UnitPlace& place, uint32_t base, uint32_t bars,
                                            int& issued) {
  using Cfg = MassCfg<D, B>;
  const int lane = threadIdx.x & 31;
  int c = 0;
  for (Units it(a, place); it.on(); it.next())
    for (int m = it.first; m < it.tiles; ++m, ++c) {
      const int st = c & 1;
      if (!bar_wait(bars + 8 * (mQE + st), ((c >> 1) & 1) ^ 1)) return false;
      const uint32_t n = it.cols(m), bytes = n * 128;
      const int64_t tile = (it.tile0 + m) * a.t.n_heads + it.h;
      const unsigned char* src = a.tiles + tile * (2 * Cfg::QT);
      if (lane == 0) {
        bar_expect(bars + 8 * (mQF + st), 2 * Cfg::NP * bytes + kQRows * 16);
        issued = c + 1;
        for (int p = 0; p < 2 * Cfg::NP; ++p)
          bulk_in(base + Cfg::QB + st * 2 * Cfg::QT + p * kQPanel, src + p * kQPanel, bytes, bars + 8 * (mQF + st));
        bulk_in(base + Cfg::ROWS + st * kQRows * 16, a.rows + tile * kQRows * 4, kQRows * 16, bars + 8 * (mQF + st));
      }
      __syncwarp();
    }
  return true;
}

// S^T of one half from a query tile of N columns: D = K_hi Q_hi, D + 64
// columns = K_lo Q_hi + K_hi Q_lo. k, q: descriptors of the high parts; the low
// ones lie KT and QT bytes behind.
template <int D, int B>
__device__ __noinline__ void issue_scores(uint32_t d, uint32_t k, uint32_t q, uint32_t idesc) {
  using Cfg = MassCfg<D, B>;
  if (elect_one()) {
#pragma unroll 1
    for (int part = 0; part < 3; ++part) {
      const uint32_t kk = k + (part == 1 ? Cfg::KT >> 4 : 0), qq = q + (part == 2 ? Cfg::QT >> 4 : 0);
      const uint32_t to = d + (part == 0 ? 0 : kQRows);
#pragma unroll
      for (int s = 0; s < D / 16; ++s)
        mma_ss(to, kk + (((s >> 2) * kKPanel + (s & 3) * 32) >> 4), qq + (((s >> 2) * kQPanel + (s & 3) * 32) >> 4), idesc,
               s > 0 || part == 2);
    }
  }
  __syncwarp();
}

template <int D, int B>
__device__ __forceinline__ bool mass_products(const MassArgs& a, const UnitPlace& place, uint32_t base, uint32_t bars) {
  using Cfg = MassCfg<D, B>;
  int c = 0, k = 0;
  for (Units it(a, place); it.on(); it.next()) {
    if (it.first >= it.tiles) continue;
    for (int m = it.first; m < it.tiles; ++m, ++c) {
      const int st = c & 1;
      if (!bar_wait(bars + 8 * (mQF + st), (c >> 1) & 1)) return false;
      const uint32_t idesc = instr_desc(128, it.cols(m), false, false);
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        if (m == it.first && !bar_wait(bars + 8 * (mKF + half), k & 1)) return false;
        if (!bar_wait(bars + 8 * (mDE + half * 2 + st), ((c >> 1) & 1) ^ 1)) return false;
        tc_after();
        issue_scores<D, B>((half * 2 + st) * 2 * kQRows, desc_low(base + Cfg::KB + half * 2 * Cfg::KT, 16),
                           desc_low(base + Cfg::QB + st * 2 * Cfg::QT, 16), idesc);
        if (elect_one()) {
          tc_commit(bars + 8 * (mDF + half * 2 + st));
          if (m + 1 == it.tiles) tc_commit(bars + 8 * (mKE + half));
          if (half == 1) tc_commit(bars + 8 * (mQE + st));
        }
        __syncwarp();
      }
    }
    ++k;
  }
  return true;
}

template <int D, int B>
__device__ __forceinline__ bool mass_sums(const MassArgs& a, const UnitPlace& place, unsigned char* sm, uint32_t bars,
                                          uint32_t tmem, int half) {
  using Cfg = MassCfg<D, B>;
  const int n = threadIdx.x & 127;
  const uint32_t D0 = tmem + (static_cast<uint32_t>((threadIdx.x >> 5) & 3) << 21) + half * 4 * kQRows;
  int c = 0;
  for (Units it(a, place); it.on(); it.next()) {
    const int slot = it.u * kUnit + half * 128 + n, k0 = slot - n;
    const bool held = slot < it.s.len, kept = held && slot < a.mass_stride;
    const int64_t at = (static_cast<int64_t>(it.i) * a.t.n_heads + it.h) * a.mass_stride + slot;
    float gamma = 0.0f, mass = 0.0f;
    if (held) {
      const int pg = max(0, page_of(a.t, it.i, slot));
      gamma = __ldg(a.gamma + (static_cast<int64_t>(pg) * a.t.n_heads + it.h) * a.t.page_size + page_offset(a.t, slot));
    }
    if (kept && a.mass_in) mass = a.decay * a.mass_in[at];
    if (held && !kept) report(a.t.status, OCTO_PAGED_BAD_LENGTH);
    float sum = 0.0f;
    for (int m = it.first; m < it.tiles; ++m, ++c) {
      const int st = c & 1;
      // the rows' numbers came with the query tile
      if (!bar_wait(bars + 8 * (mDF + half * 2 + st), (c >> 1) & 1)) return false;
      if (!bar_wait(bars + 8 * (mQF + st), (c >> 1) & 1)) return false;
      tc_after();
      const float* rows = reinterpret_cast<const float*>(sm + Cfg::ROWS) + st * kQRows * 4;
      const int cols = it.cols(m);
      // some row of the tile does not see some slot of this half, or the half runs past the sequence
      const bool masked = __float_as_int(rows[3 * kQRows]) < k0 + 128;
      const uint32_t S = D0 + st * 2 * kQRows;
      float2 part[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
      const float2 gg = make_float2(gamma, gamma);
      auto weigh = [&](const uint32_t (&s)[16], const uint32_t (&t)[16], int x0) {
#pragma unroll
        for (int x = 0; x < 16; x += 4) {
          const float4 f = *reinterpret_cast<const float4*>(rows + x0 + x);
          const float4 l = *reinterpret_cast<const float4*>(rows + kQRows + x0 + x);
          const float4 z = *reinterpret_cast<const float4*>(rows + 2 * kQRows + x0 + x);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const int i = x + 2 * y;
            const float2 sc = add_f32x2(make_float2(__uint_as_float(s[i]), __uint_as_float(s[i + 1])),
                                        make_float2(__uint_as_float(t[i]), __uint_as_float(t[i + 1])));
            const float2 e = fma_f32x2(sc, mul_f32x2(gg, y ? make_float2(f.z, f.w) : make_float2(f.x, f.y)),
                                       y ? make_float2(l.z, l.w) : make_float2(l.x, l.y));
            float2 w = make_float2(ex2(e.x), ex2(e.y));
            if (masked) {
              if (slot >= __float_as_int(rows[3 * kQRows + x0 + i])) w.x = 0.0f;
              if (slot >= __float_as_int(rows[3 * kQRows + x0 + i + 1])) w.y = 0.0f;
            }
            part[y] = fma_f32x2(w, y ? make_float2(z.z, z.w) : make_float2(z.x, z.y), part[y]);
          }
        }
      };
#pragma unroll 1
      for (int x0 = 0; x0 < cols; x0 += 16) {
        uint32_t s[16], t[16];
        tmem_ld16(s, S + x0);
        tmem_ld16(t, S + kQRows + x0);
        tc_wait_ld(s, t);
        weigh(s, t, x0);
      }
      part[0] = add_f32x2(part[0], part[1]);
      sum += part[0].x + part[0].y;
      tc_before();
      bar_arrive(bars + 8 * (mDE + half * 2 + st));
      bar_arrive(bars + 8 * (mQE + st));
    }
    if (kept) a.mass_out[at] = mass + sum;
  }
  return true;
}

template <int D, int B>
__global__ void __launch_bounds__(576, 1) paged_mass_kernel(const __grid_constant__ MassArgs a) {
  using Cfg = MassCfg<D, B>;
  using K = Code<D, B>;
  extern __shared__ __align__(1024) unsigned char sm[];
  const uint32_t base = s32(sm), bars = base + Cfg::BARS;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  UnitPlace& s_place = *reinterpret_cast<UnitPlace*>(sm + Cfg::PLACE);
  uint32_t& s_tmem = *reinterpret_cast<uint32_t*>(sm + Cfg::TMEM);
  float* s_dir = reinterpret_cast<float*>(sm + Cfg::DIR);
  float* s_rho = reinterpret_cast<float*>(sm + Cfg::RHO);
  if (tid < (1 << (B + 1))) s_dir[tid] = a.dir_c[tid];
  if (tid < K::NRHO) s_rho[tid] = a.rho_c[tid];
  if (warp == 17) {
    const UnitPlace p = find_units(a, lane);
    if (lane == 0) s_place = p;
  }
  if (tid == 0) {
    for (int q = 0; q < 2; ++q) {
      bar_init(bars + 8 * (mKF + q), 128);
      bar_init(bars + 8 * (mKE + q), 1);
      bar_init(bars + 8 * (mQF + q), 1);
      bar_init(bars + 8 * (mQE + q), 1 + 256);
    }
    for (int q = 0; q < 4; ++q) {
      bar_init(bars + 8 * (mDF + q), 1);
      bar_init(bars + 8 * (mDE + q), 128);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 16) tmem_alloc(s32(&s_tmem), 512);
  __syncthreads();
  const UnitPlace place = s_place;
  if (place.count > 0) {
    for (int e = tid; e < Cfg::NE; e += Cfg::THREADS) {
      const float3 d = field_direction<B>(Cfg::QUAD ? e & ((1 << 2 * B) - 1) : e & (K::NDIR - 1), s_dir);
      uint4 v;
      if constexpr (Cfg::SPLIT) {
        v = make_uint4(__float_as_uint(d.x), __float_as_uint(d.y), __float_as_uint(d.z), 0u);
      } else {
        const float r = s_rho[Cfg::QUAD ? e >> (2 * B) : e >> K::DIR];
        split2(d.x * r, d.y * r, kKGrid, v.x, v.z);
        split2(d.z * r, 0.0f, kKGrid, v.y, v.w);
      }
#pragma unroll
      for (int k = 0; k < Cfg::REP; ++k) *reinterpret_cast<uint4*>(sm + Cfg::TAB + (e << Cfg::SH) + k * 16) = v;
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  constexpr uint32_t tmem = 0;  // the allocation is the whole tensor memory, so it starts at column 0
  bool ok = true;
  if (place.count > 0) {
    if (warp < 8) {
      ok = mass_sums<D, B>(a, place, sm, bars, tmem, warp >> 2);
    } else if (warp < 16) {
      ok = mass_decode<D, B>(a, place, sm, bars, (warp - 8) >> 2);
    } else if (warp == 16) {
      ok = mass_products<D, B>(a, place, base, bars);
      if (!ok) {  // products in flight end before tensor memory is given back (a fresh barrier in the table's place)
        if (lane == 0) {
          bar_init(base + Cfg::PLACE, 1);
          asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
          tc_commit(base + Cfg::PLACE);
        }
        __syncwarp();
        bar_wait(base + Cfg::PLACE, 0);
      }
    } else {
      int issued = 0;
      ok = mass_copies<D, B>(a, place, base, bars, issued);
      issued = __shfl_sync(0xffffffffu, issued, 0);
      // copies in flight end before the CTA does
      for (int c = max(0, issued - 2); c < issued; ++c) bar_wait(bars + 8 * (mQF + (c & 1)), (c >> 1) & 1);
    }
  }
  if (!ok && lane == 0) report(a.t.status, OCTO_PAGED_TIMEOUT);
  tc_before();
  __syncthreads();
  if (warp == 16) tmem_free(s_tmem, 512);
}

// ---- host -------------------------------------------------------------------------
// row tiles of all sequences, at most
static int64_t most_tiles(int64_t n_rows, int n_seqs, int g) { return n_rows * g / kQRows + n_seqs; }

template <int D, int B>
static cudaError_t launch_mass(const MassArgs& a, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.n_tiles), a.t.n_heads);
  paged_mass_prep<D><<<grid, 256, 0, st>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  static LaunchCache cache;
  int resident = 0;
  e = launch_setup(paged_mass_kernel<D, B>, cache, MassCfg<D, B>::THREADS, MassCfg<D, B>::SMEM, resident);
  if (e != cudaSuccess) return e;
  paged_mass_kernel<D, B><<<sm_count(), MassCfg<D, B>::THREADS, MassCfg<D, B>::SMEM, st>>>(a);
  return cudaGetLastError();
}

}  // namespace paged
}  // namespace octo

extern "C" size_t octo_paged_mass_workspace(const octo_layout* L, int64_t n_rows, int n_seqs, int Hq, int Hkv) {
  using namespace octo::paged;
  if (check_layout(L) != OCTO_OK || L->d > 128 || n_rows < 0 || n_seqs < 0 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0)
    return 0;
  const size_t tiles = static_cast<size_t>(most_tiles(n_rows, n_seqs, Hq / Hkv)) * Hkv;
  return kDecodeFront + tiles * (static_cast<size_t>(2) * kQRows * L->d * 2 + kQRows * sizeof(float4));
}

extern "C" int octo_paged_mass(const octo_layout* L, const octo_tables* tab, const octo_pages* pages,
                               const octo_page_table* table, const int32_t* seq_lens, const void* q, int q_dtype,
                               int64_t q_row_stride, int64_t q_head_stride, int64_t n_rows, int Hq,
                               const int32_t* cu_q, int causal, float scale, const float* lse, float decay,
                               const float* mass_in, float* mass_out, int64_t mass_stride, void* workspace,
                               size_t ws_bytes, octo_stream_t stream) {
  using namespace octo::paged;
  int c = check_layout(L);
  if (c != OCTO_OK) return c;
  if (L->d > 128) return OCTO_EUNSUPPORTED;
  if ((c = check_pages(pages)) != OCTO_OK) return c;
  if ((c = check_table(table, pages->page_size)) != OCTO_OK) return c;
  if (!tab || !tab->dir_c || !tab->rho_c || !tab->signs || tab->n_heads < 1) return OCTO_EINVAL;
  if (q_dtype != OCTO_F32 && q_dtype != OCTO_BF16) return OCTO_EINVAL;
  if (n_rows < 0 || q_row_stride < 0 || q_head_stride < 0 || Hq < pages->n_heads || Hq % pages->n_heads != 0 ||
      mass_stride < 0)
    return OCTO_EINVAL;
  if (!(scale - scale == 0.0f) || !(decay - decay == 0.0f)) return OCTO_EINVAL;  // NaN or infinite
  const int g = Hq / pages->n_heads;
  if (g > 256 || n_rows * g > INT32_MAX - 1024 || pages->n_heads > 65535) return OCTO_EUNSUPPORTED;
  if (table->n_seqs == 0 || (n_rows == 0 && !mass_out)) return OCTO_OK;
  if (!mass_out || !seq_lens || !cu_q) return OCTO_EINVAL;
  if (n_rows > 0) {  // (without rows the masses still decay, and the rest is not read)
    if (!q || !lse) return OCTO_EINVAL;
    if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return OCTO_EINVAL;
    if (ws_bytes < octo_paged_mass_workspace(L, n_rows, table->n_seqs, Hq, pages->n_heads)) return OCTO_EWORKSPACE;
  }
  MassArgs a{};
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
  a.decay = decay;
  a.lse = lse;
  a.mass_in = mass_in;
  a.mass_out = mass_out;
  a.mass_stride = mass_stride;
  a.n_tiles = most_tiles(n_rows, table->n_seqs, g);
  const size_t tiles = static_cast<size_t>(a.n_tiles) * pages->n_heads;
  if (n_rows > 0) {
    a.tiles = static_cast<unsigned char*>(workspace) + kDecodeFront;
    a.rows = reinterpret_cast<float*>(a.tiles + tiles * (static_cast<size_t>(2) * kQRows * L->d * 2));
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (L->d == 64)
    e = L->b == 2 ? launch_mass<64, 2>(a, st) : L->b == 3 ? launch_mass<64, 3>(a, st) : launch_mass<64, 4>(a, st);
  else
    e = L->b == 2 ? launch_mass<128, 2>(a, st) : L->b == 3 ? launch_mass<128, 3>(a, st) : launch_mass<128, 4>(a, st);
  return e == cudaSuccess ? OCTO_OK : OCTO_ECUDA;
}
