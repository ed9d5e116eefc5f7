// Attention of a chunk of new tokens over the paged compressed cache.
//
// Per sequence and KV head the rows are the chunk's (token, query head of the
// group) pairs; row r's logits over slot n are
//   s_rn = scale * gamma_n * <R q_r, u_hat_n>,
// and its output softmax(s_r) V, by one pass over the slots with a running
// reference m_r and sum l_r (base 2): o_r accumulates 2^(s - m) v, and is
// rescaled when the weights outgrow the reference (Row below).
//
// Matrix work on tcgen05: S = Q K^T with 128-row query tiles (fp16, scaled by
// a power of two where a row leaves its range) and 128-slot key tiles, whose
// rows are the decoded unit directions in fp16 (gamma is applied to S in
// fp32, so a key's norm costs no precision); O += P V with P in bf16 in
// tensor memory, in place of its S, and V (bf16) as TMA brings it. A CTA
// holds two query tiles (256 rows), so each key tile is decoded once per 256
// rows. Tensor memory: S0, S1 (128 columns each), O0, O1 (D columns each).
//
// Warps (16): 0-3 and 4-7 the softmax of query tile 0 and 1 (a thread owns a
// row: no shuffles), and before it the rotation of their queries; 8-11 decode
// key tiles, a thread per slot, one ahead of the products; 12 issues the
// products; 13 copies V and zeroes
// the rows behind a sequence's end.
//
// Items of at most 128 rows would leave the second query tile empty and the
// softmax of few rows to few warps. There both S and O pairs serve the one
// query tile, key tiles alternating between them (so a product runs while the
// other tile's softmax does), and with at most 64 or 32 rows the query tile
// holds the rows two or four times, each copy taking its half or quarter of
// the key tile's columns (weights 0 elsewhere). The copies are rows of their
// own, with references and sums of their own, and are added at the end.
//
// Schedule: the (sequence, head, 256-row tile) items' key tiles form one
// list, cut into equal contiguous pieces, one per CTA, whatever the lengths.
// An item that several CTAs share leaves fp32 partials (m, l, O) in the
// workspace: at most the first and the last item of a CTA's piece, so two
// slots per CTA; a second kernel joins them.
//
// Bound by the softmax warps, which read S twice from tensor memory (a bound
// on the logits, then the weights) in turn with the products: 512 tokens of
// 32/8 heads over 32768 slots (d = 128, b = 3) take 370 us, 750 TFLOP/s;
// 1024 tokens of 16 heads over 65536 slots (d = 64, b = 2) 588 us. With few
// rows the decode of key tiles bounds: one token over 32767 slots takes 52 us
// for 83 MB.

#include <cudaTypedefs.h>

#include <algorithm>
#include <climits>
#include <cstring>

#include "octo_paged.cuh"

namespace octo {
namespace paged {

constexpr int kRows = 256;   // query rows of an item
constexpr int kKeys = 128;   // slots of a key tile
constexpr int kJoin = 148;    // CTAs that may share an item: the launch has no more
constexpr int kJoinRows = 4;  // rows of a block of the join
constexpr int kPanel = 128 * 128;  // bytes of a 128-row panel of 64 halves

// An item that a CTA begins and others go on with, as the join finds it: its
// rows, and the number of CTAs that hold a piece (0: the CTA begins no such item).
struct Shared {
  int pieces, rows, copies, row0, h, m, pad[2];  // copies: row copies in each piece
};

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
  int q_bf16, q_vec, Hq, g, causal, box;  // q_vec: query rows allow 16-byte loads; box: V rows per copy
  float scale;
  void* out;
  int out_bf16;
  float* lse;
  float4* part_o;  // [slots][D / 4][256]: lanes own rows, so their accesses are contiguous
  float4* copies;  // [CTAs][D / 4][256]: the row copies of an item of at most 128 rows, on their way to their sum
  float2* part_ml; // [slots][256]
  float* part_e;   // [slots][256]: sums of the weights before their rounding, where lse is asked for
  Shared* shared;  // [CTAs]
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
  int64_t start, count, total;  // the piece's first key tile in the list and their number; tiles of the list
  int i, h, m, tile;
};
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
  Place p{0, 0, total, 0, 0, 0, 0};
  if (blockIdx.x >= ctas) return p;
  const int64_t at = blockIdx.x * total / ctas;
  p.start = at;
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
  // copies of the rows in a query tile; 0: more than 128 rows, two query tiles
  __device__ int reps() const {
    const int r = rows();
    return r > 128 ? 0 : r > 64 ? 1 : r > 32 ? 2 : 4;
  }
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
  // Table entries of 8 bytes {x, y | z, z} (fp16). b = 2 and 3: every signed
  // code, copied 16 and 4 times (the lanes of a half-warp then meet none or
  // two to three in a bank; the positive quadrant alone, copied 16 times, met
  // none at b = 3 too, but restoring the signs cost more than the banks).
  // b = 4 (8192 codes): the positive quadrant's directions, copied 16 times,
  // multiplied by the norm level from a second table; the codebook and the
  // inverse map are odd in x and in y, so the signs flip sign bits.
  static constexpr bool QUAD = B == 4;
  static constexpr int NE = B == 2 ? 128 : B == 3 ? 1024 : 256, REP = B == 3 ? 4 : 16;
  static constexpr int SH = 3 + (REP == 16 ? 4 : 2);  // log2 bytes of an entry with its copies
  // gamma rows in flight: a row is written when the product of the tile two before is done, and that one may be
  // issued while the tile before it is still read
  static constexpr int GS = 4;
  static constexpr int Q = 0, KT = 2 * TILE, V = 4 * TILE, TAB = 6 * TILE, RHO = TAB + (NE << SH);
  static constexpr int GAM = RHO + (QUAD ? 8 * 8 * 4 : 0), GMAX = GAM + GS * kKeys * 4, EXPS = GMAX + GS * 16,
                       BARS = EXPS + 256;
  static constexpr int PLACE = BARS + 18 * 8, TMEM = PLACE + 40, DIR = PLACE + 48, RHOF = DIR + 128, SMEM = RHOF + 32;
  static_assert(SMEM <= 232448, "shared memory of an SM");
  static constexpr int THREADS = 512;
};

// barriers
enum { kQF = 0, kSF = 2, kPR = 4, kKF = 6, kKE = 8, kVF = 10, kVE = 12, kVZ = 14, kEND = 16, kMEET = 17, kBars = 18 };

__device__ __forceinline__ uint32_t bf16_pair(float x, float y) {
  const __nv_bfloat162 b2 = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&b2);
}

// ---- decode warps: key tiles ------------------------------------------------
template <int D, int B>
__device__ __forceinline__ bool decode_role(const AttnArgs& a, const Place& place, unsigned char* sm, uint32_t base,
                                            uint32_t bars) {
  using Cfg = AttnCfg<D, B>;
  using K = Code<D, B>;
  constexpr int W = K::W;
  const int n = threadIdx.x & 127, lane = threadIdx.x & 31;
  const uint32_t copy = (lane & (Cfg::REP - 1)) * 8, rcopy = (lane & 7) * 4;  // this lane's copies of the tables
  // Words are fetched a tile ahead, and their page id a tile before that: a
  // page lookup or a first use would otherwise wait for memory every tile.
  uint32_t w[W], wn[W];
  float gm = 0.0f, gn = 0.0f;
  Walk it(a, place);
  int tile = 0, id = 0;     // the walk's tile, and the page of this thread's slot in it (as read: checked at its use)
  bool held = false;        // the sequence holds that slot
  auto look = [&] {
    const int slot = tile * kKeys + n;
    held = it.on() && slot < it.s.len;
    if (held) id = static_cast<int>(load_now(page_entry(a.t, it.i, slot)));
  };
  auto start = [&] {
    while (it.on() && it.work() == 0) it.next();
    if (it.on()) tile = it.t0;
    look();
  };
  // words and gamma of this thread's slot of the walk's tile (0 behind the sequence); the walk steps on
  int valid = 0, vn = 0;    // slots of the current and the next tile that the sequence holds; 0: no tile
  auto fetch = [&] {
#pragma unroll
    for (int k = 0; k < W; ++k) wn[k] = 0u;
    gn = 0.0f;
    vn = 0;
    if (!it.on()) return;
    vn = it.s.len - tile * kKeys;
    if (held) {
      const int64_t row = static_cast<int64_t>(max(0, page_checked(a.t, id))) * a.t.n_heads + it.h;
      const int off = page_offset(a.t, tile * kKeys + n);
      const uint32_t* p = a.packed + row * W * a.t.page_size + off;
#pragma unroll
      for (int k = 0; k < W; ++k) wn[k] = load_now(p + static_cast<int64_t>(k) * a.t.page_size);
      gn = __uint_as_float(load_now(a.gamma + row * a.t.page_size + off));
    }
    if (++tile < it.t1) {
      look();
    } else {
      it.next();
      start();
    }
  };
  start();
  fetch();
  for (int c = 0; vn != 0; ++c) {
    {
#pragma unroll
      for (int k = 0; k < W; ++k) w[k] = wn[k];
      gm = gn;
      valid = vn;
      fetch();
      const int st = c & 1;
      if (!bar_wait(bars + 8 * (kKE + st), ((c >> 1) & 1) ^ 1)) return false;
      reinterpret_cast<float*>(sm + Cfg::GAM)[(c % Cfg::GS) * kKeys + n] = gm;
      // the warp's largest |gamma| (as bits: NaN above all)
      const uint32_t gb = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(gm)));
      if (lane == 0) reinterpret_cast<uint32_t*>(sm + Cfg::GMAX)[(c % Cfg::GS) * 4 + (n >> 5)] = gb;
      unsigned char* kt = sm + Cfg::KT + st * Cfg::TILE;
      // groups of 8 triplets: 24 halves, three 16-byte chunks of the row
      constexpr int GROUPS = (D + 23) / 24;
#pragma unroll 1
      for (int grp = 0; grp < GROUPS; ++grp) {
        uint32_t o[12];
#pragma unroll
        for (int pr = 0; pr < 4; ++pr) {
          uint2 e[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int i = 2 * pr + u;
            {  // (codes behind the key's last are zeros of the stream, and their halves go nowhere)
              // code << SH is the byte offset of its entry (QUAD: of its direction's, without the signs)
              const uint32_t code = code_at<K::C, Cfg::SH>(w, i);
              uint32_t at = code;
              if constexpr (Cfg::QUAD) at = code & ((1u << (2 * B + Cfg::SH)) - (1u << Cfg::SH));
              e[u] = *reinterpret_cast<const uint2*>(sm + Cfg::TAB + (at | copy));
              if constexpr (Cfg::QUAD) {
                const __half2 r2 = *reinterpret_cast<const __half2*>(
                    sm + Cfg::RHO + (((code >> (K::DIR + Cfg::SH - 5)) & 0xe0u) | rcopy));
                const __half2 x = __hmul2(*reinterpret_cast<const __half2*>(&e[u].x), r2);
                const __half2 z = __hmul2(*reinterpret_cast<const __half2*>(&e[u].y), r2);
                e[u].x = *reinterpret_cast<const uint32_t*>(&x);
                e[u].y = *reinterpret_cast<const uint32_t*>(&z);
                constexpr int sx = 2 * B + Cfg::SH, sy = sx + 1;  // s_xi to bit 15, s_eta to bit 31
                e[u].x ^= ((code << (15 - sx)) & 0x8000u) | ((code << (31 - sy)) & 0x80000000u);
              }
            }
          }
          o[3 * pr] = e[0].x;
          o[3 * pr + 1] = lolo(e[0].y, e[1].x);
          o[3 * pr + 2] = hilo(e[1].x, e[1].y);
        }
#pragma unroll
        for (int q = 0; q < 3; ++q) {
          const int chunk = grp * 3 + q;
          if (chunk < D / 8)
            *reinterpret_cast<uint4*>(kt + sw128(n, chunk, kPanel)) =
                make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        }
        next_codes<K::C>(w);
      }
      fence_async_shared();
      bar_arrive(bars + 8 * (kKF + st));
    }
  }
  return true;
}

// ---- V copies ---------------------------------------------------------------
template <int D, int B>
__device__ __forceinline__ bool v_role(const AttnArgs& a, const Place& place, const CUtensorMap* map, unsigned char* sm,
                                       uint32_t base, uint32_t bars, int& issued) {
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
          tma_3d(base + Cfg::V + st * Cfg::TILE + p * kPanel + b * a.box * 128, map, p * 64, page_offset(a.t, slot),
                 pg * a.t.n_heads + it.h, bars + 8 * (kVF + st));
      }
      __syncwarp();
      // V rows behind the sequence's end hold whatever the page or the stage
      // held: zero them once the copy is in (0 * NaN would reach the output).
      // This warp alone can: it knows that the stage's last products are done
      // and that the copy it waits for is the stage's newest.
      if (valid < kKeys) {
        if (!bar_wait(bars + 8 * (kVF + st), (c >> 1) & 1)) return false;
        unsigned char* vt = sm + Cfg::V + st * Cfg::TILE;
        for (int n = valid * 8 + lane; n < kKeys * 8; n += 32) {
#pragma unroll
          for (int p = 0; p < Cfg::NP; ++p)
            *reinterpret_cast<uint4*>(vt + p * kPanel + n * 16) = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_async_shared();
        bar_arrive(bars + 8 * (kVZ + st));
      }
    }
  }
  return true;
}

// ---- products ---------------------------------------------------------------
// S = query tile times key tile; O (+)= weights times V. One copy of each in
// the code (it shares the instruction caches with the other roles).
template <int D>
__device__ __noinline__ void issue_qk(uint32_t s_col, uint32_t q, uint32_t k) {
  constexpr uint32_t kDesc = instr_desc(128, kKeys, false, false);
  if (elect_one()) {
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      const uint32_t off = ((s >> 2) * kPanel + (s & 3) * 32) >> 4;
      mma_ss(s_col, q + off, k + off, kDesc, s > 0);
    }
  }
  __syncwarp();
}
template <int D>
__device__ __noinline__ void issue_pv(uint32_t o_col, uint32_t p_col, uint32_t v, uint32_t acc) {
  constexpr uint32_t kDesc = instr_desc(128, D, true, true);
  if (elect_one()) {
#pragma unroll
    for (int s = 0; s < kKeys / 16; ++s) mma_ts(o_col, p_col + s * 8, v + (s * 16 * 128 >> 4), kDesc, s > 0 ? 1u : acc);
  }
  __syncwarp();
}

template <int D, int B>
__device__ __forceinline__ bool mma_role(const AttnArgs& a, const Place& place, uint32_t base, uint32_t bars) {
  using Cfg = AttnCfg<D, B>;
  // phases of the barriers that pass once per item (QF), per softmax (PR) and per tail of V and stage (VZ)
  int c = 0, nq = 0, np0 = 0, np1 = 0;
  uint32_t nz = 0;
  auto v_ready = [&](const Walk& it, int tile) {
    const int st = c & 1;
    if (!bar_wait(bars + 8 * (kVF + st), (c >> 1) & 1)) return false;
    if ((tile + 1) * kKeys > it.s.len) {
      if (!bar_wait(bars + 8 * (kVZ + st), (nz >> st) & 1)) return false;
      nz ^= 1u << st;
    }
    return true;
  };
  auto p_ready = [&](int qt) {
    int& n = qt ? np1 : np0;
    return bar_wait(bars + 8 * (kPR + qt), n++ & 1);
  };
  auto commit = [&](int bar) {
    if (elect_one()) tc_commit(bars + 8 * bar);
    __syncwarp();
  };
  auto qk = [&](int qt, int to, int st) {  // query tile qt into S pair `to`
    issue_qk<D>(to * kKeys, desc_low(base + Cfg::Q + qt * Cfg::TILE, 16), desc_low(base + Cfg::KT + st * Cfg::TILE, 16));
    commit(kSF + to);
  };
  auto pv = [&](int qt, int st, bool acc) {
    issue_pv<D>(2 * kKeys + qt * D, qt * kKeys, desc_low(base + Cfg::V + st * Cfg::TILE, kPanel), acc);
  };
  for (Walk it(a, place); it.on(); it.next()) {
    const int nt = it.work();
    if (nt == 0) continue;
    for (int qt = 0; qt < 2; ++qt)
      if (!bar_wait(bars + 8 * (kQF + qt), nq & 1)) return false;
    ++nq;
    if (!bar_wait(bars + 8 * (kKF + (c & 1)), (c >> 1) & 1)) return false;
    tc_after();
    const bool two = it.reps() == 0;
    qk(0, 0, c & 1);
    if (two) qk(1, 1, c & 1);
    commit(kKE + (c & 1));
    for (int j = 0; j < nt; ++j, ++c) {
      const int st = c & 1, sn = st ^ 1;
      const bool more = j + 1 < nt;
      if (more && !bar_wait(bars + 8 * (kKF + sn), ((c + 1) >> 1) & 1)) return false;
      if (two) {
        if (!v_ready(it, it.t0 + j)) return false;
        for (int qt = 0; qt < 2; ++qt) {
          if (!p_ready(qt)) return false;
          tc_after();
          pv(qt, st, j > 0);
          if (more)
            qk(qt, qt, sn);
          else
            commit(kSF + qt);  // O is complete
        }
        if (more) commit(kKE + sn);
      } else {
        // S of the next tile goes to the other pair, whose weights were used a tile ago
        if (more) {
          tc_after();
          qk(0, (j + 1) & 1, sn);
          commit(kKE + sn);
        }
        if (!v_ready(it, it.t0 + j)) return false;
        if (!p_ready(j & 1)) return false;
        tc_after();
        pv(j & 1, st, j > 1);
        if (!more) {  // both O are complete
          commit(kSF);
          commit(kSF + 1);
        }
      }
      commit(kVE + st);
    }
  }
  return true;
}

// ---- softmax warps ----------------------------------------------------------
// Rotates rows first .. last - 1 of the item into the query tile (fp16, with
// the softmax scale and log2 e, and where fp16's range asks for it a power of
// two per row, whose exponent goes to `exps`); row r lands at tile row r +
// shift, and `reps` times, `apart` rows apart. D / 32 lanes hold a row, so a
// warp takes 1024 / D rows at a time, `step` rows apart from the next.
template <int D>
__device__ __forceinline__ void rotate_queries(const AttnArgs& a, const Walk& it, unsigned char* qtile, int8_t* exps,
                                               int first, int step, int last, int shift, int reps, int apart, int lane) {
  constexpr int LK = D / 32, N = 32 / LK;
  const int part = lane & (LK - 1);
  const float* sg = a.signs + (it.h % a.table_heads) * D + part * 32;
  const float pre = a.scale * 1.4426950408889634f / sqrtf(static_cast<float>(D));  // logits come in base 2
  uint32_t neg = 0;  // bit e: sign e is negative
#pragma unroll
  for (int e = 0; e < 32; ++e) neg |= (__ldg(sg + e) < 0.0f ? 1u : 0u) << e;
#pragma unroll 1
  for (int r0 = first; r0 < last; r0 += step) {
    const int r = r0 + lane / LK;
    const int rr = it.m * kRows + min(r, last - 1);  // row of the sequence's (token, group head) list
    const int64_t off = (it.s.row0 + rr / a.g) * a.q_row + (it.h * a.g + rr % a.g) * a.q_head + part * 32;
    float v[32];
    if (a.q_bf16) {
      const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(a.q) + off;
      if (a.q_vec) {
#pragma unroll
        for (int e = 0; e < 32; e += 8) {
          const uint4 x = *reinterpret_cast<const uint4*>(p + e);
          v[e] = bf16_lo(x.x); v[e + 1] = bf16_hi(x.x); v[e + 2] = bf16_lo(x.y); v[e + 3] = bf16_hi(x.y);
          v[e + 4] = bf16_lo(x.z); v[e + 5] = bf16_hi(x.z); v[e + 6] = bf16_lo(x.w); v[e + 7] = bf16_hi(x.w);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __bfloat162float(p[e]);
      }
    } else {
      const float* p = static_cast<const float*>(a.q) + off;
      if (a.q_vec) {
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 x = *reinterpret_cast<const float4*>(p + e);
          v[e] = x.x; v[e + 1] = x.y; v[e + 2] = x.z; v[e + 3] = x.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = p[e];
      }
    }
#pragma unroll
    for (int e = 0; e < 32; ++e)
      v[e] = pre * __uint_as_float(__float_as_uint(v[e]) ^ ((neg << (31 - e)) & 0x80000000u));
    fwht32_regs(v);
    fwht32_lanes<LK, 1>(v, lane);
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < 32; ++e) m = fmaxf(m, fabsf(v[e]));
#pragma unroll
    for (int o = 1; o < LK; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // rows whose largest entry lies in [2^-5, 2^14) stay as they are; others are scaled by 2^-ex, 2^ex > m (kept
    // within 2^-125 .. 2^126, so that it is a normal number)
    const int ex = (m >= 0x1p-5f && m < 0x1p14f) || m == 0.0f
                       ? 0 : min(max(static_cast<int>(__float_as_uint(m) >> 23) - 126, -125), 126);
    const float down = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
    if (r < last) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint4 h = make_uint4(half2_bits(v[8 * q] * down, v[8 * q + 1] * down),
                                   half2_bits(v[8 * q + 2] * down, v[8 * q + 3] * down),
                                   half2_bits(v[8 * q + 4] * down, v[8 * q + 5] * down),
                                   half2_bits(v[8 * q + 6] * down, v[8 * q + 7] * down));
        for (int c = 0; c < reps; ++c)
          *reinterpret_cast<uint4*>(qtile + sw128(r + shift + c * apart, part * 4 + q, kPanel)) = h;
      }
      if (part == 0)
        for (int c = 0; c < reps; ++c) exps[r + shift + c * apart] = static_cast<int8_t>(ex);
    }
  }
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// largest magnitude
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float d;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// A row's running state, and the tensor-memory columns of its S (then P) and
// O. Weights are 2^(logit - ref) for a reference that needs only be near
// (bf16 and fp32 keep their precision whatever the exponent): it is set by a
// row's first slots and raised when a logit might pass it by kAsk. So weights
// stay below 2^kAsk, and their products with values finite where a row's
// values sum to less than 2^60 in magnitude. (A smaller kAsk asks for looks at
// the logits that a wide spread of norms does not warrant.)
constexpr float kAsk = 64.0f;
template <int D, bool LSE>  // LSE: lse is asked for
struct Row {
  uint32_t S, O;
  float ref, sum, exact, up;  // exact: the sum before rounding, for lse alone; up: 2^ex of the row's queries

  // Logits less the reference of 32 slots from their raw products: times the norms g.
  __device__ __forceinline__ void logits(float2 (&y)[16], const uint32_t (&s)[32], const float* gm, float shift) const {
    const float2 sh = make_float2(shift, shift);
#pragma unroll
    for (int x = 0; x < 32; x += 4) {
      const float4 g = *reinterpret_cast<const float4*>(gm + x);
      y[x / 2] = fma_f32x2(make_float2(__uint_as_float(s[x]), __uint_as_float(s[x + 1])), make_float2(g.x, g.y), sh);
      y[x / 2 + 1] =
          fma_f32x2(make_float2(__uint_as_float(s[x + 2]), __uint_as_float(s[x + 3])), make_float2(g.z, g.w), sh);
    }
  }
  // the same where the row has a scale of its own or does not see all of them (-inf from slot `left` on)
  __device__ __forceinline__ void logits_any(float2 (&y)[16], uint32_t (&s)[32], const float* gm, int left, float shift) const {
#pragma unroll
    for (int x = 0; x < 32; ++x) s[x] = __float_as_uint(__uint_as_float(s[x]) * up);
    logits(y, s, gm, shift);
    if (left < 32) {
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        if (2 * x >= left) y[x].x = -INFINITY;
        if (2 * x + 1 >= left) y[x].y = -INFINITY;
      }
    }
  }

  // Weights of 32 slots to column c of P, rounded to bf16 (V's type, which the
  // product shares), and their sum. Summed as rounded, so that output rows
  // are averages with the very weights used, and one slot that outweighs the
  // rest costs nothing: error against 64 bits on 512 tokens over 32768 slots
  // 1.84e-3 (1.6e-3 of it the output's rounding), 2.4e-3 with the sum of the
  // unrounded weights, which took 342 us instead of 368. lse, an fp32 value,
  // is formed from the latter.
  __device__ __forceinline__ void weights(const float2 (&y)[16], uint32_t c, float2& total, float2& before) const {
    uint32_t p[16];
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      const float2 e = make_float2(ex2(y[x].x), ex2(y[x].y));
      p[x] = bf16_pair(e.x, e.y);
      if constexpr (LSE) before = add_f32x2(before, e);
    }
    tmem_st16(c, p);
#pragma unroll
    for (int x = 0; x < 16; x += 4) {  // (as a tree: a chain of sums would wait for each)
      const float2 a = add_f32x2(make_float2(bf16_lo(p[x]), bf16_hi(p[x])), make_float2(bf16_lo(p[x + 1]), bf16_hi(p[x + 1])));
      const float2 b = add_f32x2(make_float2(bf16_lo(p[x + 2]), bf16_hi(p[x + 2])), make_float2(bf16_lo(p[x + 3]), bf16_hi(p[x + 3])));
      total = add_f32x2(total, add_f32x2(a, b));
    }
  }

  // A row's reference follows its largest logit of the tile where that passes
  // it by 16 or is its first; O (o_set: it holds tiles) and the sum follow.
  __device__ __forceinline__ void follow(float top, bool o_set) {
    const bool raise = top > ref + 16.0f || (ref == -INFINITY && top > -INFINITY);
    if (!__any_sync(0xffffffffu, raise)) return;
    const float keep = raise ? ex2(ref - top) : 1.0f;
    if (raise) ref = top;
    sum *= keep;
    if constexpr (LSE) exact *= keep;
    if (o_set) {
#pragma unroll 1
      for (int d = 0; d < D; d += 16) {
        uint32_t o[16];
        tmem_ld16(o, O + d);
        tc_wait_ld(o);
#pragma unroll
        for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * keep);
        tmem_st16(O + d, o);
      }
    }
  }

  __device__ __forceinline__ float largest(const float2 (&y)[16], float top) const {
#pragma unroll
    for (int x = 0; x < 16; ++x) top = max3(top, y[x].x, y[x].y);
    return top;
  }

  // The weights of columns [col0, col0 + cols) of a key tile, for any row.
  __device__ __forceinline__ void weigh_any(const float* gm, int col0, int cols, int left, bool o_set) {
    float top = -INFINITY;
    uint32_t s[32];
    float2 y[16];
#pragma unroll 1
    for (int c = col0; c < col0 + cols; c += 32) {
      tmem_ld32(s, S + c);
      tc_wait_ld(s);
      logits_any(y, s, gm + c, left - c, 0.0f);
      top = largest(y, top);
    }
    follow(top, o_set);
    const float shift = ref == -INFINITY ? 0.0f : -ref;
    float2 total = make_float2(0.0f, 0.0f), before = total;
#pragma unroll 1
    for (int c = col0; c < col0 + cols; c += 32) {
      if (cols > 32) {
        tmem_ld32(s, S + c);
        tc_wait_ld(s);
        logits_any(y, s, gm + c, left - c, 0.0f);
      }
#pragma unroll
      for (int x = 0; x < 16; ++x) y[x] = add_f32x2(y[x], make_float2(shift, shift));
      weights(y, S + c / 2, total, before);
    }
    sum += total.x + total.y;
    if constexpr (LSE) exact += before.x + before.y;
  }

  // The weights of a whole key tile that every row of the warp sees, scales
  // all 1. First the largest |product|: times the tile's largest norm it
  // bounds the logits, and hardly ever asks for a look at the logits
  // themselves.
  // (`there`: the lane holds a row. The others' S is left over from any item;
  // neither they nor other rows have a say in what a row does.)
  __device__ __forceinline__ void weigh_full(const float* gm, float gmax, bool there, bool o_set) {
    uint32_t s[32], t[32];
    float top[2] = {0.0f, 0.0f};
#pragma unroll 1
    for (int c = 0; c < kKeys; c += 64) {
      tmem_ld32(s, S + c);
      tmem_ld32(t, S + c + 32);
      tc_wait_ld(s, t);
#pragma unroll
      for (int x = 0; x < 32; x += 2) {
        top[0] = max3_abs(top[0], __uint_as_float(s[x]), __uint_as_float(s[x + 1]));
        top[1] = max3_abs(top[1], __uint_as_float(t[x]), __uint_as_float(t[x + 1]));
      }
    }
    // (a NaN among them, or an infinite norm, fails the comparison)
    const bool ask = there && !(fmaxf(top[0], top[1]) * gmax <= ref + kAsk);
    if (__any_sync(0xffffffffu, ask)) {
      float high = -INFINITY;
      float2 y[16];
#pragma unroll 1
      for (int c = 0; c < kKeys; c += 32) {
        tmem_ld32(s, S + c);
        tc_wait_ld(s);
        logits(y, s, gm + c, 0.0f);
        high = largest(y, high);
      }
      follow(ask ? high : -INFINITY, o_set);
    }
    const float shift = ref == -INFINITY ? 0.0f : -ref;
    float2 u = make_float2(0.0f, 0.0f), before = u;
#pragma unroll 1
    for (int c = 0; c < kKeys; c += 64) {  // P's columns overlay S's from the front: behind those read here
      float2 y[16];
      tmem_ld32(s, S + c);
      tmem_ld32(t, S + c + 32);
      tc_wait_ld(s, t);
      logits(y, s, gm + c, shift);
      weights(y, S + c / 2, u, before);
      logits(y, t, gm + c + 32, shift);
      weights(y, S + c / 2 + 16, u, before);
    }
    sum += u.x + u.y;
    if constexpr (LSE) exact += before.x + before.y;
  }
};

// 32 values of an output row: bf16 or fp32.
__device__ __forceinline__ void store32(const AttnArgs& a, int64_t at, const float (&v)[32]) {
  if (a.out_bf16) {
    uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(a.out) + at);
#pragma unroll
    for (int x = 0; x < 32; x += 8) {
      uint32_t w[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[x + 2 * y], v[x + 2 * y + 1]);
        w[y] = *reinterpret_cast<const uint32_t*>(&b2);
      }
      dst[x / 8] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at);
#pragma unroll
    for (int x = 0; x < 32; x += 4) dst[x / 4] = make_float4(v[x], v[x + 1], v[x + 2], v[x + 3]);
  }
}

template <int D, int B, bool LSE>
__device__ __forceinline__ bool softmax_role(const AttnArgs& a, const Place& place, unsigned char* sm, uint32_t bars,
                                             uint32_t tmem, int qt) {
  using Cfg = AttnCfg<D, B>;
  const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
  int8_t* exps = reinterpret_cast<int8_t*>(sm + Cfg::EXPS);
  const float* gam = reinterpret_cast<const float*>(sm + Cfg::GAM);
  Row<D, LSE> row;
  row.S = tmem + lanes + qt * kKeys;
  row.O = tmem + lanes + 2 * kKeys + qt * D;
  int c = 0;
  uint32_t phase = 0;  // bit 0: of kSF, bit 1: of kMEET
  // All softmax warps meet here. Not at a hardware barrier, which has no limit: a warp whose other waits ran out has left,
  // and those that wait for it have to leave too.
  auto meet = [&] {
    __syncwarp();
    if (lane == 0) bar_arrive(bars + 8 * kMEET);
    phase ^= 2u;
    return bar_wait(bars + 8 * kMEET, (phase >> 1) ^ 1u);
  };
  for (Walk it(a, place); it.on(); it.next()) {
    const int nt = it.work(), rows = it.rows(), reps = it.reps();
    const bool two = reps == 0;
    // this thread's row of the item, and the warp's share of a key tile: columns [col0, col0 + cols)
    const int apart = two ? 128 : 128 / reps;       // rows of a copy
    const int r0 = two ? qt * 128 + warp * 32 : warp * 32 % apart, x = r0 + lane;
    const int cols = two ? kKeys : kKeys / reps, col0 = two ? 0 : warp * 32 / apart * cols;
    const int wr = min(32, max(0, rows - r0));      // rows of the warp
    const bool there = lane < wr;
    const int rr = it.m * kRows + x;
    int limit = 0;
    if (there) limit = a.causal ? max(0, it.s.len - it.s.fresh + rr / a.g + 1) : it.s.len;
    row.ref = -INFINITY;
    row.sum = 0.0f;
    row.exact = 0.0f;
    if (nt > 0) {
      if (two) {
        rotate_queries<D>(a, it, sm + Cfg::Q + qt * Cfg::TILE, exps + qt * 128, r0, 1024 / D, r0 + wr, -qt * 128, 1, 0, lane);
        __syncwarp();
      } else {
        rotate_queries<D>(a, it, sm + Cfg::Q, exps, (qt * 4 + warp) * (1024 / D), 8 * (1024 / D), rows, 0, reps, apart, lane);
        if (!meet()) return false;
      }
      fence_async_shared();
      bar_arrive(bars + 8 * (kQF + qt));
      const int ex = there ? exps[(two ? qt * 128 : 0) + warp * 32 + lane] : 0;
      row.up = ldexpf(1.0f, ex);
      const bool plain = __all_sync(0xffffffffu, ex == 0);
      for (int j = two ? 0 : qt; j < nt; j += two ? 1 : 2) {
        if (!bar_wait(bars + 8 * (kSF + qt), phase & 1)) return false;
        phase ^= 1u;
        tc_after();
        if (wr > 0) {  // a warp without rows leaves its part of P as it is: those rows go nowhere
          const float* gm = gam + ((c + j) % Cfg::GS) * kKeys;
          const int left = limit - (it.t0 + j) * kKeys;  // slots of the tile that the row sees
          const bool masked = __any_sync(0xffffffffu, there && left < kKeys);
          const bool o_set = two ? j > 0 : j > 1;
          if (cols == kKeys && plain && !masked) {
            const float4 g4 = *reinterpret_cast<const float4*>(sm + Cfg::GMAX + ((c + j) % Cfg::GS) * 16);
            row.weigh_full(gm, max3(g4.x, g4.y, fmaxf(g4.z, g4.w)), there, o_set);
          } else {
            row.weigh_any(gm, col0, cols, left, o_set);
          }
          if (cols < kKeys) {
            uint32_t zero[16];
#pragma unroll
            for (int y = 0; y < 16; ++y) zero[y] = 0u;
#pragma unroll 1
            for (int k = 0; k < kKeys; k += 32)
              if (k < col0 || k >= col0 + cols) tmem_st16(row.S + k / 2, zero);
          }
          tc_wait_st();
        }
        tc_before();
        bar_arrive(bars + 8 * (kPR + qt));
      }
      if (!bar_wait(bars + 8 * (kSF + qt), phase & 1)) return false;  // O is complete
      phase ^= 1u;
      tc_after();
    }
    c += nt;
    // ---- results of the item (or of this piece of it)
    const bool whole = it.t0 == 0 && it.t1 == it.tiles;
    if (!whole && it.t0 == 0 && (threadIdx.x & 255) == 0) {
      // the item's last tile lies with the last CTA whose piece starts at or before it
      const int64_t last = place.start + (place.count - it.left) + it.tiles - 1;
      const int64_t ctas = min(static_cast<int64_t>(gridDim.x), place.total);
      const int to = static_cast<int>(((last + 1) * ctas + place.total - 1) / place.total - 1);
      a.shared[blockIdx.x] = Shared{to - static_cast<int>(blockIdx.x) + 1, rows, two ? 1 : 2 * reps, it.s.row0, it.h, it.m, {0, 0}};
    }
    const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (it.t0 > 0 ? 0 : 1);
    const int64_t row_at = static_cast<int64_t>(it.s.row0) * a.Hq + static_cast<int64_t>(it.h) * a.g;
    auto out_row = [&](int y) {  // row y of the item in out and lse
      const int q = it.m * kRows + y;
      return row_at + static_cast<int64_t>(q / a.g) * a.Hq + q % a.g;
    };
    if (!whole) {
      // rows, or row copies, for the join
      if (there) a.part_ml[slot * 256 + qt * 128 + warp * 32 + lane] = make_float2(row.ref, row.sum);
      if (LSE && there) a.part_e[slot * 256 + qt * 128 + warp * 32 + lane] = row.exact;
      if (wr > 0) {
        float4* dst = a.part_o + slot * (D / 4) * 256 + qt * 128 + warp * 32 + lane;
#pragma unroll 1
        for (int k = 0; k < D; k += 16) {
          uint32_t o[16];
          tmem_ld16(o, row.O + k);
          tc_wait_ld(o);
          if (there) {
#pragma unroll
            for (int y = 0; y < 4; ++y)  // (a row without a slot here may find anything in O)
              dst[(k / 4 + y) * 256] = row.sum == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                                                       : make_float4(__uint_as_float(o[4 * y]), __uint_as_float(o[4 * y + 1]),
                                                                     __uint_as_float(o[4 * y + 2]), __uint_as_float(o[4 * y + 3]));
          }
        }
      }
    } else if (two || nt == 0) {
      if (wr > 0 && (two || qt == 0) && (two || warp * 32 < apart)) {
        const float sum = row.sum, inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        const int64_t orow = out_row(x);
        if (LSE && there) a.lse[orow] = sum == 0.0f ? -INFINITY : (row.ref + log2f(row.exact)) * 0.6931471805599453f;
#pragma unroll 1
        for (int k = 0; k < D; k += 32) {
          uint32_t o[32];
          float v[32];
          if (nt > 0) {
            tmem_ld32(o, row.O + k);
            tc_wait_ld(o);
          }
          // a row that saw nothing gives 0
#pragma unroll
          for (int y = 0; y < 32; ++y) v[y] = nt == 0 || sum == 0.0f ? 0.0f : __uint_as_float(o[y]) * inv;
          if (there) store32(a, orow * D + k, v);
        }
      }
    } else {
      // the copies of each row: references and sums through shared memory (the second query tile is free), O scaled
      // to the common reference through this CTA's rows in the workspace, summed in a fixed order
      float2* ml = reinterpret_cast<float2*>(sm + Cfg::Q + Cfg::TILE);  // [2][128] of the copies, then [128] of the rows
      float* before = reinterpret_cast<float*>(ml + 384);                   // their sums before rounding
      const int me = qt * 128 + warp * 32 + lane;
      ml[me] = there ? make_float2(row.ref, row.sum) : make_float2(-INFINITY, 0.0f);
      if constexpr (LSE) before[me] = there ? row.exact : 0.0f;
      if (!meet()) return false;
      float top = -INFINITY, all = 0.0f, exact = 0.0f;
      for (int k = 0; k < 2 * reps; ++k) top = fmaxf(top, ml[(k & 1) * 128 + (k >> 1) * apart + x].x);
      const float base = top == -INFINITY ? 0.0f : top;
      for (int k = 0; k < 2 * reps; ++k) {
        const float2 y = ml[(k & 1) * 128 + (k >> 1) * apart + x];
        const float w = ex2(y.x - base);
        all = fmaf(w, y.y, all);
        if constexpr (LSE) exact = fmaf(w, before[(k & 1) * 128 + (k >> 1) * apart + x], exact);
      }
      if (qt == 0 && warp * 32 < apart) {
        ml[256 + x] = make_float2(top, all);
        if constexpr (LSE) before[256 + x] = exact;
      }
      float4* mine = a.copies + static_cast<int64_t>(blockIdx.x) * (D / 4) * 256;
      if (wr > 0) {
        const float keep = row.sum == 0.0f ? 0.0f : ex2(row.ref - base);
#pragma unroll 1
        for (int k = 0; k < D; k += 16) {
          uint32_t o[16];
          tmem_ld16(o, row.O + k);
          tc_wait_ld(o);
          if (there) {
#pragma unroll
            for (int y = 0; y < 4; ++y)  // a copy without a slot may hold anything
              mine[(k / 4 + y) * 256 + me] =
                  row.sum == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                                  : make_float4(__uint_as_float(o[4 * y]) * keep, __uint_as_float(o[4 * y + 1]) * keep,
                                                __uint_as_float(o[4 * y + 2]) * keep, __uint_as_float(o[4 * y + 3]) * keep);
          }
        }
      }
      if (!meet()) return false;
      // threads along four rows, so that reads and writes both meet in sectors
      const int tid = threadIdx.x & 255, y0 = tid & 3;
      for (int e = tid >> 2; e < (rows + 3) / 4 * (D / 4); e += 64) {
        const int y = e / (D / 4) * 4 + y0, d = e % (D / 4);
        if (y >= rows) continue;
        const float2 t = ml[256 + y];
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const float4* src = mine + d * 256 + y;
#pragma unroll 2
        for (int k = 0; k < 2 * reps; ++k) {
          const float4 v = src[(k & 1) * 128 + (k >> 1) * apart];
          o.x += v.x; o.y += v.y; o.z += v.z; o.w += v.w;
        }
        const int64_t orow = out_row(y);
        const float inv = t.y == 0.0f ? 0.0f : 1.0f / t.y;
        if (a.out_bf16)
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + orow * D + 4 * d) =
              make_uint2(bf16_pair(o.x * inv, o.y * inv), bf16_pair(o.z * inv, o.w * inv));
        else
          *reinterpret_cast<float4*>(static_cast<float*>(a.out) + orow * D + 4 * d) =
              make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        if (LSE && d == 0) a.lse[orow] = t.y == 0.0f ? -INFINITY : (t.x + log2f(before[256 + y])) * 0.6931471805599453f;
      }
      if (!meet()) return false;
    }
    tc_before();
  }
  return true;
}

template <int D, int B, bool LSE>
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
  if (tid == 0) {
    for (int q = 0; q < 2; ++q) {
      bar_init(bars + 8 * (kQF + q), 128);
      bar_init(bars + 8 * (kSF + q), 1);
      bar_init(bars + 8 * (kPR + q), 128);
      bar_init(bars + 8 * (kKF + q), 128);
      bar_init(bars + 8 * (kKE + q), 1);
      bar_init(bars + 8 * (kVF + q), 1);
      bar_init(bars + 8 * (kVE + q), 1);
      bar_init(bars + 8 * (kVZ + q), 32);
    }
    bar_init(bars + 8 * kEND, 1);
    bar_init(bars + 8 * kMEET, 8);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 12) tmem_alloc(s32(&s_tmem), 512);
  if (tid == 32) a.shared[blockIdx.x].pieces = 0;
  __syncthreads();
  if (warp == 15) {
    const int64_t total = total_tiles(a, lane, blockIdx.x == 0);
    const Place p = find_place(a, lane, total);
    if (lane == 0) s_place = p;
  } else {
    // decoded codes (b = 4: directions) in fp16, and their copies
    for (int e = tid; e < Cfg::NE; e += 480) {
      const int field = Cfg::QUAD ? e & ((1 << 2 * B) - 1) : e & (K::NDIR - 1);
      const float3 d = field_direction<B>(field, s_dir);
      const float r = Cfg::QUAD ? 1.0f : s_rho[(e >> K::DIR) & (K::NRHO - 1)];
      const uint2 v = make_uint2(half2_bits(d.x * r, d.y * r), half2_bits(d.z * r, d.z * r));
#pragma unroll
      for (int k = 0; k < Cfg::REP; ++k)
        *reinterpret_cast<uint2*>(sm + Cfg::TAB + (e << Cfg::SH) + k * 8) = v;
    }
    if (Cfg::QUAD && tid < 64)
      *reinterpret_cast<uint32_t*>(sm + Cfg::RHO + tid * 4) = half2_bits(s_rho[tid >> 3], s_rho[tid >> 3]);
  }
  tc_before();
  __syncthreads();
  tc_after();
  const Place place = s_place;
  constexpr uint32_t tmem = 0;  // the allocation is the whole tensor memory, so it starts at column 0
  bool ok = true;
  if (place.count > 0) {
    if (warp < 8) {
      ok = softmax_role<D, B, LSE>(a, place, sm, bars, tmem, warp >> 2);
    } else if (warp < 12) {
      ok = decode_role<D, B>(a, place, sm, base, bars);
    } else {
      if (warp == 12) {
        ok = mma_role<D, B>(a, place, base, bars);
        // products in flight end before tensor memory is given back
        if (!ok) {
          if (elect_one()) tc_commit(bars + 8 * kEND);
          __syncwarp();
          bar_wait(bars + 8 * kEND, 0);
        }
      } else if (warp == 13) {
        int issued = 0;
        ok = v_role<D, B>(a, place, &vmap, sm, base, bars, issued);
        // copies in flight end before the CTA does
        for (int c = max(0, issued - 2); c < issued; ++c) bar_wait(bars + 8 * (kVF + (c & 1)), (c >> 1) & 1);
      }
    }
  }
  if (!ok && lane == 0) report(a.t.status, OCTO_PAGED_TIMEOUT);
  tc_before();
  __syncthreads();
  if (warp == 12) tmem_free(s_tmem, 512);
}

// ---- joining the pieces of shared items --------------------------------------
// One block per (CTA that begins an item others go on with, 4 rows of it). A
// row's entries are its copies in each piece.
template <int D>
__global__ void __launch_bounds__(256) paged_attn_join(const __grid_constant__ AttnArgs a) {
  constexpr int R = kJoinRows, TPR = D / 4, G = 256 / (R * TPR);  // rows; threads per row; groups that share the entries
  const int c0 = blockIdx.x, r0 = blockIdx.y * R, tid = threadIdx.x;
  const Shared it = a.shared[c0];
  const int n = it.pieces * it.copies, nr = min(R, it.rows - r0);
  if (n == 0 || nr <= 0) return;
  __shared__ float2 s_ml[kJoin * 8][R];
  __shared__ float s_red[8][R], s_red_e[8][R], s_ref[R], s_sum[R], s_exact[R];
  __shared__ __align__(16) float s_out[G][R][D];
  const int lc = 31 - __clz(it.copies), apart = it.copies > 1 ? 256 / it.copies : 0;
  // entry e: copy c of piece k; CTA c0's piece lies in its second slot, those that go on with it use their first
  auto slot = [&](int e) { return static_cast<int64_t>(e >> lc == 0 ? 2 * c0 + 1 : 2 * (c0 + (e >> lc))); };
  auto row = [&](int e) {
    const int c = e & (it.copies - 1);
    return (c & 1) * 128 + (c >> 1) * apart + r0;
  };
  const int r = tid & (R - 1);
  float top = -INFINITY;
  if (r < nr)
    for (int e = tid / R; e < n; e += 256 / R) {
      const float2 ml = __ldcg(a.part_ml + slot(e) * 256 + row(e) + r);
      s_ml[e][r] = ml;
      top = fmaxf(top, ml.x);
    }
#pragma unroll
  for (int o = R; o < 32; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((tid & 31) < R) s_red[tid >> 5][r] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < 8; ++w) top = fmaxf(top, s_red[w][r]);
  const float base = top == -INFINITY ? 0.0f : top;
  float sum = 0.0f, exact = 0.0f;
  if (r < nr)
    for (int e = tid / R; e < n; e += 256 / R) {  // its own entries
      const float w = ex2(s_ml[e][r].x - base);
      sum = fmaf(w, s_ml[e][r].y, sum);
      if (a.lse) exact = fmaf(w, __ldcg(a.part_e + slot(e) * 256 + row(e) + r), exact);
      s_ml[e][r].x = w;
    }
#pragma unroll
  for (int o = R; o < 32; o <<= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, o);
    exact += __shfl_xor_sync(0xffffffffu, exact, o);
  }
  __syncthreads();
  if ((tid & 31) < R) {
    s_red[tid >> 5][r] = sum;
    s_red_e[tid >> 5][r] = exact;
  }
  __syncthreads();
  if (tid < R) {
    float all = 0.0f, before = 0.0f;
    for (int w = 0; w < 8; ++w) {
      all += s_red[w][r];
      before += s_red_e[w][r];
    }
    s_sum[r] = all;
    s_exact[r] = before;
    s_ref[r] = top;
  }
  const int d = tid / R % TPR, g = tid / (R * TPR);
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (r < nr) {
#pragma unroll 8
    for (int e = g; e < n; e += G) {
      const float4 v = __ldcg(a.part_o + (slot(e) * (D / 4) + d) * 256 + row(e) + r);
      const float w = s_ml[e][r].x;
      o.x = fmaf(w, v.x, o.x);
      o.y = fmaf(w, v.y, o.y);
      o.z = fmaf(w, v.z, o.z);
      o.w = fmaf(w, v.w, o.w);
    }
  }
  *reinterpret_cast<float4*>(&s_out[g][r][4 * d]) = o;
  __syncthreads();
  for (int e = tid; e < nr * TPR; e += 256) {
    const int q = e / TPR, x = e % TPR * 4;
    float4 v = *reinterpret_cast<const float4*>(&s_out[0][q][x]);
#pragma unroll
    for (int k = 1; k < G; ++k) {
      const float4 u = *reinterpret_cast<const float4*>(&s_out[k][q][x]);
      v.x += u.x; v.y += u.y; v.z += u.z; v.w += u.w;
    }
    const float all = s_sum[q], inv = all == 0.0f ? 0.0f : 1.0f / all;
    const int rr = it.m * kRows + r0 + q, tok = rr / a.g;
    const int64_t orow = static_cast<int64_t>(it.row0 + tok) * a.Hq + it.h * a.g + (rr - tok * a.g);
    if (a.out_bf16)
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + orow * D + x) =
          make_uint2(bf16_pair(v.x * inv, v.y * inv), bf16_pair(v.z * inv, v.w * inv));
    else
      *reinterpret_cast<float4*>(static_cast<float*>(a.out) + orow * D + x) =
          make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
    if (a.lse && x == 0) a.lse[orow] = all == 0.0f ? -INFINITY : (s_ref[q] + log2f(s_exact[q])) * 0.6931471805599453f;
  }
}

// ---- host -------------------------------------------------------------------
static int attn_ctas() { return std::min(sm_count(), kJoin); }

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

template <int D, int B, bool LSE>
static cudaError_t launch_attn(const AttnArgs& a, const CUtensorMap& map, int ctas, cudaStream_t st) {
  static LaunchCache cache;
  int resident = 0;
  cudaError_t e = launch_setup(paged_attn_kernel<D, B, LSE>, cache, 512, AttnCfg<D, B>::SMEM, resident);
  if (e != cudaSuccess) return e;
  paged_attn_kernel<D, B, LSE><<<ctas, 512, AttnCfg<D, B>::SMEM, st>>>(a, map);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  const unsigned groups = static_cast<unsigned>((std::min<int64_t>(a.n_rows * a.g, kRows) + kJoinRows - 1) / kJoinRows);
  paged_attn_join<D><<<dim3(ctas, groups), 256, 0, st>>>(a);
  return cudaGetLastError();
}
template <int D, int B>
static cudaError_t launch_lse(const AttnArgs& a, const CUtensorMap& map, int ctas, cudaStream_t st) {
  return a.lse ? launch_attn<D, B, true>(a, map, ctas, st) : launch_attn<D, B, false>(a, map, ctas, st);
}

}  // namespace paged
}  // namespace octo

extern "C" size_t octo_paged_attn_workspace(const octo_layout* L, int64_t n_rows, int n_seqs, int Hq, int Hkv) {
  using namespace octo::paged;
  if (check_layout(L) != OCTO_OK || L->d > 128 || n_rows < 0 || n_seqs < 0 || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0)
    return 0;
  // two partial slots and the row copies of each CTA, whatever the sizes
  return kDecodeFront + attn_ctas() * (3 * 256 * L->d * sizeof(float) + 2 * 256 * (sizeof(float2) + sizeof(float)) + sizeof(Shared));
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
  const int ctas = attn_ctas();
  a.part_o = reinterpret_cast<float4*>(static_cast<unsigned char*>(workspace) + kDecodeFront);
  a.copies = a.part_o + static_cast<size_t>(2) * ctas * (L->d / 4) * 256;
  a.part_ml = reinterpret_cast<float2*>(a.copies + static_cast<size_t>(ctas) * (L->d / 4) * 256);
  a.part_e = reinterpret_cast<float*>(a.part_ml + static_cast<size_t>(2) * ctas * 256);
  a.shared = reinterpret_cast<Shared*>(a.part_e + static_cast<size_t>(2) * ctas * 256);
  const int qe = q_dtype == OCTO_BF16 ? 2 : 4;
  a.q_vec = reinterpret_cast<uintptr_t>(q) % 16 == 0 && q_row_stride * qe % 16 == 0 && q_head_stride * qe % 16 == 0;
  // V comes in boxes that lie inside one page: the largest power of two (8-row swizzle groups) that divides it
  a.box = 16;
  while (a.box < kKeys && pages->page_size % (2 * a.box) == 0) a.box *= 2;
  CUtensorMap map;
  if (!encode_v_map(&map, pages, L->d, a.box)) return OCTO_ECUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (L->d == 64)
    e = L->b == 2 ? launch_lse<64, 2>(a, map, ctas, st) : L->b == 3 ? launch_lse<64, 3>(a, map, ctas, st) : launch_lse<64, 4>(a, map, ctas, st);
  else
    e = L->b == 2 ? launch_lse<128, 2>(a, map, ctas, st) : L->b == 3 ? launch_lse<128, 3>(a, map, ctas, st) : launch_lse<128, 4>(a, map, ctas, st);
  return e == cudaSuccess ? OCTO_OK : OCTO_ECUDA;
}
