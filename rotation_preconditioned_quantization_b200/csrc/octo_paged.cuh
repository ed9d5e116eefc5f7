// Shared by the paged-cache kernels: the page table as the device sees it,
// bounded mbarrier waits, tcgen05 / TMA wrappers, and the code table that
// turns a triplet code into fp16 coordinates of the rotated direction.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/octopus.h"
#include "octo_common.cuh"

namespace octo {
namespace paged {

// ---- host: argument checks shared by the paged entry points -----------------
// The paged set: the OCTOPUS split (b + 1, b - 1) without the sketch.
inline int check_layout(const octo_layout* L) {
  if (!L) return OCTO_EINVAL;
  if (L->d != 64 && L->d != 128 && L->d != 256) return OCTO_EUNSUPPORTED;
  if (L->b < 2 || L->b > 4 || L->b_dir != L->b + 1 || L->qjl != 0) return OCTO_EUNSUPPORTED;
  octo_layout chk;
  if (octo_layout_init(&chk, L->d, L->b, 0, L->rounding) != OCTO_OK) return OCTO_EINVAL;
  if (chk.words != L->words || chk.T != L->T || chk.code_bits != L->code_bits || chk.b_rho != L->b_rho)
    return OCTO_EINVAL;
  return OCTO_OK;
}

inline int check_pages(const octo_pages* p) {
  if (!p || !p->packed || !p->gamma) return OCTO_EINVAL;
  if (p->n_pages < 1 || p->n_heads < 1 || p->page_size < 16 || p->page_size % 16 != 0) return OCTO_EINVAL;
  if (p->n_pages > INT32_MAX) return OCTO_EINVAL;  // page ids are 32-bit
  // the tensor map of V counts (page, head) rows in 32 bits
  if (p->n_pages * p->n_heads > INT32_MAX) return OCTO_EUNSUPPORTED;
  if (reinterpret_cast<uintptr_t>(p->V) % 16 != 0) return OCTO_EINVAL;
  return OCTO_OK;
}

inline int check_table(const octo_page_table* t, int page_size) {
  if (!t || t->n_seqs < 0 || t->max_pages < 0 || t->stride < t->max_pages) return OCTO_EINVAL;
  if (t->n_seqs > 0 && t->max_pages > 0 && !t->pages) return OCTO_EINVAL;
  // slots are 32-bit, also rounded up to the tiles and clusters that share them (eviction: 4096 slots)
  if (static_cast<int64_t>(t->max_pages) * page_size > INT32_MAX - 65536) return OCTO_EUNSUPPORTED;
  return OCTO_OK;
}

// SMs of the current device.
inline int sm_count() {
  static std::atomic<int> known[kLaunchCacheDevices];
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  const bool cached = dev >= 0 && dev < kLaunchCacheDevices;
  if (cached && (sms = known[dev].load(std::memory_order_relaxed)) > 0) return sms;
  if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 148;
  if (cached) known[dev].store(sms, std::memory_order_relaxed);
  return sms;
}

// The paged calls' scratch starts behind what octo_decode_attn keeps at the
// front of a workspace from one call to the next: a status word, and at byte
// 256 an arrival counter per cache head, at most 65535.
constexpr size_t kDecodeFront = 256 + 4 * 65536;

// ---- device: the table ------------------------------------------------------
struct Table {
  const int32_t* pages;
  int64_t stride;
  int32_t n_seqs, max_pages, page_size, n_heads;
  int32_t page_shift;  // log2 page_size where that is a power of two, else -1
  int64_t n_pages;
  int32_t* status;
};

inline Table make_table(const octo_pages* p, const octo_page_table* t) {
  int shift = 0;
  while ((p->page_size >> shift) > 1) ++shift;
  if ((1 << shift) != p->page_size) shift = -1;
  return Table{t->pages, t->stride, t->n_seqs, t->max_pages, p->page_size, p->n_heads, shift, p->n_pages, p->status};
}

__device__ __forceinline__ void report(int32_t* status, int bits) {
  if (status) atomicOr(status, bits);
}

// Table index and offset of a slot (an integer division only for page sizes
// that are no power of two).
__device__ __forceinline__ int page_index(const Table& t, int s) {
  return t.page_shift >= 0 ? s >> t.page_shift : s / t.page_size;
}
__device__ __forceinline__ int page_offset(const Table& t, int s) {
  return t.page_shift >= 0 ? s & (t.page_size - 1) : s % t.page_size;
}
// A page id read from the table, or -1 (reported) when it is outside the pool.
__device__ __forceinline__ int page_checked(const Table& t, int id) {
  if (id >= 0 && id < t.n_pages) return id;
  report(t.status, OCTO_PAGED_BAD_PAGE);
  return -1;
}
__device__ __forceinline__ const int32_t* page_entry(const Table& t, int i, int s) {
  return t.pages + static_cast<int64_t>(i) * t.stride + page_index(t, s);
}
// Page of slot s of sequence i, or -1 (reported). s must be below max_pages * page_size.
__device__ __forceinline__ int page_of(const Table& t, int i, int s) { return page_checked(t, __ldg(page_entry(t, i, s))); }

// Rows of the chunk and cache length of one sequence, clamped to what the
// tables hold.
struct Seq {
  int row0, fresh, len;
};
__device__ __forceinline__ Seq seq_of(const Table& t, const int32_t* seq_lens, const int32_t* cu, int64_t n_rows,
                                      int i, bool tell = false) {
  const int a = __ldg(cu + i), z = __ldg(cu + i + 1), n = __ldg(seq_lens + i);
  const int rows = static_cast<int>(n_rows), cap = t.max_pages * t.page_size;
  Seq s;
  s.row0 = min(max(a, 0), rows);
  s.fresh = min(max(z, s.row0), rows) - s.row0;
  s.len = min(max(n, 0), cap);
  if (tell && (s.row0 != a || s.fresh != z - a || s.len != n)) report(t.status, OCTO_PAGED_BAD_LENGTH);
  return s;
}

// Sums over the lanes up to this one.
__device__ __forceinline__ int64_t warp_scan(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// A load that starts here: the compiler neither moves it to its use nor the
// use to it.
__device__ __forceinline__ uint32_t load_now(const void* p) {
  uint32_t v;
  asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

// ---- mbarriers --------------------------------------------------------------
__device__ __forceinline__ uint32_t s32(const void* p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint32_t bar_poll(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok;
}
// Waits for the phase of this parity, a whole warp; false when it did not end
// within the limit (about a second of polls), and then the caller gives up.
// All lanes get one answer: lanes that went on without the others would wait
// for them at the warp's next collective instruction, which has no limit. So
// lanes that ran out poll once more: if another lane of the warp saw the phase
// end, they see it now (it stays ended until this warp arrives somewhere
// again), and else they are the whole warp and agree.
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
#pragma unroll 1
  for (int it = 0; it < (1 << 22); ++it)
    if (bar_poll(bar, parity)) return true;
  return __any_sync(__activemask(), bar_poll(bar, parity));
}
__device__ __forceinline__ void fence_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// ---- TMA --------------------------------------------------------------------
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void bulk_in(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
               "r"(bytes), "r"(bar)
               : "memory");
}

// ---- tcgen05 ----------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
// Loads from tensor memory are complete, those into r among them. The values
// are made new behind the wait: nothing else keeps the compiler from using
// the registers before it.
template <int N>
__device__ __forceinline__ void landed(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
template <int N>
__device__ __forceinline__ void tc_wait_ld(uint32_t (&r)[N]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
  landed(r);
}
template <int N>
__device__ __forceinline__ void tc_wait_ld(uint32_t (&r)[N], uint32_t (&q)[N]) {
  tc_wait_ld(r);
  landed(q);
}
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory matrix descriptors with the 128-byte swizzle, as two words:
// the high word is the same for all (groups of 8 rows 1024 bytes apart); the
// low word is the address and, for an MN-major operand (rows along K), the
// `lead` bytes between its 64-element column panels.
constexpr uint32_t kDescHigh = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lead) { return (addr >> 4) | ((lead >> 4) << 16); }

// One product of kind f16, D (fp32, tensor memory) (+)= A * B, by one thread.
// The issue rate of that thread bounds short products, so the descriptors are
// sums of a uniform word and a constant. A in shared memory, or in tensor memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.u32 p, %5, 0;\n mov.b64 x, {%1, %4};\n mov.b64 y, {%2, %4};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "n"(kDescHigh), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.u32 p, %5, 0;\n mov.b64 y, {%2, %4};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "n"(kDescHigh), "r"(acc)
      : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
// Instruction descriptor, kind f16, fp32 accumulator. bf16: both operands
// bf16 (else fp16); bmn: B is MN-major.
__host__ __device__ constexpr uint32_t instr_desc(int m, int n, bool bf16, bool bmn) {
  return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (bmn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

#define OCTO_R8(r, o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), "=r"(r[o + 6]), "=r"(r[o + 7])
#define OCTO_I8(r, o) "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), "r"(r[o + 5]), "r"(r[o + 6]), "r"(r[o + 7])
// 32 consecutive columns of this thread's lane
__device__ __forceinline__ void tmem_ld32(uint32_t (&r)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : OCTO_R8(r, 0), OCTO_R8(r, 8), OCTO_R8(r, 16), OCTO_R8(r, 24)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(addr),
      OCTO_I8(r, 0), OCTO_I8(r, 8), OCTO_I8(r, 16), OCTO_I8(r, 24)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t (&r)[16], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : OCTO_R8(r, 0), OCTO_R8(r, 8)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16};" ::"r"(addr),
      OCTO_I8(r, 0), OCTO_I8(r, 8)
      : "memory");
}
#undef OCTO_R8
#undef OCTO_I8

// 2^x, PTX ex2.approx (relative error about 2^-22; 2^-inf = 0)
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Byte of 16-byte chunk c (8 halves) of row r in a K-major tile of 64-half
// panels with the 128-byte swizzle; `panel` bytes between panels.
__device__ __forceinline__ uint32_t sw128(int r, int c, int panel) {
  return static_cast<uint32_t>((c >> 3) * panel + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// ---- triplet codes ----------------------------------------------------------
template <int D, int B>
struct Code {
  static constexpr int T = (D + 2) / 3, C = 3 * B + 1, W = (T * C + 31) / 32;
  static constexpr int DIR = 2 * (B + 1);          // direction bits of a code, the low ones
  static constexpr int NDIR = 1 << DIR, NRHO = 1 << (B - 1);
};

// Decoded unit direction of a direction field (the codebook cells' inverse
// octahedral map) in fp32.
template <int B>
__device__ __forceinline__ float3 field_direction(uint32_t f, const float* dir_c) {
  int ix, iy;
  direction_cells<B>(f, ix, iy);
  return oct_inverse(dir_c[ix], dir_c[iy]);
}

// (lo half of a | lo half of b << 16) and (hi half of a | lo half of b << 16)
__device__ __forceinline__ uint32_t lolo(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
__device__ __forceinline__ uint32_t hilo(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5432); }

__device__ __forceinline__ uint32_t half2_bits(float x, float y) {
  const __half2 h = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Code i (0..7) of a key's stream as code << SH (the byte offset of a table
// entry of 1 << SH bytes).
template <int C, int SH, int W>
__device__ __forceinline__ uint32_t code_at(const uint32_t (&w)[W], int i) {
  constexpr uint32_t mask = ((1u << C) - 1u) << SH;
  const int p = i * C - SH;
  if (p < 0) return (w[0] << -p) & mask;
  const int q = p >> 5, s = p & 31;
  if (s + C + SH <= 32 || q + 1 >= W) return (w[q] >> s) & mask;
  return __funnelshift_r(w[q], w[q + 1], s) & mask;
}
// The stream 8 codes on. Decode loops take 8 triplets at a time and shift,
// rather than unroll over the key: unrolled, the roles' code did not fit the
// instruction caches together, and a third of the warps' time went to fetches.
template <int C, int W>
__device__ __forceinline__ void next_codes(uint32_t (&w)[W]) {
  constexpr int q = 8 * C / 32, s = 8 * C % 32;
#pragma unroll
  for (int k = 0; k < W; ++k) {
    const uint32_t lo = k + q < W ? w[k + q] : 0u, hi = k + q + 1 < W ? w[k + q + 1] : 0u;
    w[k] = s == 0 ? lo : __funnelshift_r(lo, hi, s);
  }
}

}  // namespace paged
}  // namespace octo
