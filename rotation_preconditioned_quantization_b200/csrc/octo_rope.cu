// Rotary positions with up to four axes on queries and keys, the step before
// the encoder. A pair (a, b) of frequency i at token t becomes
//   (a cos w - b sin w, b cos w + a sin w),  w = pos[axis(i)][t] * f_i,
// and the inverse uses -w (the transpose, so also the gradient).
//
// Angles: f_i is held in 2^-64 turns per position, and pos * f_i is formed
// mod 2^64 in integers, so whole turns drop out exactly and the fraction is
// right to 2^-32 of a turn at every 32-bit position (an fp32 product would be
// off by 0.06 rad at a million). Its fp32 value, of which the cosine and sine
// are taken, is off by at most 2^-26 of a turn.
//
// Bound by memory: each block takes a few tokens, forms their cosines and
// sines once in shared memory (they serve every head of both tensors), then
// its threads turn 16-byte pieces. Rows whose addresses or section sizes do
// not allow 16-byte pieces take the same path element by element. 16384 tokens
// of 16 + 16 heads (d = 64, bf16, 134 MB) take 26 us: 5.1 TB/s.

#include <cmath>

#include <algorithm>

#include "octo_paged.cuh"

namespace octo {
namespace {

struct RopeTensor {
  const void* x;
  void* y;
  int64_t xt, xh, yt, yh;
};
struct RopeArgs {
  RopeTensor a, b;
  int heads0, heads;  // of the first tensor; of both
  int64_t n_tokens;
  int d, F;
  const int32_t* pos;
  int64_t pos_stride;
  int ends[4];  // frequencies of axis k are below ends[k]
  const uint64_t* freqs;
  int inverse, tok;  // tok: tokens per block
};

template <typename T>
__device__ __forceinline__ float up(T v) {
  if constexpr (sizeof(T) == 2)
    return __bfloat162float(v);
  else
    return v;
}
template <typename T>
__device__ __forceinline__ T down(float v) {
  if constexpr (sizeof(T) == 2)
    return __float2bfloat16_rn(v);
  else
    return v;
}

// VEC: frequencies per piece. Half-split: VEC elements of each half (one
// 16-byte access each for VEC = 16 / sizeof(T)); interleaved: VEC pairs.
template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(256) rope_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ float2 cs[];  // [tok][F]
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tok;
  const int nt = static_cast<int>(min(static_cast<int64_t>(a.tok), a.n_tokens - t0));
  for (int k = threadIdx.x; k < nt * a.F; k += 256) {
    const int t = k / a.F, i = k - t * a.F;
    const int axis = (i >= a.ends[0]) + (i >= a.ends[1]) + (i >= a.ends[2]);
    const int64_t pos = a.pos[axis * a.pos_stride + t0 + t];
    const uint64_t turn = static_cast<uint64_t>(pos) * a.freqs[i];
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &s, &c);
    cs[k] = make_float2(c, a.inverse ? -s : s);
  }
  __syncthreads();
  const int pieces = a.F / VEC, rest = (a.d - 2 * a.F + 2 * VEC - 1) / (2 * VEC);  // rest: pieces of unturned coordinates
  const int per = pieces + rest;
  const int tasks = nt * a.heads * per;
#pragma unroll 4
  for (int k = threadIdx.x; k < tasks; k += 256) {
    const int p = k % per, th = k / per;
    const int h = th % a.heads, t = th / a.heads;
    const bool first = h < a.heads0;
    const RopeTensor& r = first ? a.a : a.b;
    const int hh = first ? h : h - a.heads0;
    const T* x = static_cast<const T*>(r.x) + (t0 + t) * r.xt + hh * r.xh;
    T* y = static_cast<T*>(r.y) + (t0 + t) * r.yt + hh * r.yh;
    struct alignas(sizeof(T) * VEC) Piece {
      T v[VEC];
    };
    if (p >= pieces) {  // behind the turned coordinates: copied
      const int at = 2 * a.F + (p - pieces) * 2 * VEC;
      for (int e = at; e < min(a.d, at + 2 * VEC); ++e) y[e] = x[e];
      continue;
    }
    const float2* w = cs + t * a.F + p * VEC;
    const int lo = INTER ? 2 * p * VEC : p * VEC, hi = INTER ? lo + VEC : lo + a.F;
    Piece u = *reinterpret_cast<const Piece*>(x + lo), v = *reinterpret_cast<const Piece*>(x + hi);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      // the e-th pair: (u_e, v_e), or neighbours of the 2 VEC elements u, v when interleaved
      T& pa = INTER ? (2 * e < VEC ? u.v[(2 * e) % VEC] : v.v[(2 * e) % VEC]) : u.v[e];
      T& pb = INTER ? (2 * e + 1 < VEC ? u.v[(2 * e + 1) % VEC] : v.v[(2 * e + 1) % VEC]) : v.v[e];
      const float fa = up<T>(pa), fb = up<T>(pb);
      const float2 cw = w[e];
      pa = down<T>(fa * cw.x - fb * cw.y);
      pb = down<T>(fb * cw.x + fa * cw.y);
    }
    *reinterpret_cast<Piece*>(y + lo) = u;
    *reinterpret_cast<Piece*>(y + hi) = v;
  }
}

template <typename T, int VEC>
cudaError_t launch(const RopeArgs& a, int interleaved, cudaStream_t st) {
  const size_t smem = sizeof(float2) * a.tok * a.F;
  const unsigned grid = static_cast<unsigned>((a.n_tokens + a.tok - 1) / a.tok);
  if (interleaved)
    rope_kernel<T, VEC, true><<<grid, 256, smem, st>>>(a);
  else
    rope_kernel<T, VEC, false><<<grid, 256, smem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace octo

extern "C" int octo_rope_freqs(double theta, int n_axes, const int32_t* sections, int per_axis, uint64_t* freqs) {
  if (!sections || !freqs || !(theta >= 1.0) || !(theta <= 1e300)) return OCTO_EINVAL;
  if (n_axes < 1 || n_axes > 4) return OCTO_EUNSUPPORTED;
  int64_t F = 0;
  for (int k = 0; k < n_axes; ++k) {
    if (sections[k] < 0) return OCTO_EINVAL;
    F += sections[k];
  }
  if (F > 512) return OCTO_EUNSUPPORTED;
  const long double full = 18446744073709551616.0L / 6.283185307179586476925286766559005768L;  // 2^64 / (2 pi)
  int i = 0;
  for (int k = 0; k < n_axes; ++k)
    for (int j = 0; j < sections[k]; ++j, ++i) {
      const long double e = per_axis ? static_cast<long double>(j) / sections[k] : static_cast<long double>(i) / F;
      freqs[i] = static_cast<uint64_t>(powl(theta, -e) * full + 0.5L);
    }
  return OCTO_OK;
}

extern "C" int octo_rope(const octo_rope_tensor* t0, const octo_rope_tensor* t1, int dtype, int64_t n_tokens, int d,
                         const int32_t* positions, int64_t pos_stride, int n_axes, const int32_t* sections,
                         const uint64_t* freqs, int interleaved, int inverse, octo_stream_t stream) {
  using namespace octo;
  if (!t0 || !sections) return OCTO_EINVAL;
  if (dtype != OCTO_F32 && dtype != OCTO_BF16) return OCTO_EINVAL;
  if (n_axes < 1 || n_axes > 4) return OCTO_EUNSUPPORTED;
  if (n_tokens < 0 || d < 2 || d % 2 != 0 || pos_stride < n_tokens) return OCTO_EINVAL;
  if (d > 1024) return OCTO_EUNSUPPORTED;
  RopeArgs a{};
  int64_t F = 0;
  for (int k = 0; k < n_axes; ++k) {
    if (sections[k] < 0) return OCTO_EINVAL;
    F += sections[k];
    if (F > d / 2) return OCTO_EINVAL;
    a.ends[k] = static_cast<int>(F);
  }
  for (int k = n_axes; k < 4; ++k) a.ends[k] = static_cast<int>(F);
  const int esz = dtype == OCTO_F32 ? 4 : 2, vec = 16 / esz;
  const octo_rope_tensor none{};
  const octo_rope_tensor& u = t1 ? *t1 : none;
  const octo_rope_tensor* both[2] = {t0, &u};
  RopeTensor* to[2] = {&a.a, &a.b};
  bool wide = F % vec == 0;
  for (int k = 0; k < 2; ++k) {
    const octo_rope_tensor& r = *both[k];
    if (r.heads < 0 || r.x_token_stride < 0 || r.x_head_stride < 0 || r.y_token_stride < 0 || r.y_head_stride < 0)
      return OCTO_EINVAL;
    if (r.heads > 0 && n_tokens > 0 && (!r.x || !r.y)) return OCTO_EINVAL;
    if (r.heads > 65535) return OCTO_EUNSUPPORTED;
    *to[k] = RopeTensor{r.x, r.y, r.x_token_stride, r.x_head_stride, r.y_token_stride, r.y_head_stride};
    if (r.heads > 0)
      wide = wide && reinterpret_cast<uintptr_t>(r.x) % 16 == 0 && reinterpret_cast<uintptr_t>(r.y) % 16 == 0 &&
             (r.x_token_stride * esz) % 16 == 0 && (r.x_head_stride * esz) % 16 == 0 &&
             (r.y_token_stride * esz) % 16 == 0 && (r.y_head_stride * esz) % 16 == 0;
  }
  a.heads0 = t0->heads;
  a.heads = t0->heads + u.heads;
  if (n_tokens == 0 || a.heads == 0) return OCTO_OK;
  if (!positions || (F > 0 && !freqs)) return OCTO_EINVAL;
  a.n_tokens = n_tokens;
  a.d = d;
  a.F = static_cast<int>(F);
  a.pos = positions;
  a.pos_stride = pos_stride;
  a.freqs = freqs;
  a.inverse = inverse != 0;
  // tokens per block: enough 16-byte pieces for four per thread, but no fewer blocks than two per SM
  const int64_t pieces = std::max<int64_t>(1, static_cast<int64_t>(a.heads) * d / (2 * vec));
  int64_t tok = std::max<int64_t>(1, 1024 / pieces);
  tok = std::max<int64_t>(1, std::min<int64_t>(tok, n_tokens / 296));
  tok = std::min<int64_t>(tok, std::max<int64_t>(1, 4096 / std::max<int64_t>(1, F)));  // 32 KB of cosines and sines
  a.tok = static_cast<int>(tok);
  if ((n_tokens + tok - 1) / tok > INT32_MAX) return OCTO_EUNSUPPORTED;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == OCTO_BF16)
    e = wide ? launch<__nv_bfloat16, 8>(a, interleaved, st) : launch<__nv_bfloat16, 1>(a, interleaved, st);
  else
    e = wide ? launch<float, 4>(a, interleaved, st) : launch<float, 1>(a, interleaved, st);
  return e == cudaSuccess ? OCTO_OK : OCTO_ECUDA;
}
