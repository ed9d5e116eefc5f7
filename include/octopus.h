/*
 * octopus.h - C ABI of the OCTOPUS KV-cache codec for NVIDIA B200 (sm_100a).
 *
 * OCTOPUS (the paper "OCTOPUS: Optimized KV Cache for Transformers via
 * Octahedral Parametrization Under optimal Squared error quantization",
 * abstract; method as described in the youleyou.com explainer, sections
 * "triplet decomposition", "octahedral folding", "non-uniform bit allocation",
 * "joint rounding", "optional residual correction", "engineering
 * implementation") stores each key k as its norm gamma = ||k|| (fp32) and a
 * bit-packed code of its unit direction: the direction is rotated by a
 * seeded sign-flipped Walsh-Hadamard transform, cut into coordinate
 * triplets, and each triplet's norm rho and octahedrally mapped direction
 * (xi, eta) are Lloyd-Max quantised with (b-1, b+1, b+1) bits.
 *
 * Conventions for every entry point
 * ---------------------------------
 *  - Return value: OCTO_OK (0) or a negative OCTO_E* status; nothing aborts,
 *    no C++ exception crosses this boundary. octo_status_string() names it.
 *  - The caller owns every buffer. The library allocates and frees no
 *    memory and keeps no data between calls. The one exception is
 *    octo_decode_attn_static's fixed scratch array. Each kernel's launch
 *    set-up (shared-memory opt-in, blocks resident per SM, SM count) is
 *    looked up on its first call on a device and reused.
 *  - "device" pointers are CUDA global-memory addresses of the current
 *    device; "host" pointers are ordinary process memory.
 *  - Device entry points are asynchronous on the given stream; they return
 *    after the launch (OCTO_ECUDA if the launch itself failed). Arguments
 *    are validated on the host before anything is launched; an invalid
 *    argument returns OCTO_EINVAL and launches nothing.
 *  - Sizes are element counts unless stated otherwise.
 *
 * Supported shapes: head dimension d in {64, 128, 256}; bit budget
 * b in {2, 3, 4}; query rows per KV head (GQA group x query tokens) <= 8.
 *
 * Cache layout in device memory (word-planar, token-contiguous):
 *   packed   uint32 [n_heads][W][cache_cap]       W = ceil(T (3b+1) / 32)
 *   gamma    float  [n_heads][cache_cap]
 *   qjl_bits uint32 [n_heads][d/32][cache_cap]    (OCTOPUS-QJL only)
 *   qjl_norm float  [n_heads][cache_cap]          (OCTOPUS-QJL only)
 * Word w of token n's bit stream is packed[h][w][n]. Within the stream,
 * the (3b+1)-bit code of triplet i starts at bit i(3b+1), LSB first (bit p
 * of the stream is bit p mod 32 of word p / 32); a code is
 *   m_xi | m_eta << b | s_xi << 2b | s_eta << (2b+1) | i_rho << 2(b+1),
 * where a direction cell index i in [0, 2^(b+1)) of the odd-symmetric
 * codebook is stored as a sign s (1 for the lower half, i < 2^b) and the
 * rank m of |level| among the positive levels (m = i - 2^b above the
 * middle, 2^b - 1 - i below).
 */
#ifndef OCTOPUS_B200_H
#define OCTOPUS_B200_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define OCTO_API __attribute__((visibility("default")))
#else
#define OCTO_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* CUDA stream handle (cudaStream_t); 0 is the legacy default stream. */
typedef void* octo_stream_t;

enum octo_status {
  OCTO_OK = 0,
  OCTO_EINVAL = -1,       /* bad argument: null pointer, size, stride, alignment, range */
  OCTO_EUNSUPPORTED = -2, /* valid but not built: d, b or query rows outside the supported set */
  OCTO_ECUDA = -3,        /* a CUDA launch or runtime call failed */
  OCTO_EWORKSPACE = -4    /* workspace smaller than octo_decode_attn_workspace() */
};

enum octo_rounding {
  OCTO_ROUND_SCALAR = 0, /* each of xi, eta, rho to its nearest centroid */
  OCTO_ROUND_JOINT = 1   /* 3x3 joint search ("joint rounding" section); the default */
};

enum octo_dtype { OCTO_F32 = 0, OCTO_BF16 = 1 };

/* Sizes that follow from (d, b). Filled by octo_layout_init. */
typedef struct octo_layout {
  int32_t d;          /* key / head dimension */
  int32_t b;          /* bit budget per coordinate */
  int32_t T;          /* triplets per key, ceil(d/3); the last one is zero-padded if 3 does not divide d */
  int32_t b_dir;      /* bits of xi and of eta: b+1 */
  int32_t b_rho;      /* bits of rho: b-1 */
  int32_t code_bits;  /* bits per triplet: 3b+1 */
  int32_t words;      /* W, 32-bit words per key */
  int32_t n_dir;      /* direction codebook levels, 2^(b+1) */
  int32_t n_rho;      /* norm codebook levels, 2^(b-1) */
  int32_t qjl;        /* 1: keep the OCTOPUS-QJL residual sign sketch (d bits + fp32 norm) */
  int32_t qjl_words;  /* d/32 when qjl, else 0 */
  int32_t rounding;   /* enum octo_rounding */
} octo_layout;

/* Device pointers to the data-independent tables (built by the host
 * functions below, copied to the device by the caller). A cache head h
 * uses table row (h mod n_heads): with caches laid out [batch][kv_head],
 * n_heads = number of KV heads shares one rotation across the batch. */
typedef struct octo_tables {
  const float* dir_c;  /* [n_dir]     direction centroids, increasing */
  const float* dir_t;  /* [n_dir-1]   direction thresholds (cell k = #thresholds <= x) */
  const float* rho_c;  /* [n_rho]     norm centroids, increasing */
  const float* rho_t;  /* [n_rho-1]   norm thresholds */
  const float* signs;  /* [n_heads][d] +1/-1 diagonal of the sign-flipped WHT */
  const float* qjl_S;  /* [n_heads][d][d] row-major Gaussian projection, 16-byte aligned; NULL unless layout.qjl */
  int64_t n_heads;     /* rows in signs / qjl_S, >= 1 */
} octo_tables;

/* Fills *L for head dimension d, bit budget b, QJL flag and rounding mode
 * (explainer, "non-uniform bit allocation": b+1 bits for each direction
 * coordinate, b-1 for the triplet norm). Returns OCTO_EUNSUPPORTED for d or
 * b outside the supported set, OCTO_EINVAL for a NULL L or a bad flag. */
OCTO_API int octo_layout_init(octo_layout* L, int d, int b, int qjl, int rounding);

/* Fills *L for another split of the bit budget (explainer, "non-uniform bit
 * allocation": each direction coordinate gets b + delta bits and the triplet
 * norm b - delta; the OCTOPUS allocation is delta = +1, which
 * octo_layout_init uses). code_bits = 3b + delta. Supported: b in {2, 3, 4}
 * with 2 <= b + delta <= 5 and 1 <= b - delta <= 5 for octo_codebook_build;
 * octo_encode and octo_dequant run delta = +1 for every d and, at d = 128
 * without the sketch, also b = 3 with delta in {-1, 0, +2} and b = 4 with
 * delta in {-1, 0} (the sweep the explainer reports); octo_decode_attn runs
 * delta = +1 only. Other combinations return OCTO_EUNSUPPORTED from the call
 * that cannot run them; qjl with delta != +1 returns OCTO_EUNSUPPORTED here.
 * Errors as octo_layout_init. */
OCTO_API int octo_layout_init_delta(octo_layout* L, int d, int b, int delta, int qjl, int rounding);

/* Host. Lloyd-Max codebooks for layout L (explainer, "triplet
 * decomposition": Lloyd-Max quantisers designed for the marginal law; the
 * abstract: "implementation-matched marginals", data-oblivious). The
 * direction codebook is designed for the marginal of the octahedral map of
 * a uniform direction on the sphere (shared by xi and eta); the norm
 * codebook for the law of the norm of three coordinates of a uniform unit
 * vector in R^d. Outputs are caller-allocated host arrays of n_dir,
 * n_dir-1, n_rho, n_rho-1 floats. Thresholds are the midpoints of adjacent
 * centroids. Deterministic; takes about a second for b = 4. */
OCTO_API int octo_codebook_build(const octo_layout* L, float* dir_c, float* dir_t, float* rho_c, float* rho_t);

/* Host. Rotation signs for n_heads heads of dimension d into the
 * caller-allocated host array signs[n_heads][d] (explainer, "rotation":
 * sign-flipped Walsh-Hadamard transform; abstract: deterministic given a
 * seed). signs[h][j] = -1 if the top bit of SplitMix64 output number
 * h*d + j + 1 (generator seeded with `seed`) is set, else +1. */
OCTO_API int octo_rotation_build(uint64_t seed, int d, int64_t n_heads, float* signs);

/* Host. OCTOPUS-QJL projections S[n_heads][d][d] (caller-allocated host
 * array; explainer, "optional residual correction"). Entry
 * e = (h*d + i)*d + j is the float32 rounding of the Box-Muller normal
 * sqrt(-2 ln u1) cos(2 pi u2), u1 = ((z1 >> 11) + 1) 2^-53,
 * u2 = (z2 >> 11) 2^-53, z1, z2 = SplitMix64 outputs 2e+1 and 2e+2. */
OCTO_API int octo_qjl_build(uint64_t seed, int d, int64_t n_heads, float* S);

/* Device. Encodes n_tokens keys of each of n_heads heads into the cache at
 * token positions [token_offset, token_offset + n_tokens) (explainer,
 * "triplet decomposition" steps 1-4 and "joint rounding"; with layout.qjl
 * also the residual sketch of "optional residual correction").
 *   keys        device, element (h, n, j) at keys[h*head_stride + n*token_stride + j];
 *               key_dtype OCTO_F32 or OCTO_BF16; j is contiguous. Each lane
 *               of a warp loads d/32 consecutive elements at once, so the
 *               base address and both strides (in bytes) must be multiples
 *               of min(16, (d/32) * element size).
 *   cache_cap   tokens per head in the cache arrays (see layout above).
 *   packed, gamma               device, required.
 *   qjl_bits, qjl_norm          device, required iff layout.qjl, else ignored.
 * Errors: OCTO_EINVAL if a pointer is NULL, n_heads < 0, n_tokens < 0,
 * token_offset < 0, token_offset + n_tokens > cache_cap, or a key is
 * misaligned. n_tokens == 0 or n_heads == 0 launches nothing. */
OCTO_API int octo_encode(const octo_layout* L, const octo_tables* tables,
                const void* keys, int key_dtype,
                int64_t n_heads, int64_t n_tokens, int64_t head_stride, int64_t token_stride,
                int64_t cache_cap, int64_t token_offset,
                uint32_t* packed, float* gamma, uint32_t* qjl_bits, float* qjl_norm,
                octo_stream_t stream);

/* Bytes of device workspace octo_decode_attn needs for these sizes (at
 * least 256: the workspace also carries a status word). Returns 0 for
 * unsupported arguments. */
OCTO_API size_t octo_decode_attn_workspace(const octo_layout* L, int B, int Hq, int Hkv, int Lq, int64_t kv_len);

/* Device. One fused decode-attention step over a compressed cache
 * (explainer, "engineering implementation"; abstract: keys are
 * reconstructed on the fly and never materialised). The queries are
 * rotated once by the same transform as the keys, so the raw logit of key n
 * is gamma_n * sum_i rho_hat_i (q_rot_i . n_hat_i) (+ the QJL term
 * gamma_n * nu_n * sqrt(pi/2)/d * <S q_rot, 2 bits_n - 1> when layout.qjl);
 * then softmax(scale * logits) and the product with bf16 V, all on chip.
 *   q        device, [B][Hq][Lq][d], q_dtype OCTO_F32 or OCTO_BF16, contiguous.
 *   Hq = g*Hkv; query head hq reads KV head hq / g. Cache head index is
 *   b*Hkv + h_kv in packed / gamma / qjl_* / V.
 *   packed, gamma, qjl_bits, qjl_norm: the cache (layout above), capacity
 *   cache_cap, the first kv_len tokens are attended. The code rows are
 *   staged into shared memory by 16-byte bulk copies, so cache_cap must be
 *   a multiple of 4 and these four base addresses 16-byte aligned.
 *   V        device bf16 [B*Hkv][cache_cap][d] (16-byte aligned), or NULL
 *            for logits only.
 *   scale    softmax temperature (1/sqrt(d) for standard attention).
 *   out      device fp32 [B][Hq][Lq][d]; required iff V != NULL.
 *   logits   device fp32 [B][Hq][Lq][kv_len] raw (unscaled) logits, or NULL.
 *   workspace device, >= octo_decode_attn_workspace() bytes, 256-byte
 *            aligned, always required. Bytes [0, 4) are a status word: the
 *            kernel ORs in 1 if one of its bounded on-chip waits expired
 *            (the outputs of that call are then invalid). Bytes [256, 256 +
 *            4*B*Hkv) are arrival counters. Status and counters must be zero
 *            before the first call (zero the whole workspace once); every
 *            completed call leaves the counters zero again. The rest is
 *            the call's scratch (per-slice partial results; with
 *            layout.qjl and d <= 128 also the rotated queries and S q_rot of
 *            every KV head). Calls that share a workspace must not overlap
 *            on the GPU.
 * The call launches one kernel on `stream`, two with layout.qjl and
 * d <= 128 (a per-KV-head query preparation into the workspace, then the
 * decode, which reads it).
 * kv_len == 0 gives out = 0. Errors: OCTO_EINVAL (NULL required pointer,
 * bad sizes, kv_len > cache_cap, both V and logits NULL, misalignment),
 * OCTO_EUNSUPPORTED (g*Lq > 8 or B*Hkv > 65535), OCTO_EWORKSPACE. */
OCTO_API int octo_decode_attn(const octo_layout* L, const octo_tables* tables,
                     const void* q, int q_dtype, int B, int Hq, int Hkv, int Lq,
                     int64_t kv_len, int64_t cache_cap,
                     const uint32_t* packed, const float* gamma,
                     const uint32_t* qjl_bits, const float* qjl_norm,
                     const void* V, float scale, float* out, float* logits,
                     void* workspace, size_t ws_bytes, octo_stream_t stream);

/* Device. octo_decode_attn without a caller-provided workspace, for callers
 * that cannot allocate device memory themselves: for example a plugin whose
 * host framework owns every device allocation, or a caller whose allocator
 * cannot be reached from the code that issues the decode step. It allocates
 * nothing: the split-merge scratch is a fixed array of
 * OCTO_STATIC_SCRATCH_BYTES (8 MiB) in the library's own device memory,
 * reserved on every GPU that loads the library until the process exits.
 * (Not part of the method: the paper has no counterpart; this is a
 * deployment convenience.)
 * Arguments and results are those of octo_decode_attn, minus the workspace.
 *   - Returns OCTO_EWORKSPACE when the sizes need more scratch than
 *     OCTO_STATIC_SCRATCH_BYTES (octo_decode_attn_workspace() tells).
 *   - The first call on a device (with that device current) looks up the
 *     array's device address; make that first call outside any stream
 *     capture.
 *   - Arguments are checked exactly as octo_decode_attn checks them (same
 *     status codes, same order) before anything touches the GPU; a
 *     rejected call launches nothing and leaves the array alone.
 *   - Each accepted call zeroes the array's status word and arrival
 *     counters on `stream` before the decode kernel. All calls on a device
 *     share the array, which keeps the last call's contents: calls that
 *     overlap on the GPU (other streams, or other threads) race on it and
 *     must not be issued.
 *   - The kernel's timeout flag (bit 0 of the status word, see
 *     octo_decode_attn) lives in the array; read it with
 *     octo_decode_attn_static_status. */
#define OCTO_STATIC_SCRATCH_BYTES (8u << 20)
OCTO_API int octo_decode_attn_static(const octo_layout* L, const octo_tables* tables,
                                     const void* q, int q_dtype, int B, int Hq, int Hkv, int Lq,
                                     int64_t kv_len, int64_t cache_cap,
                                     const uint32_t* packed, const float* gamma,
                                     const uint32_t* qjl_bits, const float* qjl_norm,
                                     const void* V, float scale, float* out, float* logits,
                                     octo_stream_t stream);

/* Host. The status word that the last octo_decode_attn_static call on the
 * current device left in the library's scratch array (bit 0 set: one of
 * the kernel's bounded on-chip waits expired, and that call's outputs are
 * invalid). Waits for the work queued on `stream` (the stream of that
 * call) to finish, then copies the word into *status. Not part of the
 * method; it serves octo_decode_attn_static's callers, who have no
 * workspace to read the word from. Errors: OCTO_EINVAL (status NULL),
 * OCTO_ECUDA. */
OCTO_API int octo_decode_attn_static_status(int* status, octo_stream_t stream);

/* Device. Fills the whole scratch array of octo_decode_attn_static on the
 * current device with the byte value `byte` & 0xff, on `stream`. A
 * diagnostic: it lets a test leave nonzero status and counter bytes behind,
 * as an interrupted call would, and check that the next call still clears
 * what must start at zero. Normal use never needs it. Same race rules as
 * octo_decode_attn_static. */
OCTO_API int octo_decode_attn_static_fill(int byte, octo_stream_t stream);

/* Device. Reconstructs keys from the cache: k_hat = gamma * R^T u_hat
 * (explainer, "triplet decomposition" steps 1-4 undone, for the codec's
 * compress-and-reconstruct use). u_hat concatenates rho_hat_i * n_hat_i over
 * the T triplets (inverse octahedral map of section "octahedral folding"),
 * padding dropped; R = (1/sqrt(d)) H diag(s_h) is the encoder's rotation, so
 * k_hat_j = gamma * s_h[j] * (H u_hat)_j / sqrt(d). The QJL sketch, if the
 * layout keeps one, is not read: it estimates inner products, it does not
 * correct keys.
 *   packed, gamma  device cache (layout above), cache_cap tokens per head;
 *                  tokens [token_offset, token_offset + n_tokens) of each of
 *                  the first n_heads cache heads are read. Cache head h uses
 *                  sign row h mod tables->n_heads.
 *   out            device [n_heads][n_tokens][d], row-major, out_dtype
 *                  OCTO_F32 or OCTO_BF16 (round to nearest even); 16-byte
 *                  aligned. Computed in fp32.
 * Errors: OCTO_EINVAL (NULL pointer, negative sizes, token_offset +
 * n_tokens > cache_cap, misaligned out, bad out_dtype), OCTO_EUNSUPPORTED
 * (d or b outside the supported set). n_heads == 0 or n_tokens == 0
 * launches nothing. */
OCTO_API int octo_dequant(const octo_layout* L, const octo_tables* tables,
                          int64_t n_heads, int64_t n_tokens, int64_t cache_cap, int64_t token_offset,
                          const uint32_t* packed, const float* gamma, void* out, int out_dtype,
                          octo_stream_t stream);

/* ---------------------------------------------------------------------------
 * Paged cache
 * -----------
 * The compressed cache of many sequences in a pool of pages of page_size
 * token slots, each page holding every KV head (word-planar like the
 * contiguous cache above; a contiguous cache of n_heads = B*Hkv heads is the
 * pool of B pages of Hkv heads and page_size = cache_cap slots). Slot s of
 * sequence i lives in page pages[i*stride + s / page_size] at offset
 * s mod page_size; cache head h uses sign row h mod tables->n_heads. The
 * layout must be the OCTOPUS split without the sketch (else
 * OCTO_EUNSUPPORTED).
 *
 * Page ids, lengths and offsets are device data that the host does not see.
 * The kernels never read or write outside the pool and the tables because of
 * them: they OR bits into *status (when not NULL) and go on, see
 * octo_paged_status. The outputs of the sequences concerned are then
 * unspecified. */
typedef struct octo_pages {
  uint32_t* packed;  /* [n_pages][n_heads][W][page_size] */
  float* gamma;      /* [n_pages][n_heads][page_size] */
  void* V;           /* bf16 [n_pages][n_heads][page_size][d], 16-byte aligned */
  int64_t n_pages;   /* >= 1 */
  int32_t n_heads;   /* KV heads */
  int32_t page_size; /* token slots per page, a multiple of 16 */
  int32_t* status;   /* device word of octo_paged_status bits, or NULL */
} octo_pages;

typedef struct octo_page_table {
  const int32_t* pages; /* device [n_seqs][stride]; entries behind a sequence's last page are not read */
  int64_t stride;       /* entries between rows, >= max_pages */
  int32_t n_seqs;
  int32_t max_pages;    /* entries per row that may be read; max_pages * page_size at most 2^31 - 1 - 65536 */
} octo_page_table;

enum octo_paged_status {
  OCTO_PAGED_TIMEOUT = 1,   /* a bounded on-chip wait expired: the call's outputs are invalid */
  OCTO_PAGED_BAD_PAGE = 2,  /* a page id outside [0, n_pages): reads took page 0 instead, writes were dropped */
  OCTO_PAGED_BAD_LENGTH = 4 /* a length or offset that the tables do not hold (negative, behind the table, not ascending): clamped */
};

/* Device. Rotary positions with up to four axes on the rows of two tensors
 * (queries and, optionally, keys: the step before octo_encode). Row t, head
 * h, frequency i in [0, F), F = the sum of the sections: the pair
 * (x_i, x_{i+F}) (half-split), or (x_2i, x_2i+1) when interleaved, is turned
 * by the angle pos[axis(i)][t] * theta^(-e_i); coordinates from 2F on are
 * copied. The first sections[0] frequencies belong to axis 0, the next
 * sections[1] to axis 1, and so on. e_i = i / F with one frequency scale over
 * all axes, or j / sections[axis] for the j-th frequency of its axis
 * (per_axis). inverse turns back: it is the transpose, so also the gradient
 * of the forward call. Angles are formed to 2^-32 of a turn at every 32-bit
 * position and rounded to fp32 for their cosine and sine: 2^-26 of a turn.
 *   x0, y0  device rows [n_tokens][heads0][d] in and out, dtype OCTO_F32 or
 *           OCTO_BF16, element strides (token, head), the last axis
 *           contiguous; y may be x, and must not overlap it otherwise, nor the
 *           other pair's tensors.
 *   x1, y1  the second pair of tensors, heads1 heads (0: none).
 *   positions device int32 [n_axes][pos_stride].
 *   freqs   device uint64 [F], from octo_rope_freqs.
 * Errors: OCTO_EINVAL (NULL pointer, negative size, odd d, 2F > d, bad
 * dtype, pos_stride < n_tokens), OCTO_EUNSUPPORTED (d > 1024, n_axes outside
 * 1..4). n_tokens == 0 or no heads launches nothing. */
typedef struct octo_rope_tensor {
  const void* x;
  void* y;
  int32_t heads;
  int64_t x_token_stride, x_head_stride, y_token_stride, y_head_stride;
} octo_rope_tensor;
OCTO_API int octo_rope(const octo_rope_tensor* a, const octo_rope_tensor* b, int dtype, int64_t n_tokens, int d,
                       const int32_t* positions, int64_t pos_stride, int n_axes, const int32_t* sections,
                       const uint64_t* freqs, int interleaved, int inverse, octo_stream_t stream);

/* Host. Frequencies of octo_rope in 2^-64 turns per position (caller-allocated
 * host array of sum(sections) values): round(theta^(-e_i) / (2 pi) * 2^64).
 * Errors: OCTO_EINVAL (NULL, a negative section, theta not finite or below
 * 1), OCTO_EUNSUPPORTED (n_axes outside 1..4). */
OCTO_API int octo_rope_freqs(double theta, int n_axes, const int32_t* sections, int per_axis, uint64_t* freqs);

/* Device. Writes new tokens into pages: token t of sequence i (packed row
 * r = cu[i] + t, 0 <= t < cu[i+1] - cu[i]) goes to slot starts[i] + t.
 *   packed, gamma  the tokens' codes as octo_encode left them in a contiguous
 *                  staging cache of pages->n_heads heads, capacity
 *                  staged_cap >= n_rows, rows [0, n_rows).
 *   V              device bf16, row r of head h at V + r*v_row_stride +
 *                  h*v_head_stride (elements), d contiguous; pointer and
 *                  strides multiples of 16 bytes. The pool's V may be NULL
 *                  with V NULL (keys only).
 *   starts, cu     device int32 [n_seqs], [n_seqs + 1]. Rows from cu[n_seqs]
 *                  on (a batch padded to a fixed size) are left alone, as in
 *                  the chunk calls; others without a place are reported.
 * Two tokens must not go to one slot. Errors: OCTO_EINVAL, and
 * OCTO_EUNSUPPORTED for a layout outside the paged set. n_rows == 0 launches
 * nothing. */
OCTO_API int octo_paged_write(const octo_layout* L, const octo_pages* pages, const octo_page_table* table,
                              const uint32_t* packed, const float* gamma, int64_t staged_cap,
                              const void* V, int64_t v_row_stride, int64_t v_head_stride, int64_t n_rows,
                              const int32_t* starts, const int32_t* cu, octo_stream_t stream);

/* Device. Attention of a chunk of new query tokens over a paged cache that
 * already holds them (octo_paged_write first): packed query rows
 * cu_q[i] .. cu_q[i+1] - 1 are the last new_i = cu_q[i+1] - cu_q[i] tokens
 * of sequence i, whose cache holds seq_lens[i] slots. With causal != 0, new
 * token t sees the slots below seq_lens[i] - new_i + t + 1, else all
 * seq_lens[i]. Logits are scale * gamma_n * <R q, u_hat_n> as in
 * octo_decode_attn; a row that sees nothing gives out = 0, lse = -inf.
 *   q    device, row r head h at q + r*q_row_stride + h*q_head_stride
 *        (elements), q_dtype OCTO_F32 or OCTO_BF16, d contiguous.
 *        Query head hq reads KV head hq / (Hq / n_heads).
 *   out  device [n_rows][Hq][d], out_dtype OCTO_F32 or OCTO_BF16, 16-byte aligned; must not overlap q.
 *   lse  device fp32 [n_rows][Hq] ln sum exp(logits), or NULL.
 *   workspace  device, 256-byte aligned, octo_paged_attn_workspace() bytes of
 *        scratch; nothing in it needs to be kept or cleared between calls.
 *        It may be octo_decode_attn's workspace too: bytes [0, 262400), the
 *        front where that call keeps its status word and counters, are left
 *        alone. Calls that share it must not overlap on the GPU.
 * Keys and queries enter the tensor cores as fp16 (queries scaled by a power
 * of two per row), weights and V as bf16; sums and softmax statistics are
 * fp32 (out is divided by the sum of the rounded weights, lse is that of the
 * unrounded ones). An fp32 out therefore carries no more than these types do,
 * errors of about 1e-3 relative; octo_decode_attn keeps about 16 bits of
 * both. Rows of no sequence are left as they were. Values of slots that a row does not see, but another row of its
 * sequence does, must be finite, and the magnitudes of a sequence's values sum
 * to less than 2^60 per coordinate. Two launches.
 * Supported: d in {64, 128}, b in {2, 3, 4}, Hq / n_heads <= 256.
 * Errors: OCTO_EINVAL, OCTO_EUNSUPPORTED, OCTO_EWORKSPACE. n_rows == 0
 * launches nothing. */
OCTO_API size_t octo_paged_attn_workspace(const octo_layout* L, int64_t n_rows, int n_seqs, int Hq, int Hkv);
OCTO_API int octo_paged_attn(const octo_layout* L, const octo_tables* tables, const octo_pages* pages,
                             const octo_page_table* table, const int32_t* seq_lens, const void* q, int q_dtype,
                             int64_t q_row_stride, int64_t q_head_stride, int64_t n_rows, int Hq, const int32_t* cu_q,
                             int causal, float scale, void* out, int out_dtype, float* lse,
                             void* workspace, size_t ws_bytes, octo_stream_t stream);

/* Device. The attention weight that each cached token gathers from a chunk
 * (what eviction by accumulated weight ranks): for every sequence i, cache
 * head h and slot j < seq_lens[i]
 *   mass_out[i][h][j] = decay * mass_in[i][h][j]
 *                       + sum over the chunk's rows and the head's query heads of exp(logit_j - lse)
 * with the logits, masks and rows of octo_paged_attn and its lse. Slots from
 * seq_lens[i] on are left as they were. The sums have a fixed order. A
 * sequence without new rows gives decay * mass_in, also when the chunk has no
 * rows at all (n_rows == 0: q, lse and workspace may then be NULL, and with a
 * NULL mass_out nothing is launched).
 *   mass_in, mass_out device fp32 [n_seqs][n_heads][mass_stride] (the same
 *        array, or not overlapping); mass_in NULL reads as 0. Slots at and
 *        beyond mass_stride are not counted (OCTO_PAGED_BAD_LENGTH).
 * Logits are formed from fp16 pairs (hi + lo) on the tensor cores, the high
 * parts on fixed grids whose products sum exactly: about fp32's precision.
 * Two launches. Supported shapes, workspace rules and errors as
 * octo_paged_attn. */
OCTO_API size_t octo_paged_mass_workspace(const octo_layout* L, int64_t n_rows, int n_seqs, int Hq, int Hkv);
OCTO_API int octo_paged_mass(const octo_layout* L, const octo_tables* tables, const octo_pages* pages,
                             const octo_page_table* table, const int32_t* seq_lens, const void* q, int q_dtype,
                             int64_t q_row_stride, int64_t q_head_stride, int64_t n_rows, int Hq, const int32_t* cu_q,
                             int causal, float scale, const float* lse, float decay, const float* mass_in,
                             float* mass_out, int64_t mass_stride, void* workspace, size_t ws_bytes,
                             octo_stream_t stream);

/* Device. Cuts sequences back to at most `keep` slots per cache head: of the
 * n = min(seq_lens[i], mass_stride) slots of each (sequence, head) the first
 * `sink`, the last `recent` and those of the largest mass between them stay
 * (ties: the lower slot; NaN ranks below every number), keep in all, or all
 * n when n <= keep. They keep their order and move to slots 0.. of the
 * sequence's row in dst_table, in the pool `dst` (which may be `src`; the
 * pages written must not be read by this call). Two launches.
 *   mass     device fp32 [n_seqs][n_heads][mass_stride].
 *   kept     device int32 [n_seqs][n_heads][keep]: the slots kept, ascending; -1 from n on.
 *   new_lens device int32 [n_seqs]: min(n, keep); may be seq_lens itself, and must not overlap it otherwise.
 *   new_mass device fp32 [n_seqs][n_heads][keep] (0 from n on), or NULL; must not overlap mass.
 * Errors: OCTO_EINVAL (NULL pointer, keep < 1, sink or recent < 0, sink +
 * recent > keep, new_mass over mass, new_lens over a part of seq_lens, pools of different heads or page size, one pool with V and
 * the other without, a destination table shorter than keep), OCTO_EUNSUPPORTED (layout; n_seqs * n_heads
 * > 65535). n_seqs == 0 launches nothing. */
OCTO_API int octo_paged_evict(const octo_layout* L, const octo_pages* src, const octo_page_table* src_table,
                              const int32_t* seq_lens, const float* mass, int64_t mass_stride, int32_t keep,
                              int32_t sink, int32_t recent, const octo_pages* dst, const octo_page_table* dst_table,
                              int32_t* kept, int32_t* new_lens, float* new_mass, octo_stream_t stream);

/* Static string for a status code. */
OCTO_API const char* octo_status_string(int status);

/* ABI version of this header (major*100 + minor). */
OCTO_API int octo_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* OCTOPUS_B200_H */
