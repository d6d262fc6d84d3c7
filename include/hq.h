/*
 * hq.h -- C ABI of the MI355X (gfx950) RHT + lattice + bit-strip + Rice codec.
 *
 * The method is the per-tile pipeline of the HyperQuant technical summary
 * (gist.science/ko/paper/2606.23406; Japanese version gist.science/ja/paper/2606.23406), section
 * "Methodology: the HyperQuant pipeline":
 *   component 1  per-tile randomized Hadamard transform RHT_n(x) = H_n D x (D: random +-1), on
 *                tiles of n = 128 values (the summary's example size), or of 64 or 256,
 *   component 2  nearest-point quantisation onto E8 (or D4, A2, or scalar Z) in an integer
 *                embedding, scaled so the rotated tile matches the lattice,
 *   component 3  stripping of the bits that lattice membership fixes, then Rice coding, with the
 *                realised rate within ~0.01 bits per value of the target,
 *   component 4  for KV caches: a per-layer +-1 rotation (folded into D through the seed) and a
 *                subtractive dither U ~ Uniform(V(lattice)) added before and removed after.
 *
 * Conventions of every entry point:
 *  - Pointers named x, out, stream, workspace are DEVICE pointers (HIP global memory of the current
 *    device); `params`, `info`, `out_bytes` are HOST pointers.  `stream` arguments of type
 *    hq_stream_t are hipStream_t values (0 = the null stream).
 *  - The caller owns every buffer.  The library allocates no device memory and keeps no state
 *    between calls apart from immutable constants and a counter that numbers calls (a workspace
 *    reports the errors recorded under the number of its last call, so nothing has to be cleared
 *    before a call); one workspace serves one call in flight.
 *  - Tensors are flat arrays of n values, n a multiple of the tile length TL (64, 128 or 256; 128
 *    by default); tile t is values [TL t, TL t + TL).
 *  - Every call returns HQ_OK (0) or a negative hq_status code; no exception crosses the ABI.
 *  - Errors found on the device (non-finite input, too small an output buffer, corrupt stream) are
 *    recorded in the workspace; blocking calls return them, hq_status() reads them otherwise.
 *
 * Bitstream (format version 1, little-endian; the pages give no format, this is the codec's own):
 *   header, 128 bytes: u32 magic 'HQ01' | u16 version | u8 lattice | u8 dither flags |
 *     u16 tile TL | u8 rice k | u8 log2 tiles per chunk (log2(8192 / TL)) | u32 step (binary32 bits) |
 *     u64 seed | u64 n | u64 tiles | u32 chunks | u32 F (fixed bits per tile) | u64 fixed_off |
 *     u64 unary_off | u64 unary_words | u64 unary_bits | u64 payload_bits | u64 total_bytes | 32 B 0
 *   chunk index at byte 128: chunks+1 u32 offsets, in 64-bit words, into the unary plane; a chunk
 *     is 8192 values (8192 / TL tiles)
 *   fixed plane at fixed_off = align256(128 + 4 (chunks+1)); chunk c = its tiles' records;
 *     tile record at bit t F (bit i of a plane = bit i%8 of byte i/8): bf16 tile scale (16) |
 *     coset bits (E8: octet o at bit o, TL/8 bits; A2: pair j of octet o at bit 4o+j, TL/2 bits;
 *     none for D4 and Z) | octet 0..TL/8-1, slot 0..7: Rice remainder, width k (full slots) or
 *     max(k-1,0) (halved slots: the parity-fixed slot 7 of E8, 3 and 7 of D4; the stretched odd
 *     slots of A2), LSB first
 *   unary plane at unary_off = align256(fixed_off + chunks (8192 / TL) F / 8): chunk c's segment
 *     starts at word index[c]; each symbol in (tile, octet, slot) order contributes
 *     (symbol >> width) zero bits and a one; segments are zero-padded to 64 bits.
 *   Symbols per octet (8 consecutive coordinates): E8: z in 2E8, p = z0 & 1, u = (z-p)/2,
 *     slots zz(u0..u6), zz((u7 - (u0+..+u6 & 1))/2); D4 (two blocks): zz(x0..x2),
 *     zz((x3 - (x0+x1+x2 & 1))/2); A2 (four pairs, stretched coordinates, z = 2c with
 *     z_2j = z_2j+1 mod 2): p_j = z_2j & 1, slots zz((z_2j - p_j)/2), zz((z_2j+1 - p_j)/2);
 *     Z: zz(z0..z7); zz(a) = (a << 1) ^ (a >> 31).
 *   A2 is the hexagonal lattice with minimal distance 1; each pair (v0, v1) is quantised as
 *     (v0, v1 / sqrt 3) onto Z^2 u (Z+1/2)^2 under the distance dw0^2 + 3 dw1^2: its odd slots use
 *     the multiplier 1 / ((s step) R) and reconstruct with (s step) R, R = binary32 sqrt 3.
 *   Dither flags (0: no dither): bit 0 dither on; bit 1 the dither's Philox4x32 calls take 7 rounds
 *     instead of 10; bit 2 a 24-bit draw instead of 16 bits (valid: 0, 1, 3, 5, 7).  Octet o of
 *     tile t draws b in [0, 2)^8 from Philox with key = seed and counter (o, t lo, t hi, 1): the
 *     eight 16-bit halves (low first) / 2^15; with 24 bits, words w0..w3 of that call and w4..w7
 *     of counter (o, t lo, t hi, 2) give (w_i >> 8) / 2^23.  U = b - Q(b), Q the lattice's
 *     nearest point: uniform on the Voronoi cell to the draw's resolution.  The pages fix neither
 *     the round count nor the resolution; 10 rounds and 16 bits are the defaults.
 */
#ifndef HQ_H_
#define HQ_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef void *hq_stream_t; /* a hipStream_t */

typedef enum {
  HQ_OK = 0,
  HQ_ERR_INVALID_ARG = -1, /* null pointer, bad enum, n % TL != 0, n > 2^35, step outside 2^+-12  */
  HQ_ERR_UNSUPPORTED = -2, /* tile size other than 64, 128, 256; or a unary plane of 2^32 words+     */
  HQ_ERR_NONFINITE = -3,   /* a tile whose transformed energy is NaN or Inf                         */
  HQ_ERR_CAPACITY = -4,    /* output buffer too small; *out_bytes holds the size needed            */
  HQ_ERR_CORRUPT = -5,     /* stream fails validation (header, index, segment, terminator count)   */
  HQ_ERR_RATE = -6,        /* target outside [1.125 (E8), 1.5 (A2) or 1.0 (D4, Z), 12] bits / value */
  HQ_ERR_HIP = -7,         /* a HIP runtime call failed                                             */
  HQ_ERR_TIMEOUT = -8,     /* reserved: no longer produced (every cross-workgroup wait now ends)   */
  HQ_ERR_SCRATCH = -9      /* hq_encode_noalloc: n above its static workspace's maximum (2^30 values) */
} hq_status_code;

typedef enum { HQ_Z = 0, HQ_D4 = 1, HQ_E8 = 2, HQ_A2 = 3 } hq_lattice;
typedef enum { HQ_F32 = 0, HQ_BF16 = 1 } hq_dtype;

typedef struct {
  uint32_t tile;       /* values per tile: 64, 128 or 256 (component 1: "tiles, e.g. 128")         */
  int32_t lattice;     /* hq_lattice                                                                */
  float target_bps;    /* payload bits per value (coset + Rice bits / n); used when step == 0       */
  uint64_t seed;       /* Philox key of the sign diagonal D and of the dither                        */
  uint32_t dither;     /* dither flags: 0 off; 1 subtractive dither (component 4); + 2: 7-round     */
                       /* Philox for the draw; + 4: 24-bit draw (3, 5, 7; see the format above)     */
  float step;          /* 0 = choose by rate control; > 0 = fixed lattice step (KV append, tests);
                          -1 (hq_encode only) = the step and k the workspace holds: those that a
                          preceding hq_rate or hq_encode on the same workspace chose            */
  int32_t rice_k;      /* -1 = automatic; 0..15 = fixed Rice parameter                              */
} hq_params;

typedef struct {
  float step;           /* lattice step used                                                         */
  int32_t rice_k;       /* Rice parameter used                                                       */
  uint64_t bytes;       /* stream size                                                              */
  uint64_t payload_bits;/* coset + remainder + unary bits                                            */
  double payload_bps;   /* payload_bits / n: the rate that rate control targets                     */
  double side_bps;      /* (tile scales + header + index + padding) bits / n                          */
  double total_bps;     /* 8 bytes / n                                                              */
} hq_info;

/* Library and format version: returns (major << 16) | format_version.
 * Defined by this codec (the pages give no format); the format is the one described above. */
uint32_t hq_version(void);

/* Human-readable text of a status code (static storage).  Host only; no device call. */
const char *hq_strerror(int code);

/* Bytes of device workspace that hq_encode / hq_rate / hq_decode / hq_codes need for n values
 * (host only; no device call).  The workspace needs no initialisation.
 * The workspace holds the state of components 1-3 of "Methodology: the HyperQuant pipeline"
 * across the kernels of one call: the operating point that rate targeting (component 3) picks, its
 * sample counters, and the encoder's per-chunk offset flags.  HQ_ERR_INVALID_ARG: bytes == NULL or
 * n not a multiple of 64. */
int hq_workspace_size(uint64_t n, const hq_params *params, size_t *bytes);

/* Stream size for n values at a fixed step, Rice k and tile length, without the unary plane (host
 * only): the header, index and fixed plane.  The unary plane adds (symbol >> width) + 1 bits per value,
 * which depends on the data (hq_encode_bound bounds it).  Component 3 of "Methodology: the
 * HyperQuant pipeline" (Rice codes: a fixed-width remainder per symbol).  HQ_ERR_INVALID_ARG for a
 * bad lattice or k, or n % tile != 0; HQ_ERR_UNSUPPORTED for another tile length. */
int hq_stream_fixed_bytes(uint64_t n, int32_t lattice, int32_t rice_k, uint32_t tile, uint64_t *bytes);

/* Worst-case stream size in bytes for n values encoded with `params` (host only; no device call),
 * so that a caller can size the output of an asynchronous hq_encode, or of a KV-cache append at a
 * fixed operating point, before the data exist.  Component 3 of "Methodology: the HyperQuant
 * pipeline" codes lattice symbols with Rice codes and no overload region (the codebook is
 * unbounded), so the size is bounded only through the energy normalisation of component 2: each
 * tile's scale s (the bf16 RMS of its transformed values, 16 bits) makes the lattice inputs w of a
 * tile satisfy sum w^2 <= TL K^2 / step^2, K = 1 + 2^-7 (the bf16 rounding of s and the binary32
 * roundings).  By Cauchy-Schwarz, sum |w| <= TL K / step; a lattice point lies within the covering
 * radius of its input (and the dither of component 4 within the Voronoi cell), and a Rice unary
 * part of a symbol of magnitude u with parameter k is at most u / 2^k + 1 bits.  Summed per tile:
 *   unary bits <= TL + (A TL K / step + (TL / 8) B) / 2^k,
 * A = 2 (E8, D4, Z) or sqrt(14/3) (A2), B per octet: E8 2 sqrt 8 d + 12, D4 8 d + 8, Z 8 d,
 * A2 (4 sqrt 28 / 3) d + 12, where d = 1 without dither and 2 with it; then the stream layout
 * (header, index, fixed plane, 64-bit padding per chunk).  params->step > 0 is used as given;
 * step == 0 or -1 (the step is chosen later) takes the smallest step of the range, 2^-12;
 * params->rice_k == -1 takes the largest bound over k = 0..15.  target_bps and seed play no part.
 * The bound holds for every input whose tiles are each all zero or hold a value of magnitude at
 * least 2^-60 (it then covers the binary32 rounding of the tile energy; a tile whose values all lie
 * below 2^-60 in magnitude can round its energy down and exceed it).  An encode whose stream would
 * exceed the buffer is never written past it: hq_encode then reports HQ_ERR_CAPACITY.
 * HQ_ERR_INVALID_ARG for a null pointer, a bad lattice, dither flags or k, n % tile != 0,
 * n > 2^35 or a step outside [2^-12, 2^12]; HQ_ERR_UNSUPPORTED for another tile length. */
int hq_encode_bound(uint64_t n, const hq_params *params, uint64_t *max_bytes);

/* Rate control alone: component 3 of "Methodology: the HyperQuant pipeline" (rate targeting, the
 * realised rate within ~0.01 bits per value of the target).  Chooses the lattice step and Rice
 * parameter for x so that the payload rate of a jittered stratified sample of min(T, 8192) tiles
 * meets params->target_bps (a coarse pass on min(T, 2048) tiles first).  With info != NULL the call
 * blocks and fills info (payload_bps is the target); with info == NULL it only enqueues work, and a
 * following hq_encode with params->step == -1 on the same workspace and stream encodes at the chosen
 * point (the pair then does exactly what one hq_encode with rate control does).  x must be 16-byte
 * aligned and the workspace 256-byte aligned (HQ_ERR_INVALID_ARG otherwise), as for hq_encode.
 * Errors: HQ_ERR_INVALID_ARG (null or misaligned pointers, bad params, step == -1, a workspace
 * smaller than hq_workspace_size), HQ_ERR_RATE (target outside the lattice's range),
 * HQ_ERR_UNSUPPORTED (tile length); device-side HQ_ERR_NONFINITE / HQ_ERR_TIMEOUT when blocking. */
int hq_rate(const void *x, int32_t dtype, uint64_t n, const hq_params *params, hq_info *info,
            void *workspace, size_t workspace_bytes, hq_stream_t stream);

/* Encode x (n values, dtype hq_dtype) into `out` (device, out_capacity bytes): components 1-4 of
 * "Methodology: the HyperQuant pipeline" (per-tile RHT H D x; nearest point of the scaled lattice;
 * stripping of the bits lattice membership fixes and Rice coding; the subtractive dither of the KV
 * path when params->dither is set).
 * With out_bytes != NULL the call blocks, stores the stream size in *out_bytes (also when the
 * result is HQ_ERR_CAPACITY: the size needed) and fills *info (may be NULL).  With out_bytes == NULL
 * the call only enqueues work on `stream`; the size is in the stream header (total_bytes) and
 * device-side errors are returned later by hq_status(workspace).  Rate control runs when
 * params->step == 0; step > 0 fixes the step; step == -1 takes the operating point that the
 * workspace holds: the one a preceding hq_rate, or a preceding hq_encode with step >= 0, chose on
 * it (repeated step == -1 calls, e.g. appends to a KV cache at one operating point, keep using
 * it).  Every call resets the workspace's status, results and offset flags first; an encode with
 * step == -1 on a workspace that holds no operating point reports HQ_ERR_INVALID_ARG (blocking) or
 * through hq_status.  x, out: 16-byte aligned; workspace: 256-byte aligned, at least
 * hq_workspace_size(n) bytes.  Errors: as hq_rate, plus HQ_ERR_CAPACITY (out too small; nothing
 * is written past out_capacity) and HQ_ERR_UNSUPPORTED (a unary plane of 2^32 words or more). */
int hq_encode(const void *x, int32_t dtype, uint64_t n, const hq_params *params, void *out,
              uint64_t out_capacity, uint64_t *out_bytes, hq_info *info, void *workspace,
              size_t workspace_bytes, hq_stream_t stream);

/* For callers that cannot allocate device memory (code under HIP graph capture, tight serving
 * loops, harnesses that forbid hipMalloc): hq_encode without a workspace argument.  The workspace
 * is a static device array of the library, 1,065,472 bytes on each GPU the library runs on, held
 * until the process ends; it serves n up to 2^30 values (HQ_ERR_SCRATCH above that).  The call
 * allocates nothing.  Arguments, results and errors are those of hq_encode with the same params
 * (the same kernels, the same stream bytes); step == -1 takes the operating point of the previous
 * hq_encode_noalloc on this GPU.  Every call on a GPU shares that GPU's array: each call resets its
 * status, results and offset flags first, and calls that overlap on one GPU (other streams, other
 * host threads) race and may corrupt each other's streams.  With out_bytes == NULL the call only
 * enqueues work; its device-side errors then have no workspace to be read from (the stream
 * header's total_bytes still gives the size, and a stream is complete when that is at most
 * out_capacity), so callers that must learn of non-finite input use the blocking form. */
int hq_encode_noalloc(const void *x, int32_t dtype, uint64_t n, const hq_params *params, void *out,
                      uint64_t out_capacity, uint64_t *out_bytes, hq_info *info, hq_stream_t stream);

/* Decode a stream of `stream_bytes` bytes into out (n values of out_dtype; bf16 is round to nearest
 * even of the fp32 reconstruction): the exact inverse of components 1-4 of "Methodology: the
 * HyperQuant pipeline" (Rice and unstrip are lossless; yhat = (c - U) s step; x = D H yhat / TL,
 * the transform being orthogonal up to the factor TL).  Asynchronous: header and per-chunk
 * validation happen on the device; call hq_status(workspace) to learn of HQ_ERR_CORRUPT.  On a
 * corrupt stream the output contents are unspecified, but no access leaves the given buffers.
 * out: n values, 16-byte aligned; stream_data 16-byte aligned; workspace 256-byte aligned, at least
 * hq_workspace_size(0) bytes.  HQ_ERR_INVALID_ARG on the host for bad pointers, dtype or n. */
int hq_decode(const void *stream_data, uint64_t stream_bytes, void *out, int32_t out_dtype,
              uint64_t n, void *workspace, size_t workspace_bytes, hq_stream_t stream);

/* Waits for `stream` and returns the first device-side error recorded in `workspace` since the last
 * hq_encode / hq_decode / hq_rate / hq_codes / hq_gemv that used it (HQ_OK when none).  Reports
 * the device-side outcome of the calls above (no step of the method of its own). */
int hq_status(void *workspace, hq_stream_t stream);

/* Diagnostic of the last call that used `workspace` (waits for `stream`): which of its bounded
 * cross-workgroup waits ran out of their spin budget and computed the awaited value themselves.
 * No passage of the pages defines these waits: they are this codec's way of running rate targeting
 * (component 3 of "Methodology: the HyperQuant pipeline") and the stream's chunk offsets in single
 * launches.  A fallback gives the same result as the normal path, only later (microseconds to
 * milliseconds), so the flags concern speed, never correctness.  *flags receives bit 0: a
 * look-back computed a predecessor chunk's offset contribution from its input; bit 1: a rate
 * workgroup solved pass A itself instead of waiting for its published centre; bit 2: a rate
 * solver evaluated a pass's whole sample itself.  Errors: HQ_ERR_INVALID_ARG (null pointer),
 * HQ_ERR_HIP. */
int hq_fallbacks(const void *workspace, hq_stream_t stream, uint32_t *flags);

/* Workspace bytes for hq_gemv on a [rows][cols] matrix (host only; enough for any tile length).
 * Holds the rotated activation and the per-tile partial products of the fused product below. */
int hq_gemv_workspace_size(uint64_t rows, uint64_t cols, size_t *bytes);

/* Fused decode + matrix-vector product y = W_hat x, where the stream encodes a row-major
 * [rows][cols] matrix (n = rows * cols; tiles of TL values along cols, so cols % TL == 0) and W_hat
 * is the decoder's reconstruction taken in exact arithmetic.  x: cols values of x_dtype (device),
 * y: rows binary32 values (device).  Since tile (r, j) decodes to D H yhat / TL (component 1's
 * transform is orthogonal up to the factor TL and H is symmetric), its contribution is
 * <yhat, H D x_j> / TL: the activation is rotated once per column tile (binary32, the encoder's
 * butterfly order) and no matrix tile is inverse-transformed.  Per tile, yhat = (c - U) * s * step
 * rounded to binary32, the octet products are a fixed-order chain, the tile sum a fixed tree, and
 * the row sum adds the tiles in column order, so results are deterministic; they differ from an
 * exact product by rounding only (relative to sum |yhat| |x~|, a few hundred units of 2^-24).
 * Components 1-3 of the HyperQuant technical summary (section "Methodology: the HyperQuant
 * pipeline"); fused decode + matrix products are the direction its section "Significance and
 * claims" names for a wall-clock gain.  Asynchronous;
 * stream validation as for hq_decode (a stream whose tile length does not divide cols is corrupt
 * for this call), errors through hq_status(workspace). */
int hq_gemv(const void *stream_data, uint64_t stream_bytes, uint64_t rows, uint64_t cols, const void *x,
            int32_t x_dtype, float *y, void *workspace, size_t workspace_bytes, hq_stream_t stream);

/* The per-layer Haar-uniform rotation of a seed (component 4 of "Methodology: the HyperQuant
 * pipeline": the full-matrix alternative to the +-1 sign diagonal), written to q (HOST pointer, 128 * 128 floats, q[128 i + j] = Q[i][j]).
 * Construction (the pages give none; the textbook one): G with independent N(0,1) entries, entry
 * e = 128 i + j from Philox4x32-10 with key = seed and counter (e / 4, 0, 0, 2), two Box-Muller
 * pairs per call (u(w) = (w + 1/2) 2^-32; r = sqrt(-2 ln u(w0)); (r cos 2pi u(w1), r sin 2pi u(w1)),
 * then (w2, w3)); G = Q R with diag(R) > 0, computed in binary64 and rounded to binary32.
 * Host only, deterministic. */
int hq_haar_matrix(uint64_t seed, float *q);

/* y_v = Q x_v (transpose = 0; the rotation before hq_encode) or Q^T x_v (transpose = 1; after
 * hq_decode) for every 128-value vector v of x.  x, y: DEVICE, n bf16 values each (n % 128 == 0),
 * 16-byte aligned, may not overlap; q: DEVICE, 128 * 128 binary32 as from hq_haar_matrix.
 * On MFMA (bf16 inputs, Q split into two bf16 parts, binary32 accumulation); y is rounded to bf16
 * (nearest even).  Asynchronous on `stream`.  Component 4 of "Methodology: the HyperQuant
 * pipeline" (the per-layer rotation of the KV path, applied before the codec and undone after).
 * HQ_ERR_INVALID_ARG for null or misaligned pointers or n % 128 != 0. */
int hq_rotate(const void *x, uint64_t n, const float *q, int32_t transpose, void *y, hq_stream_t stream);

/* ---------------------------------------------------------------------------------------------
 * SRFT fixed-rate KV codec ("When quantization is free" technical summary,
 * gist.science/ko/paper/2605.05699, section "Methodology" 1-3): per 128-value vector,
 * v = pack(F diag(s) x) / lambda with F the unitary DFT, s the sign diagonal of `seed` (the same
 * signs as the lattice codec's D), pack the orthogonal real form (X_0, X_64, sqrt 2 Re X_1,
 * sqrt 2 Im X_1, ...), lambda a per-coordinate calibration scale; then 16 groups of 8 coordinates,
 * scale Delta = binary16(absmax / L) (L = 7 for int4, 127 for int8; nearest even, saturating at
 * 65504) and codes q = clamp(rint(v * (1 / Delta)), -L, L).  Fixed rate: 4 (or 8) bits per value
 * plus 16 binary16 scales per vector (96 bytes per vector at int4, 2.67x smaller than bf16).
 *
 * codes: DEVICE, n / 2 bytes (bits = 4: codes 2j and 2j + 1 of a vector in the low and high nibble
 * of its byte j, two's complement) or n bytes (bits = 8, int8); scales: DEVICE, n / 128 * 16
 * binary16 values (vector-major).  x / out: DEVICE, n values of `dtype` / `out_dtype` (HQ_F32 or
 * HQ_BF16), n % 128 == 0.  All device pointers 16-byte aligned.  lambda: HOST, 128 binary32 values,
 * each finite and > 0 (HQ_ERR_INVALID_ARG otherwise), or NULL for all ones; encoder and decoder
 * must be given the same lambda and seed.  A vector whose packed coordinates are not all finite is
 * stored with zero codes and NaN (0x7E00) scales and decodes to NaN.  Decode outputs bf16 rounded
 * to nearest even (or binary32), exact zeros as +0.  Both calls are asynchronous on `stream`, use
 * no workspace and allocate nothing. */
int hq_srft_encode(const void *x, int32_t dtype, uint64_t n, uint64_t seed, const float *lambda, int32_t bits,
                   void *codes, void *scales, hq_stream_t stream);
int hq_srft_decode(const void *codes, const void *scales, uint64_t n, uint64_t seed, const float *lambda,
                   int32_t bits, void *out, int32_t out_dtype, hq_stream_t stream);

/* ---------------------------------------------------------------------------------------------
 * The paged SRFT cache of one layer: the SRFT codec's codes and scales, kept by page so that a serving
 * loop can append tokens, attend over the codes, and evict tokens.
 *
 * data: DEVICE, [pages][heads][page bytes], 16-byte aligned.  A page holds `page` tokens (a power of two,
 * 16 to 4096) of one KV head, 128 values each.  With E = `bits` (4 or 8) bytes for a group's 8 codes:
 *   K codes [page][16][E] | K scales [page][16] binary16 |
 *   V codes [page/4][16][4][E] | V scales [page/4][16][4] binary16
 * (values lie in blocks of four tokens, group by group), in all page * 2 * (16 E + 32) bytes.  Codes,
 * scales and the treatment of non-finite vectors are those of hq_srft_encode with the same seed and
 * lambda (lambda_k for keys, lambda_v for values; HOST, 128 binary32 values or NULL for ones).
 * A slot is page * P + offset.  Token t of sequence b is slot offset t mod P of page
 * table[b * table_width + t / P]; a table entry outside [0, pages) is an absent page, whose tokens take
 * no part, and so does a token whose K scales are -0 (hq_kv_append writes none; hq_kv_evict does).  All calls below are asynchronous on `stream`, allocate nothing and may be captured. */
typedef struct {
  void *data;
  uint32_t pages, heads, page;
  int32_t bits;
  uint64_t seed;
  const float *lambda_k, *lambda_v;
} hq_kv_cache;

/* Encodes the K and V vectors of `tokens` tokens into their slots.  k, v: DEVICE, value c of head h of
 * token i at k[i strides[0] + h strides[1] + c] and v[i strides[2] + h strides[3] + c] (strides in
 * values; 16-byte aligned rows are read fastest).  slots: DEVICE, int64; a slot outside [0, pages * page)
 * writes nothing; the slots of one call must differ.  Codes and scales equal hq_srft_encode's.
 * HQ_ERR_INVALID_ARG: null or misaligned pointers, a bad cache, dtype or lambda, over 2^31 tokens. */
int hq_kv_append(const hq_kv_cache *cache, const void *k, const void *v, int32_t dtype, uint64_t tokens,
                 const int64_t strides[4], const int64_t *slots, hq_stream_t stream);

/* Decodes slots into k and v (DEVICE, [tokens][heads][128] of out_dtype, 16-byte aligned; one may be
 * NULL), as hq_srft_decode does.  A slot outside the cache reads as zeros.  Errors as hq_kv_append. */
int hq_kv_read(const hq_kv_cache *cache, const int64_t *slots, uint64_t tokens, void *k, void *v,
               int32_t out_dtype, hq_stream_t stream);

/* Softmax attention of queries over the cache.  Query i of a sequence's m queries stands at position
 * n - m + i of its n = lens[b] cached tokens (its own token is cached first); it sees tokens up to its
 * position (all tokens when causal == 0), and with window > 0 only the last `window` of those up to its
 * position.  Scores are scale q.k, then softcap tanh(score / softcap) when softcap > 0; a row that sees
 * nothing gives 0.  Query head j reads KV head j / (q_heads / heads).  Transformed queries, keys, values
 * and softmax weights enter the products as binary16, each off by at most 2^-11 of itself whatever its
 * size (next to a scale of 2^13, at 8 bits 2^9, or more, scales of the same 16 tokens are off by up to
 * 2^-18); sums, maxima and softmax statistics are binary32.  With weights asked for, queries and keys
 * enter in two parts, and a score is off by about 2^-20 of scale sum |q_c k_c|; out then differs from a
 * call without weights by that much. */
typedef struct {
  const void *q;            /* DEVICE, value c of head j of query i at q[i stride_token + j stride_head + c] */
  void *out;                /* DEVICE, [total_q][q_heads][128], 16-byte aligned                              */
  int32_t q_dtype, out_dtype;
  int64_t q_stride_token, q_stride_head;
  uint64_t total_q;
  uint32_t q_heads;         /* a multiple of the cache's heads                                             */
  uint32_t seqs;
  uint32_t max_q;           /* most queries of a sequence; further ones count in m but are not computed     */
  uint32_t max_len;         /* most tokens of a sequence; a larger length counts as this                    */
  const int32_t *q_start;   /* DEVICE, seqs + 1 query offsets that do not decrease (cut to [0, total_q]);
                               NULL: total_q / seqs queries each                                            */
  const int32_t *table;     /* DEVICE, [seqs][table_width]                                                  */
  uint32_t table_width;
  const int32_t *lens;      /* DEVICE, [seqs]; a negative length counts as 0                                */
  float scale, softcap;
  int32_t causal;
  uint32_t window;          /* 0: none                                                                      */
  float *weights;           /* DEVICE or NULL: weights[(b heads + h) weights_stride + t] += the softmax
                               weights of token t summed over the rows of KV head h, in a fixed order       */
  uint64_t weights_stride;  /* at least max_len                                                             */
} hq_kv_attend_args;

/* Workspace bytes of hq_kv_attend for these sizes (host only; pointers are not read; the errors are
 * hq_kv_attend's).  About 264 bytes a row of total_q x q_heads (520 with weights), and up to 300 MB for the
 * outputs of split tiles; where no sequence has more than 16 rows a KV head, 4 bytes a row and, with weights,
 * 4 bytes for each of max_len tokens a row.  The workspace needs no initialisation, is 256-byte aligned, and
 * serves one call in flight. */
int hq_kv_attend_workspace_size(const hq_kv_cache *cache, const hq_kv_attend_args *args, size_t *bytes);

/* HQ_ERR_INVALID_ARG: null or misaligned pointers, sizes outside their ranges, q_heads not a multiple of
 * heads, q_start == NULL with total_q not a multiple of seqs, a scale that is not a number in
 * [-2^126, 2^126], a softcap that is neither 0 nor in [2^-125, 2^125], weights_stride < max_len, max_len over 2^30, a launch of 2^32 threads or more (2^28
 * rows of queries and heads), or a workspace that is too small.  Rows of `out` that no sequence's queries name are not written. */
int hq_kv_attend(const hq_kv_cache *cache, const hq_kv_attend_args *args, void *workspace,
                 size_t workspace_bytes, hq_stream_t stream);

/* hq_kv_attend for a tree of drafted tokens.  The last m cached tokens of a sequence are drafts, the tokens of its m
 * queries in order, and parents[i] (DEVICE, int32 [total_q]) is the draft, counted within its sequence, that query i's
 * draft follows; a value that is not in [0, i) means that it follows the n - m tokens held before the drafts.  Query i
 * sees those and, of the drafts, its own and its ancestors; with window > 0 only the last `window` of what it sees.
 * args->causal must not be 0 and args->weights must be NULL (a rejected draft's weights could not be taken back);
 * args->max_q is at most 256; the launch is sized for sequences of that many drafts, so the most that there are is best.  The workspace is hq_kv_attend's kind, of its own size.  Errors as hq_kv_attend. */
int hq_kv_attend_tree_workspace_size(const hq_kv_cache *cache, const hq_kv_attend_args *args, size_t *bytes);
int hq_kv_attend_tree(const hq_kv_cache *cache, const hq_kv_attend_args *args, const int32_t *parents,
                      void *workspace, size_t workspace_bytes, hq_stream_t stream);

/* Places for tokens: pages come from, and go back to, a stack of free ones.  counts[b] > 0: sequence b gets that many
 * more tokens; < 0: its last -counts[b] tokens go (all of them, if there are fewer) and the pages that they leave empty
 * return, their table entries becoming -1.  Pages return from the last sequence's last to the first's first, an entry
 * outside [0, pages) does not, and what the stack cannot hold is dropped; then sequences grow in order, each taking its
 * pages from the top.  A sequence whose table is too narrow takes nothing; from the first that the stack cannot serve on,
 * no sequence grows.  So a call with the counts that a call granted, negated, undoes it.
 * Sequence b's new tokens are `slots` and `positions` q_start[b] .. q_start[b + 1] - 1 (q_start counts what was asked for): token i of them
 * stands at position t = lens[b] + i in slot table[b][t / page] page + t mod page, or -1 if the sequence did not grow or
 * the entry is outside [0, pages).  Places past the last have slot -1 and position 0.
 * A sequence that did not grow (granted[b] == 0 where counts[b] > 0) still has its rows in q_start, but its last tokens are not
 * those rows': for hq_kv_attend, hq_kv_attend_tree and hq_kv_accept it is given a length of 0 until it grows (its rows see
 * nothing and nothing of it moves), and the change that hq_kv_accept returns for it is left out.
 * Asynchronous, allocates nothing, may be captured. */
typedef struct {
  int32_t *table;            /* DEVICE, [seqs][table_width], in and out                              */
  int32_t *lens;             /* DEVICE, [seqs], in and out: tokens held (cut to 0 .. table_width page) */
  const int32_t *counts;     /* DEVICE, [seqs]                                                       */
  int32_t *free;             /* DEVICE, [pages], in and out: free[0 .. *free_count - 1] are free        */
  int32_t *free_count;       /* DEVICE, in and out (cut to 0 .. pages)                               */
  uint32_t seqs, table_width, pages, page;  /* page: tokens of a page, a power of two from 16 to 4096 */
  uint64_t tokens;           /* places in slots and positions                                       */
  int64_t *slots;            /* DEVICE, [tokens]                                                    */
  int32_t *positions;        /* DEVICE or NULL, [tokens]                                            */
  int32_t *q_start;          /* DEVICE, [seqs + 1]; saturates at 2^31 - 1                           */
  int32_t *granted;          /* DEVICE, [seqs]: by how much the sequence's length changed              */
} hq_kv_reserve_args;
/* HQ_ERR_INVALID_ARG: null or misaligned pointers, a bad page, over 2^31 tokens, pages, or table_width page, a table of 2^31
 * entries or more. */
int hq_kv_reserve(const hq_kv_reserve_args *args, hq_stream_t stream);

/* Acceptance of drafted tokens.  Draft i of a sequence's m drafts (its last m cached tokens, m and the offsets as in
 * hq_kv_attend_tree) is token tokens[i] behind parents[i], and the model's choice behind it is target[i].  Draft 0, which
 * an earlier step chose, is accepted; behind the accepted draft i the first draft j with parents[j] = i and
 * tokens[j] = target[i] is, and so on.  The K and V of the accepted drafts move, head by head, to tokens n - m, n - m + 1, ...;
 * those behind them are left as they are.  An absent page's draft becomes one that takes no part (zeros, K scales -0).
 * path [seqs][max_q]: the accepted drafts, then -1; accepted [seqs]: how many; next [seqs]: the target behind the last
 * (-1 without drafts); change [seqs]: accepted - m, the change of the sequence's length (hq_kv_reserve takes it).
 * Only the first max_q drafts are looked at, at most 256.  lens is not changed.  Of a sequence whose drafts are not cached, as it got
 * no places for them, held tokens would be taken for drafts: see hq_kv_reserve for what it is given instead. */
typedef struct {
  const int32_t *table;      /* DEVICE, [seqs][table_width]                                */
  const int32_t *lens;       /* DEVICE, [seqs], the drafts among them                      */
  const int32_t *q_start;    /* DEVICE, [seqs + 1], or NULL: total_q / seqs drafts each       */
  const int32_t *tokens, *target, *parents;  /* DEVICE, [total_q]                           */
  uint64_t total_q;
  uint32_t seqs, table_width, max_q;
  int32_t *path, *accepted, *next, *change;  /* DEVICE                                      */
} hq_kv_accept_args;
/* HQ_ERR_INVALID_ARG: null or misaligned pointers, a bad cache, max_q over 256, sizes outside hq_kv_attend's ranges,
 * q_start == NULL with total_q not a multiple of seqs.  Asynchronous, allocates nothing, may be captured. */
int hq_kv_accept(const hq_kv_cache *cache, const hq_kv_accept_args *args, hq_stream_t stream);

/* Softmax attention within packed prompts, on queries, keys and values as they are: what a model computes for a whole
 * prompt beside appending it to the cache.  Sequence b is rows start[b] .. start[b + 1] - 1 of q, k and v; query i of
 * it sees its tokens up to i (all of them when causal == 0), and with window > 0 only the last `window` of those up to
 * i.  Scores are scale q.k, then softcap tanh(score / softcap) when softcap > 0.  Query head j reads KV head
 * j / (q_heads / heads).  Types: bf16; 128 values a head.  Products are bf16 x bf16 into binary32; the softmax's
 * weights enter the second one as bf16, each off by at most 2^-8 of itself; scores, maxima, sums and outputs are
 * binary32, and a capped score is off by up to 2^-21 of softcap more.  A value that a row does not see does not reach it, whatever it holds. */
typedef struct {
  const void *q, *k, *v;     /* DEVICE, 16-byte aligned: value c of head j of row i at q[i q_stride[0] + j q_stride[1] + c] */
  void *out;                 /* DEVICE, [rows][q_heads][128], 16-byte aligned                       */
  int32_t dtype, out_dtype;  /* dtype: HQ_BF16                                                      */
  int64_t q_stride[2], k_stride[2], v_stride[2];  /* in values, multiples of 8; of k and v rows: 0 to
                                2^23 - 8.  Those of one row or one head are not looked at              */
  uint64_t rows;
  uint32_t q_heads, heads;   /* q_heads a multiple of heads                                         */
  uint32_t seqs;
  const int32_t *start;      /* DEVICE, seqs + 1 offsets that do not decrease (cut to [0, rows])        */
  float scale, softcap;
  int32_t causal;
  uint32_t window;           /* 0: none                                                             */
} hq_attend_prompt_args;
/* Asynchronous, allocates nothing, may be captured.  HQ_ERR_INVALID_ARG: null or misaligned pointers, strides outside
 * their ranges, another dtype, sizes outside their ranges (2^30 rows, 2^28 rows times query heads, 2^31 - 1 sequences), a scale
 * or softcap as hq_kv_attend's.  Rows of `out` that no sequence names are not written. */
int hq_attend_prompt(const hq_attend_prompt_args *args, hq_stream_t stream);

/* Eviction by accumulated weight.  Of each (sequence, head)'s n tokens, m = min(n, budget) stay: the first
 * `sink`, the last `recent`, and of the others those of most weight (ties to the lowest index; NaN counts
 * least).  They move, in order, to tokens 0..m-1 of the pages of dst_table, which must not be pages that
 * any table of the call reads; slots past m are not written.  A token of an absent page that stays (as
 * one of the first or last, or within the budget) becomes one that takes no part: zeros, its K scales -0. */
typedef struct {
  const int32_t *table;      /* DEVICE, [seqs][table_width]                                */
  const int32_t *lens;       /* DEVICE, [seqs]                                             */
  const float *weights;      /* DEVICE, as hq_kv_attend's                                  */
  uint64_t weights_stride;
  uint32_t seqs, table_width;
  uint32_t max_len;          /* most tokens of a sequence, at most weights_stride; a larger
                                length counts as this: tokens past it are not kept         */
  uint32_t budget, sink, recent;   /* sink + recent <= budget <= dst_width * page           */
  const int32_t *dst_table;  /* DEVICE, [seqs][dst_width]                                  */
  uint32_t dst_width;
  int32_t *kept;             /* DEVICE, [seqs][heads][budget]: indices that stay, then -1  */
  int32_t *new_lens;         /* DEVICE, [seqs]: m                                          */
  float *new_weights;        /* DEVICE or NULL, [seqs][heads][budget]: their weights, then 0 */
} hq_kv_evict_args;
int hq_kv_evict(const hq_kv_cache *cache, const hq_kv_evict_args *args, hq_stream_t stream);

/* Diagnostic front half of the encoder at a fixed step (components 1 and 2 of "Methodology: the
 * HyperQuant pipeline", with component 4's dither when params->dither is set; the integer codes
 * before component 3's stripping): per-value integer lattice codes (int32;
 * E8 and A2 codes are twice the lattice point (A2 in stretched coordinates), D4 and Z codes are the
 * point) and per-tile bf16 scale bits (uint16).  codes: n values, scales: n / params->tile
 * values, both device buffers, 16-byte aligned.  params->step must be positive (a fixed step);
 * the dither flags apply as for hq_encode.  Asynchronous; non-finite tiles are reported through
 * hq_status.  HQ_ERR_INVALID_ARG for step <= 0, bad params or misaligned pointers. */
int hq_codes(const void *x, int32_t dtype, uint64_t n, const hq_params *params, int32_t *codes,
             uint16_t *scales, void *workspace, size_t workspace_bytes, hq_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* HQ_H_ */
