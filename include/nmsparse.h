/*
 * nmsparse.h -- N:M structured weight sparsity on AMD Instinct MI355X (gfx950).
 *
 * A C ABI over plain pointers and sizes.  Every device pointer is HIP device
 * memory owned by the caller; no entry point allocates device or host memory,
 * synchronises the caller's stream (nm_check_perm excepted, a debug aid) or
 * keeps state between calls beyond read-only caches of device properties
 * (CU count, LDS limit).  Streams are passed as `void*` holding a hipStream_t
 * (NULL = the legacy default stream).
 *
 * Notation.  W is R x K (rows = output features, K = the reduction axis).
 * An N:M pattern keeps N of every M consecutive weights along a row of W;
 * S = K*N/M survivors per row; b = ceil(log2 M) index bits per survivor.
 *
 * Sources.  "M:N sparsity on NVIDIA tensor cores" (COE-592 lecture 04-2):
 * the opening section defines the pattern (groups along rows, survivor
 * positions per group) and the survivors:block notation; section "Where this
 * sits among the three case studies" gives the storage format (survivors
 * pushed left, small per-survivor indices), the product rule (only the weight
 * operand is compressed; sparse times dense is dense) and the shape rule (the
 * reduction dimension a multiple of 16 for 16-bit types, other layers stay
 * dense); section "The recipe" gives the pruning rule (keep the largest
 * magnitudes).  "SHUFFLESPARSE" technical summary, section 2 and its item on
 * inference efficiency: y = (W Pi) x with the hardened permutation applied as
 * a precomputed index map on the input reads.
 *
 * Error behaviour.  Every entry point validates its arguments on the host
 * before any HIP call and returns a status; on failure nothing is enqueued
 * and nm_last_error() describes the problem.  NM_OK means the work was
 * enqueued on `stream` (asynchronous, stream-ordered); device-side faults
 * surface at the caller's next synchronisation.  No exception or abort
 * crosses this boundary.  Results are bitwise reproducible (no atomics).
 */
#ifndef NMSPARSE_H
#define NMSPARSE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  NM_OK = 0,
  NM_ERR_NULL = 1,         /* a required pointer is NULL                          */
  NM_ERR_SHAPE = 2,        /* R, K or T out of range; K % 16 (K % 32 for 8-bit W) or K % M non-zero */
  NM_ERR_UNSUPPORTED = 3,  /* (n, m) pair or dtype combination not provided       */
  NM_ERR_STRIDE = 4,       /* leading dimension smaller than the row width        */
  NM_ERR_ALIAS = 5,        /* output overlaps an input                            */
  NM_ERR_HIP = 6,          /* a HIP call failed (launch error, no device, ...)    */
  NM_ERR_ALIGN = 7         /* pointer or leading dimension misaligned (see below) */
} nm_status;

typedef enum { NM_F16 = 0, NM_BF16 = 1, NM_F32 = 2, NM_I8 = 3, NM_I32 = 4, NM_FP8 = 5 } nm_dtype;

/*
 * INT8 weights (NM_I8).  The 2:4 pattern is also offered for 8-bit integer
 * weights; the index stays 2 bits per stored value, so a group of four costs
 * 2*8 + 2*2 = 20 bits (37.5% below dense), and the reduction length must be a
 * multiple of 32 (COE-592 lecture 04-2, "M:N sparsity on NVIDIA tensor cores":
 * opening section, and section "Where this sits among the three case
 * studies").  With dtype NM_I8 every entry point below takes only (n, m) =
 * (2, 4) (else NM_ERR_UNSUPPORTED) and K % 32 == 0 (else NM_ERR_SHAPE); values
 * are one byte each; magnitude is |w| as an integer (-128 ranks above 127,
 * equal magnitudes go to the lower position); act is int8 and Y is int32
 * (out_dtype NM_I32, the only one), the exact integer product; leading
 * dimensions of int8 matrices (ldw, ldx) must be multiples of 16.
 * nm_spmm_perm does not take NM_I8 (NM_ERR_UNSUPPORTED).
 *
 * FP8 weights (NM_FP8, OCP E4M3: sign, 4 exponent bits with bias 7, 3
 * mantissa bits, no infinities, S.1111.111 is NaN).  The pages name 16-bit
 * and INT8 2:4 types only; an 8-bit float takes the one-byte layout and every
 * rule of NM_I8 above (2:4 only, K % 32, ldw and ldx multiples of 16, no
 * nm_spmm_perm), with these differences: magnitude is compared on the stored
 * pattern with the sign bit cleared (bits & 0x7F, so +x and -x tie, equal keys
 * going to the lower position), act is E4M3 and Y is fp32 (out_dtype NM_F32,
 * the only one).  The hardware's fp8 sparse multiply-accumulate sums with
 * somewhat less than fp32 precision (relative error near 1e-4 of the result
 * at K = 2048); NaN inputs give NaN outputs.
 */

/* Version of this ABI (major * 100 + minor): 101 adds NM_I8 / NM_I32,
 * 102 adds NM_FP8; 200 replaces the process-wide nm_set_variant by the
 * per-call nm_spmm_variant and gives nm_spmm_perm a caller-owned workspace in
 * place of memory the library allocated; 201 adds the hybrid tiles
 * (nm_hybrid_*), the training products (nm_spmm_dx, nm_spmm_dw) and the
 * block / diagonal structures (nm_block_*, nm_diag_*).  Layer norm, the adapters
 * and cross entropy (nm_layernorm*, nm_adapter_*, nm_xent*), and the products
 * grouped by expert, the 4-bit format and the gradients' norm (nm_group_*, nm_mx_*,
 * nm_grad_*) only add entry points and came under 201. */
int nm_version(void);

/* Short fixed text for a status code (never NULL). */
const char* nm_status_string(int status);

/* Detail for the last failing call on this thread (empty string if none). */
const char* nm_last_error(void);

/*
 * Sizes of the packed format.  Pure host arithmetic, no device access.
 *   values_bytes  = R * S * 2            (values [R, S], same type as W; R * S for 8-bit W)
 *   idx_row_words = ceil(S * b / 32)     (uint32 words per row)
 *   idx_bytes     = R * idx_row_words * 4
 * Any output pointer may be NULL.  Same validation as nm_compress.
 *
 * Packed format (the canonical one every entry point reads and writes):
 *   values[r, g*N + j]  the j-th survivor of group g of row r, survivors of a
 *                       group in ascending position order, bits copied
 *                       unchanged from W;
 *   idx row r           an LSB-first bitstream: the in-group position (0..M-1)
 *                       of survivor s = g*N + j sits in bits [s*b, s*b + b);
 *                       stream bit i is bit (i % 32) of word (i / 32); words
 *                       are little-endian uint32, the tail is zero-padded.
 * With 2:4, one group of four 16-bit weights costs 2*16 + 2*2 = 36 bits (8-bit: 20)
 * (+ per-row padding to a whole word when S*b is not a multiple of 32).
 */
nm_status nm_packed_sizes(int64_t R, int64_t K, int n, int m, int dtype,
                          size_t* values_bytes, size_t* idx_bytes, int64_t* idx_row_words);

/*
 * Prune + pack (magnitude top-N of every M along the rows of W).
 *   W       device, [R, K] row-major, leading dimension ldw >= K (elements),
 *           dtype NM_F16, NM_BF16, NM_I8 or NM_FP8 (see above).
 *   values  device, [R, S] contiguous, same dtype (written).
 *   idx     device, [R, idx_row_words] uint32 contiguous (written, padding
 *           bits zero).
 * Selection: magnitude is compared on the stored 16-bit pattern with the sign
 * bit cleared (bits & 0x7FFF), so +0/-0 tie and +x/-x tie; the N largest keys
 * of a group are kept, equal keys going to the lower position.  Exactly N
 * slots are stored per group even when the group holds fewer non-zeros.
 * Supported (n, m): (2, 4), (1, 4), (1, 8).  K % 16 == 0 and K % m == 0.
 * Alignment: W, values and idx 16-byte aligned; ldw % 8 == 0.
 */
nm_status nm_compress(const void* W, int64_t R, int64_t K, int64_t ldw, int dtype, int n, int m,
                      void* values, uint32_t* idx, void* stream);

/*
 * Decompress: dense W_nm [R, K] (leading dimension ldw) with the survivors
 * back in place and zeros elsewhere.  Same format rules as nm_compress.
 */
nm_status nm_decompress(const void* values, const uint32_t* idx, int64_t R, int64_t K, int n,
                        int m, int dtype, void* W_out, int64_t ldw, void* stream);

/*
 * Sparse GEMM  Y = W_nm X,  X = act^T.
 *   values, idx  packed W (see nm_packed_sizes), dtype NM_F16, NM_BF16, NM_I8 or
 *                NM_FP8.
 *   act          device, [T, K] row-major (each token's K features contiguous),
 *                leading dimension ldx >= K, same dtype as values.
 *   Y            device, [T, R] row-major, leading dimension ldy >= R, i.e. the
 *                transpose of Y = W_nm X (the layout of a linear layer's output);
 *                out_dtype NM_F32 (default) or the input dtype (RNE rounded);
 *                NM_I32 for NM_I8 (exact); NM_F32 only for NM_FP8.
 *   Y[t, r] = sum_k W_nm[r, k] * act[t, k], products and sums in fp32.
 * Shapes: R >= 1, T >= 0 (T == 0 enqueues nothing), K >= 16, K % 16 == 0,
 * K % m == 0.  Alignment: every pointer 16-byte aligned, ldx % 8 == 0 (ldy
 * is free).  Y must not overlap values, idx or act (NM_ERR_ALIAS).
 */
nm_status nm_spmm(const void* values, const uint32_t* idx, int64_t R, int64_t K, int n, int m,
                  int dtype, const void* act, int64_t T, int64_t ldx, void* Y, int64_t ldy,
                  int out_dtype, void* stream);

/*
 * Permuted sparse GEMM  y = (W Pi) x:  Y[t, r] = sum_k W_nm[r, k] * act[t, perm[k]]
 * (SHUFFLESPARSE technical summary, section 2, and the inference-efficiency
 * item of its technical components: the hardened permutation is a
 * precomputed index map applied while the GEMM reads its input).
 *   perm       device int32 [K], a permutation of 0..K-1 (precondition, not
 *              checked on the hot path; an entry outside [0, K) is clamped into
 *              the row, so it gives a wrong value for its column, never an
 *              out-of-bounds access).
 *   workspace  device memory owned by the caller, or NULL; workspace_bytes its
 *              size.  With at least nm_spmm_perm_workspace_size() bytes, one
 *              gather pass writes X' = act[:, perm] there and the fastest
 *              unpermuted kernel multiplies X' (the workspace is overwritten;
 *              calls that share a workspace must be ordered on one stream).
 *              Otherwise the kernel applies the map as it reads act: the few-
 *              token kernel (T <= 16), the resident-tile kernel (2:4,
 *              K % 256 == 0, K <= 4096: each tile of tokens is staged through
 *              the map once, in LDS, and every weight row streams past it) or
 *              the generic kernel (correct, slower).  Nothing is allocated.
 *              16-byte aligned; must not overlap any other argument
 *              (NM_ERR_ALIAS).
 * All other arguments as nm_spmm.
 */
nm_status nm_spmm_perm(const void* values, const uint32_t* idx, int64_t R, int64_t K, int n, int m,
                       int dtype, const void* act, int64_t T, int64_t ldx, const int32_t* perm,
                       void* Y, int64_t ldy, int out_dtype, void* workspace, size_t workspace_bytes,
                       void* stream);

/*
 * Workspace bytes nm_spmm_perm uses for its gather pass on this shape (T * K *
 * 2 for 16-bit weights with K % 8 == 0, K <= 65536 and T > 16; 0 when the shape
 * always applies the map inside the kernel).  Pure host arithmetic; same
 * format checks as nm_packed_sizes.
 */
nm_status nm_spmm_perm_workspace_size(int64_t R, int64_t K, int64_t T, int n, int m, int dtype,
                                      size_t* bytes);

/*
 * nm_spmm_perm for callers that cannot allocate memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation): the same
 * product, with the gather pass's workspace taken from a device array the
 * library holds on each GPU it runs on, 32 MiB (33554432 bytes), from first
 * use until the process ends.  Shapes whose workspace (nm_spmm_perm_workspace_size)
 * exceeds 32 MiB are refused with NM_ERR_SHAPE before anything is enqueued;
 * shapes with no gather pass (T <= 16, ...) use no workspace.  Every call on
 * one GPU shares that GPU's array: calls that overlap in time on one GPU (on
 * different streams, or from different threads) race and give wrong results;
 * calls ordered on one stream are safe.  Allocates nothing and synchronises
 * nothing; arguments and errors as nm_spmm_perm.
 */
nm_status nm_spmm_perm_static(const void* values, const uint32_t* idx, int64_t R, int64_t K, int n,
                              int m, int dtype, const void* act, int64_t T, int64_t ldx,
                              const int32_t* perm, void* Y, int64_t ldy, int out_dtype, void* stream);

/*
 * Host-side check that perm is a permutation of 0..K-1 (copies perm to the
 * host and synchronises `stream`).  NM_ERR_SHAPE if it is not.  Debug aid.
 */
nm_status nm_check_perm(const int32_t* perm, int64_t K, void* stream);

/*
 * nm_spmm (perm NULL; workspace ignored) or nm_spmm_perm (perm non-NULL) with
 * the kernel family named by the call (tests and ablations; no state is kept;
 * with a large enough workspace the named family multiplies the gathered X'):
 *   0  choose by shape (what nm_spmm / nm_spmm_perm do)
 *   1  generic tiled kernel (LDS-staged operands, any shape, any map)
 *   2  register-prefetch pipelined kernel (K % 64 == 0, T >= 64, R >= 128;
 *      not permuted)
 *   3  all-LDS direct-load kernel with 256 x 128 tiles (2:4; K % 128 == 0,
 *      T >= 128, R >= 256; not permuted)
 *   4  few-token kernel (T <= 16, K <= 4096)
 *   5  resident-tile kernel (2:4; K % 256 == 0, K <= 4096)
 *   6  all-LDS direct-load kernel with 128 x 64 tiles (1:4 and 1:8;
 *      K % 256 == 0, T >= 64, R >= 128; not permuted)
 * For 8-bit weights there are two: the LDS-staged kernel (whole 256 x 128 tiles,
 * K % 128 == 0) and, for variant 1 or any other shape, a kernel that loads
 * its operands straight into registers.
 * A named family that does not take the shape falls back to the choice by
 * shape.  Every family computes the same product; all but 4 and 6 add the
 * 64-wide K steps in the same order and give the same bits (4 splits K over
 * waves, 6 sums the even and the odd K steps apart and then adds the two:
 * the same result within the fp32 summation bound, and the same bits on
 * every run).
 * NM_ERR_UNSUPPORTED outside 0..6.
 */
nm_status nm_spmm_variant(const void* values, const uint32_t* idx, int64_t R, int64_t K, int n, int m,
                          int dtype, const void* act, int64_t T, int64_t ldx, const int32_t* perm,
                          void* Y, int64_t ldy, int out_dtype, void* workspace, size_t workspace_bytes,
                          int variant, void* stream);

/*
 * Training-side products of an N:M layer.  Source: COE-592 lecture 04-2,
 * "M:N sparsity on NVIDIA tensor cores", section "The recipe", step 3 (the
 * pruned network is retrained with the zeros held fixed, so the pattern
 * survives), and the RNM-TD3 abstract of thelatestinai.com's "Structured
 * Sparsity" cards (row-wise N:M sparsity kept throughout training).  With the
 * forward product Yt[t, r] = sum_k W_nm[r, k] act[t, k] (nm_spmm) and
 * G = dL/dYt, the gradient of the output in Yt's layout:
 *
 * nm_spmm_dx: dX[t, k] = sum_r G[t, r] W_nm[r, k]  (dX = G W_nm, the gradient
 *   of act).
 *   values, idx  packed W (nm_compress), NM_F16 or NM_BF16, patterns as nm_spmm.
 *   G            device [T, R] row-major, ldg >= R, ldg % 8 == 0, dtype of W.
 *   dX           device [T, K] row-major, lddx >= K; out_dtype NM_F32 or the
 *                input dtype (RNE rounded).  Overwritten; with R == 0 it is
 *                filled with zeros.
 *   The reduction runs over R, across W's rows, so the N:M groups give the
 *   matrix cores nothing to skip: the product runs at the dense rate and reads
 *   the packed weights.  Sums in fp32.
 *
 * nm_spmm_dw: dW[r, s] = sum_t G[t, r] act[t, k(r, s)], the gradient of every
 *   stored survivor s of row r (k(r, s) the column it came from), in the
 *   packed values' layout [R, S] (S = K*n/m), contiguous.  Dropped weights are
 *   held at zero and get no gradient; a stored slot that holds a zero is a
 *   weight like any other and gets its gradient.
 *   idx          the packed W's index words (the values are not read).
 *   G            [T, R], ldg as above;  act  [T, K], ldx >= K, ldx % 8 == 0.
 *   dW           device [R, S], out_dtype NM_F32 or the input dtype.
 *                Overwritten; with T == 0 it is filled with zeros.
 *
 * Both: R % 8 == 0 and K % 32 == 0 besides nm_spmm's format rules
 * (NM_ERR_SHAPE); every pointer 16-byte aligned; the output must not overlap
 * an input (NM_ERR_ALIAS); stream-ordered, nothing allocated or synchronised.
 * NM_ERR_UNSUPPORTED for 8-bit weights; NM_ERR_SHAPE for a packed W or index
 * array of 4 GiB or more, a 128-token block of G of 4 GiB or more (dX), or G
 * or act of 4 GiB or more (dW).
 */
nm_status nm_spmm_dx(const void* values, const uint32_t* idx, int64_t R, int64_t K, int n, int m, int dtype,
                     const void* G, int64_t T, int64_t ldg, void* dX, int64_t lddx, int out_dtype, void* stream);
nm_status nm_spmm_dw(const uint32_t* idx, int64_t R, int64_t K, int n, int m, int dtype, const void* G, int64_t T,
                     int64_t ldg, const void* act, int64_t ldx, void* dW, int out_dtype, void* stream);

/*
 * Hybrid dense / 2:4 weight tiles.  Source: thelatestinai.com "Structured
 * Sparsity" topic cards, the PATCH abstract: the weight matrix is cut into
 * tiles and each tile is either kept dense or made 2:4 sparse (the choice is
 * a learned mask, an input here), so the zero fraction can be set anywhere
 * between 0 and 50%; a 2:4 tile is pruned with the nm_compress rule.
 *
 * Tiles are tile_rows x tile_cols blocks on a regular grid (both positive
 * multiples of 64; tile_cols divides K; at most 8192 tile-columns; the last
 * tile-row may be shorter when tile_rows does not divide R).  RB = ceil(R /
 * tile_rows) tile-rows, KB = K / tile_cols tile-columns.
 *   flags[b*KB + j]  host uint8: 1 keeps tile (b, j) dense, 0 makes it 2:4.
 * Packed layout: a row stores its tiles in column order, a dense tile as its
 * tile_cols values (bits unchanged), a 2:4 tile as its tile_cols/2 survivors
 * (the nm_compress format on the tile's columns).  Within every block of 16
 * columns a dense tile stores the values at positions 0 and 1 of the block's
 * four groups of four, then those at positions 2 and 3 (block columns 0 1 4 5
 * 8 9 12 13, then 2 3 6 7 10 11 14 15), the operand order of the two fixed-
 * position 2:4 products a dense step takes.  The row's index bytes are
 * the 2:4 tiles' LSB-first 2-bit streams, tile_cols/8 bytes each, in the
 * same order.  The rows of tile-row b share one length, Lv[b] values and
 * Li[b] index bytes; rows follow each other and tile-rows follow each other,
 * in `values` (dtype of W) and in `idx` (bytes).
 *
 * nm_hybrid_layout (host only, no device access) writes the layout tables:
 *   tile_meta  [RB*KB*2] int64: per tile, the offset of its first value in
 *              the first row of its tile-row (elements into values) and of its
 *              first index byte (bytes into idx), or -1 for a dense tile;
 *   row_meta   [RB*4] int64: per tile-row, Lv, Li and the offsets of its
 *              first value and first index byte;
 *   values_count, idx_bytes  the packed sizes (elements, bytes); the index
 *              array is zero-padded to a multiple of 16 bytes.
 * Any output may be NULL (a size query).  NM_ERR_SHAPE for a bad grid, a flag
 * other than 0 or 1, or packed values or index bytes of 2 GiB or more.
 *
 * nm_hybrid_compress packs W (device, [R, K] row-major, ldw >= K, ldw % 8 ==
 * 0; NM_F16 or NM_BF16) into values / idx (device, caller-allocated with the
 * sizes above); tile_meta / row_meta are the tables of nm_hybrid_layout for
 * the same flags, copied to the device by the caller (8-byte aligned).  idx
 * may be NULL when idx_bytes is 0 (every tile dense).
 *
 * nm_hybrid_spmm computes Y[t, r] = sum_k W_hat[r, k] act[t, k] (fp32
 * accumulation) where W_hat is W with every 2:4 tile pruned: act [T, K]
 * (K <= ldx <= 2^22, ldx % 8 == 0), Y [T, R] (ldy >= R), out_dtype NM_F32 or the
 * input dtype.  On a dense tile each K step runs dense MFMAs, on a 2:4 tile
 * the sparse MFMA.  Layout tables that do not match the packed arrays give
 * wrong values, but every weight access stays inside values_count /
 * idx_bytes.  Same pointer, alignment and alias rules as nm_spmm; nothing is
 * allocated and the stream is not synchronised.
 */
nm_status nm_hybrid_layout(int64_t R, int64_t K, int64_t tile_rows, int64_t tile_cols, const uint8_t* flags,
                           int64_t* tile_meta, int64_t* row_meta, int64_t* values_count, int64_t* idx_bytes);

nm_status nm_hybrid_compress(const void* W, int64_t R, int64_t K, int64_t ldw, int dtype, int64_t tile_rows,
                             int64_t tile_cols, const int64_t* tile_meta, const int64_t* row_meta,
                             int64_t values_count, int64_t idx_bytes, void* values, uint8_t* idx, void* stream);

nm_status nm_hybrid_spmm(const void* values, const uint8_t* idx, const int64_t* tile_meta, const int64_t* row_meta,
                         int64_t R, int64_t K, int64_t tile_rows, int64_t tile_cols, int64_t values_count,
                         int64_t idx_bytes, int dtype, const void* act, int64_t T, int64_t ldx, void* Y,
                         int64_t ldy, int out_dtype, void* stream);

/*
 * The column permutation on two other host structures.  Source: searcharxiv
 * author page, the SHUFFLESPARSE abstract (one learned permutation applied the
 * same way to block, N:M and diagonal structures) and the DynaDiag abstract
 * (a diagonal pattern); gist.science "Technische Samenvatting: SHUFFLESPARSE",
 * section "2. Methodologie" (y = (W Pi) x, W following a fixed structured
 * pattern) and the item "Efficiëntie bij Inferentie" (the hardened Pi as a
 * precomputed index map on the structured kernel's input reads).  The pages
 * name the structures only; the geometry and storage below are this
 * library's.  Both products read act through perm the way nm_spmm_perm does,
 * Y[t, r] = sum_k W[r, k] act[t, perm[k]] (perm NULL: act as it is; an entry
 * outside [0, K) reads column K - 1), with fp32 accumulation; 16-bit weights
 * (NM_F16, NM_BF16) and activations of the same type; Y [T, R] row-major,
 * ldy >= R, out_dtype NM_F32 or the input dtype (RNE).  Every pointer 16-byte
 * aligned, ldx and ldw multiples of 8, outputs not overlapping inputs
 * (NM_ERR_ALIAS); stream-ordered, nothing allocated or synchronised.  act of
 * 4 GiB or more is NM_ERR_SHAPE.
 *
 * Block-sparse: W [R, K] (R and K multiples of 32) cut into 32 x 32 blocks,
 * each kept whole or dropped.  Stored as block-sparse rows:
 *   row_ptr  int32 [R/32 + 1]: the kept blocks of block-row b are entries
 *            row_ptr[b] .. row_ptr[b+1]-1;
 *   col      int32 [nnzb]: their block-columns, ascending within a row;
 *   values   [nnzb][32][32]: each kept block row-major, bits of W unchanged.
 * nm_block_structure (host only, no device access) builds row_ptr and col
 *   from mask[(R/32) * (K/32)] (host uint8, 1 keeps block (b, c) at
 *   b*(K/32) + c); any output may be NULL (a size query); NM_ERR_SHAPE for a
 *   bad shape or a mask entry other than 0 or 1.
 * nm_block_compress copies the kept blocks of W (device, [R, K], ldw >= K)
 *   into values (device, nnzb*2048 bytes); row_ptr and col on the device.
 * nm_block_spmm: Y[t, r] = sum over kept blocks (r/32, c) of
 *   sum_j values[blk][r%32][j] * act[t, perm[32c + j]]; act [T, K], ldx >= K;
 *   perm int32 [K] or NULL.  Runs the kept blocks on the dense matrix cores.
 * Entries of row_ptr or col outside their range are clamped on the device: a
 * malformed structure gives wrong values but no access outside the arrays.
 *
 * Diagonal-sparse: W [R, K] non-zero only on D wrap-around diagonals with
 * distinct offsets o_d in [0, K) (offsets int32 [D], any order; others are
 * reduced mod K, and a repeated offset adds its diagonal twice): row r of
 * diagonal d sits at column (r + o_d) mod K.  Stored as values [D][R],
 * values[d][r] = W[r, (r + o_d) mod K].  K % 8 == 0, K <= 1792, 0 <= D <= K,
 * values below 4 GiB.
 * nm_diag_compress gathers values from W (device, [R, K], ldw >= K).
 * nm_diag_spmm: Y[t, r] = sum_d values[d][r] * act[t, perm[(r + o_d) mod K]].
 *   Every row reads a different activation column per diagonal, so the
 *   product runs on the vector ALUs (fp32 FMA), not the matrix cores.
 */
nm_status nm_block_structure(int64_t R, int64_t K, const uint8_t* mask, int32_t* row_ptr, int32_t* col,
                             int64_t* nnzb);
nm_status nm_block_compress(const void* W, int64_t R, int64_t K, int64_t ldw, int dtype, const int32_t* row_ptr,
                            const int32_t* col, int64_t nnzb, void* values, void* stream);
nm_status nm_block_spmm(const void* values, const int32_t* row_ptr, const int32_t* col, int64_t nnzb, int64_t R,
                        int64_t K, int dtype, const void* act, int64_t T, int64_t ldx, const int32_t* perm,
                        void* Y, int64_t ldy, int out_dtype, void* stream);
nm_status nm_diag_compress(const void* W, int64_t R, int64_t K, int64_t ldw, int dtype, const int32_t* offsets,
                           int64_t D, void* values, void* stream);
nm_status nm_diag_spmm(const void* values, const int32_t* offsets, int64_t D, int64_t R, int64_t K, int dtype,
                       const void* act, int64_t T, int64_t ldx, const int32_t* perm, void* Y, int64_t ldy,
                       int out_dtype, void* stream);

/*
 * Layer norm over the H features of each of T tokens: with mu the mean, var the
 * mean of (x - mu)^2 and rstd = (var + eps)^(-1/2) of a row,
 *   nm_layernorm:     xh = (x - mu) rstd,  y = xh * weight + bias;
 *   nm_layernorm_bwd: with p = dy * weight,
 *                     dx = rstd (p - mean(p) - xh mean(p xh)),
 *                     dw[h] = sum_t dy xh,  db[h] = sum_t dy.
 *   x, y, dy, dx   device [T, H] row-major with leading dimensions >= H,
 *                  dtype NM_F16, NM_BF16 or NM_F32 (one for all); 1 <= H <= 2^24.
 *   weight, bias   device [H] of dtype, or NULL (ones, zeros).
 *   mean, rstd     device fp32 [T]; written by the forward pass (both NULL: not
 *                  kept), read by the backward pass.
 *   dw, db         device [H], out_dtype NM_F32 or dtype, or NULL (not wanted);
 *                  T == 0 writes zeros.
 *   workspace      device, nm_layernorm_bwd_workspace_size bytes, 16-byte
 *                  aligned; only needed for dw or db.
 * Statistics and sums are fp32 (the variance taken about the mean), outputs are
 * rounded once.  Pointers need the alignment of their element only, leading
 * dimensions are free.  Outputs must not overlap inputs or each other
 * (NM_ERR_ALIAS).  An x that holds Inf or NaN gives NaN in its own row of y and dx
 * and in all of dw, not in db; a dy that does, in its own row of dx (any weight not
 * zero) and in its columns of dw and db.
 */
nm_status nm_layernorm(const void* x, int64_t T, int64_t H, int64_t ldx, int dtype, const void* weight,
                       const void* bias, float eps, void* y, int64_t ldy, float* mean, float* rstd, void* stream);
nm_status nm_layernorm_bwd_workspace_size(int64_t T, int64_t H, size_t* bytes);
nm_status nm_layernorm_bwd(const void* dy, int64_t ldg, const void* x, int64_t ldx, int64_t T, int64_t H, int dtype,
                           const float* mean, const float* rstd, const void* weight, void* dx, int64_t lddx, void* dw,
                           void* db, int out_dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Low-rank adapters of many requests beside a shared N:M projection.  Token t
 * names adapter a = adapter[t]; an entry outside [0, adapters) (-1, say) means
 * the shared projection alone.
 *   nm_adapter_spmm:      xa[t] = A_a act[t],
 *                         Y[t] = W_nm act[t] + scale_a B_a xa[t];
 *   nm_adapter_spmm_bwd:  with G = dL/dY, W_nm frozen, u[t] = scale_a B_a^T G[t],
 *                         dX[t] = W_nm^T G[t] + A_a^T u[t],
 *                         dA_a = sum over a's tokens of u[t] act[t]^T,
 *                         dB_a = scale_a sum over a's tokens of G[t] xa[t]^T.
 *   values, idx, act, Y, G, dX   as nm_spmm and nm_spmm_dx (16-bit weights; the
 *              backward pass with their R % 8 and K % 32); Y and dX in
 *              out_dtype NM_F32 or the input dtype.
 *   adapter    device int32 [T], in any order; requests whose tokens are
 *              adjacent are the fastest.
 *   A          device [adapters, rank, K],  B  device [adapters, R, rank], dtype
 *              of the weight, contiguous; 1 <= rank <= 256, 0 <= adapters <=
 *              65535.  Adapters of several ranks are padded with zeros.
 *   scale      device fp32 [adapters].
 *   xa         device fp32 [T, rank]: written by the forward pass (zeros for a
 *              token without an adapter), read by the backward pass.
 *   dX         may be NULL (not wanted);  dA, dB  device fp32, shaped as A and B,
 *              overwritten: an adapter without tokens gets zeros.
 *   workspace  device, the bytes of the matching _workspace_size, 16-byte aligned.
 * xa and u stay fp32; between the two low-rank products they enter the matrix
 * cores as three bf16 parts, which hold their 24 bits.  Inf or NaN in one token
 * or adapter reaches the outputs of that token or adapter only (there an Inf may
 * turn to NaN: it meets the parts that are zero).  Equal calls give equal bits; a
 * token's last bits can change with its neighbours (the kernel goes by T, and the
 * term is summed onto the product where a tile's tokens share one adapter, apart
 * from it where they do not).
 * T <= 2^24, R and K <= 2^22.  Pointers 16-byte aligned (adapter, scale: 4),
 * ldx and ldg multiples of 8 below 2^24; outputs and workspace must not overlap anything
 * (NM_ERR_ALIAS).  Stream-ordered; nothing is allocated or synchronised.
 */
nm_status nm_adapter_spmm_workspace_size(int64_t R, int64_t K, int n, int m, int dtype, int64_t T, int64_t ldx,
                                         int64_t adapters, int64_t rank, int out_dtype, size_t* bytes);
nm_status nm_adapter_spmm(const void* values, const uint32_t* idx, int64_t R, int64_t K, int n, int m, int dtype,
                          const void* act, int64_t T, int64_t ldx, const int32_t* adapter, const void* A,
                          const void* B, const float* scale, int64_t adapters, int64_t rank, float* xa, void* Y,
                          int64_t ldy, int out_dtype, void* workspace, size_t workspace_bytes, void* stream);
nm_status nm_adapter_spmm_bwd_workspace_size(int64_t R, int64_t K, int n, int m, int dtype, int64_t T,
                                             int64_t adapters, int64_t rank, int out_dtype, size_t* bytes);
nm_status nm_adapter_spmm_bwd(const void* values, const uint32_t* idx, int64_t R, int64_t K, int n, int m, int dtype,
                              const void* G, int64_t T, int64_t ldg, const void* act, int64_t ldx, const float* xa,
                              const int32_t* adapter, const void* A, const void* B, const float* scale,
                              int64_t adapters, int64_t rank, void* dX, int64_t lddx, float* dA, float* dB,
                              int out_dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Softmax cross entropy over a large vocabulary, the logits never kept: the
 * head and the loss of a model whose layers are retrained (the head itself
 * stays dense).  With l[t][v] = sum_h x[t][h] w[v][h]:
 *   nm_xent:      lse[t] = log sum_v exp l[t][v],  loss[t] = lse[t] - l[t][labels[t]];
 *   nm_xent_bwd:  d[t][v] = dloss[t] (exp(l[t][v] - lse[t]) - [v == labels[t]]),
 *                 dx[t][h] = sum_v d[t][v] w[v][h],  dw[v][h] = sum_t d[t][v] x[t][h].
 *   x, w       device [T, H] and [V, H] row-major, NM_F16 or NM_BF16, H % 8 == 0,
 *              ldx, ldw >= H and multiples of 8, below 2^23.
 *   labels     device int32 [T]; a label outside [0, V) (-100, say) is ignored:
 *              loss 0, no gradient, lse still written.
 *   loss, lse  device fp32 [T];  dloss  device fp32 [T], dL/dloss (1 over the
 *              count of labels for a mean).
 *   dx, dw     device, NM_F32 or the input dtype each (dx_dtype, dw_dtype),
 *              lddx, lddw >= H and multiples of 4; either may be NULL (not
 *              wanted).  T == 0 writes zeros to dw.
 *   workspace  device, the bytes of the matching _workspace_size (the backward
 *              pass: for the same choice of dx and dw), 16-byte aligned.
 * Logits, statistics and sums are fp32.  The backward pass walks the vocabulary
 * in pieces and computes the logits again; softmax - onehot (for dw: times dloss
 * over its largest magnitude) enters its two products in the inputs' 16-bit type:
 * rounded once for a 16-bit dx or dw (relative 2^-8 in bf16, 2^-11 in fp16 an
 * element), in two parts that add up to it to 2^-16 or 2^-22 for an fp32 one,
 * which costs that product twice.  fp16 operands are held in steps of 2^-38, so
 * below 2^-28 an element has an absolute error of up to 2^-39 instead: for dw that
 * is 2^-39 of the largest |dloss|, and tokens whose dloss is far below the largest
 * keep fewer bits there (not in dx, and not in bf16, which has fp32's range).
 * dloss itself multiplies the fp32 results.
 * T <= 2^22, V <= 2^24, H <= 2^20 and ceil(T / 16) ceil(V / 128) <= 2^26 (T x V up
 * to 2^37; NM_ERR_SHAPE past it).  Matrices and workspace 16-byte aligned, vectors 4;
 * outputs and workspace must not overlap anything (NM_ERR_ALIAS).
 * Stream-ordered; nothing is allocated or synchronised.
 */
nm_status nm_xent_workspace_size(int64_t T, int64_t V, int64_t H, int dtype, size_t* bytes);
nm_status nm_xent(const void* x, int64_t T, int64_t H, int64_t ldx, const void* w, int64_t V, int64_t ldw, int dtype,
                  const int32_t* labels, float* loss, float* lse, void* workspace, size_t workspace_bytes,
                  void* stream);
nm_status nm_xent_bwd_workspace_size(int64_t T, int64_t V, int64_t H, int dtype, int need_dx, int need_dw,
                                     size_t* bytes);
nm_status nm_xent_bwd(const void* x, int64_t T, int64_t H, int64_t ldx, const void* w, int64_t V, int64_t ldw,
                      int dtype, const int32_t* labels, const float* lse, const float* dloss, void* dx, int64_t lddx,
                      int dx_dtype, void* dw, int64_t lddw, int dw_dtype, void* workspace, size_t workspace_bytes,
                      void* stream);

/*
 * Products grouped by expert: a layer of E experts, each with its own packed N:M
 * weight of R x K, over tokens ordered by expert.  Expert e owns the rows
 * offsets[e] <= t < offsets[e+1] of act, Y, G and dX:
 *   nm_group_spmm:     Y[t][r]  = sum_k W_e[r][k] act[t][k]           (nm_spmm),
 *   nm_group_spmm_dx:  dX[t][k] = sum_r G[t][r] W_e[r][k]             (nm_spmm_dx),
 *   nm_group_spmm_dw:  dW[e][r][s] = sum_t G[t][r] act[t][k(r, s)]    (nm_spmm_dw).
 *   values, idx   E packed weights one after the other (each as nm_packed_sizes
 *                 says), 16-bit types;  dW  E packed gradients likewise.
 *   offsets       device int32 [E + 1], ascending, 0 <= offsets[0], offsets[E] <=
 *                 T; read on the device, so a captured graph follows them.  An
 *                 expert may own no rows (its dW is zeros).  Rows before
 *                 offsets[0] and from offsets[E] on belong to none: they are not
 *                 read, and stay as they were in Y and dX.  Offsets that break the
 *                 rule are clamped into [0, T] and to ascend one by one: wrong
 *                 values, but no access outside the arrays.
 *   act, Y, G, dX as nm_spmm and nm_spmm_dx (ldx, ldg below 2^23); out_dtype NM_F32
 *                 or the input dtype.  dX and dW need R % 8 == 0 and K % 32 == 0.
 *   workspace     device, the bytes of the matching _workspace_size, 16-byte aligned.
 * Products and sums are fp32, outputs rounded once.  Equal calls give equal bits; the
 * kernel, and the shares a long reduction of few tiles is summed in, go by the sizes,
 * so a token's last bits can change with T and E.  Inf
 * or NaN in one row reaches the outputs of its expert's row (dW: of its expert) only.
 * 1 <= E <= 65535, T <= 2^24, R and K <= 2^22; NM_ERR_SHAPE as in nm_spmm_dx and
 * nm_spmm_dw for one expert's arrays, and for T x ldg or T x ldx of 4 GiB in dW.
 * Outputs and workspace must not overlap anything (NM_ERR_ALIAS).  Stream-ordered;
 * nothing is allocated or synchronised.
 */
nm_status nm_group_spmm_workspace_size(int64_t E, int64_t R, int64_t K, int n, int m, int dtype, int64_t T,
                                       int out_dtype, size_t* bytes);
nm_status nm_group_spmm(const void* values, const uint32_t* idx, int64_t E, int64_t R, int64_t K, int n, int m,
                        int dtype, const void* act, int64_t T, int64_t ldx, const int32_t* offsets, void* Y,
                        int64_t ldy, int out_dtype, void* workspace, size_t workspace_bytes, void* stream);
nm_status nm_group_spmm_dx_workspace_size(int64_t E, int64_t R, int64_t K, int64_t T, size_t* bytes);
nm_status nm_group_spmm_dx(const void* values, const uint32_t* idx, int64_t E, int64_t R, int64_t K, int n, int m,
                           int dtype, const void* G, int64_t T, int64_t ldg, const int32_t* offsets, void* dX,
                           int64_t lddx, int out_dtype, void* workspace, size_t workspace_bytes, void* stream);
nm_status nm_group_spmm_dw_workspace_size(int64_t E, int64_t R, int64_t K, int n, int m, int64_t T, size_t* bytes);
nm_status nm_group_spmm_dw(const uint32_t* idx, int64_t E, int64_t R, int64_t K, int n, int m, int dtype, const void* G,
                           int64_t T, int64_t ldg, const void* act, int64_t ldx, const int32_t* offsets, void* dW,
                           int out_dtype, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Microscaled 4-bit floats: a row's values in blocks of 32, each value a sign and
 * one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (E2M1) times the block's power of two (E8M0):
 * 4.25 bits a value.
 *   q      [T][K/2] bytes: value 2i of a row in the low four bits of byte i, value
 *          2i + 1 in the high four (bit 3 the sign, bits 0..2 the magnitude's number
 *          in the list above);
 *   scale  [ceil(K/256)][T][8] bytes: byte b of a block means 2^(b - 127), 255 NaN;
 *          block i of row t is scale[i / 8][t][i % 8].  The eight bytes of a row's
 *          256 columns lie together and the rows after one another (a product's tile
 *          then reads one run); those past K in the last panel are written as 0 and
 *          not looked at.
 * nm_mx_quantize: the exponent of a block is that of its largest magnitude less 2
 *   (not below 2^-127; a block of zeros has byte 0), each value goes to the nearest
 *   representable one, ties to the even mantissa, magnitudes above 6 in the block's
 *   scale to 6.  A block that holds Inf or NaN becomes NaN.
 *   x      device [T, K] row-major, ldx >= K, NM_F16, NM_BF16 or NM_F32, aligned to
 *          its element; K % 32 == 0.
 * nm_mx_dequantize: y [T, K] (ldy >= K; NM_F16, NM_BF16 or NM_F32), the values,
 *   rounded once where the type does not hold them.
 * nm_mx_quantize_stack, nm_mx_dequantize_stack: the same of E matrices [R, K], q and scale one matrix after the other (as nm_mx_gemm reads E weights),
 *   x and y `stride` elements apart (x: any, 0 repeats one; y: no less than a matrix).
 *   E <= 2^24; E = 0 does nothing.  With E = 1 for one matrix of such a stack, whose
 *   scales begin on 8 bytes only.
 * nm_mx_gemm: Y[t][r] = sum_k x[t][k] w[r][k] of two quantised operands.
 *   wq, wscale  E weights of R rows one after the other, each as above (E = 1
 *               without offsets);  xq, xscale  T rows.
 *   offsets     device int32 [E + 1] or NULL: rows ordered by expert, as in
 *               nm_group_spmm.
 *   Y           device [T, R] row-major, ldy >= R, NM_F32, NM_F16 or NM_BF16.
 * Products are exact, sums fp32, outputs rounded once.  T <= 2^24, R and K <= 2^22,
 * an operand's scales below 4 GiB.  Device pointers 16-byte aligned (x, y: their
 * element; offsets: 4; the scales of nm_mx_gemm and of the _stack calls: 8); outputs
 * and workspace must not overlap anything (NM_ERR_ALIAS).  Stream-ordered; nothing is
 * allocated or synchronised.
 */
nm_status nm_mx_sizes(int64_t T, int64_t K, size_t* q_bytes, size_t* scale_bytes);
nm_status nm_mx_quantize(const void* x, int64_t T, int64_t K, int64_t ldx, int dtype, uint8_t* q, uint8_t* scale,
                         void* stream);
nm_status nm_mx_dequantize(const uint8_t* q, const uint8_t* scale, int64_t T, int64_t K, void* y, int64_t ldy,
                           int dtype, void* stream);
nm_status nm_mx_quantize_stack(const void* x, int64_t E, int64_t R, int64_t K, int64_t ldx, int64_t stride, int dtype,
                               uint8_t* q, uint8_t* scale, void* stream);
nm_status nm_mx_dequantize_stack(const uint8_t* q, const uint8_t* scale, int64_t E, int64_t R, int64_t K, void* y,
                                 int64_t ldy, int64_t stride, int dtype, void* stream);
nm_status nm_mx_gemm_workspace_size(int64_t E, int64_t R, int64_t K, int64_t T, int grouped, int out_dtype,
                                    size_t* bytes);
nm_status nm_mx_gemm(const uint8_t* wq, const uint8_t* wscale, int64_t E, int64_t R, int64_t K, const uint8_t* xq,
                     const uint8_t* xscale, int64_t T, const int32_t* offsets, void* Y, int64_t ldy, int out_dtype,
                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * Global norm of the gradients in many tensors, and their clipping:
 *   norm = (sum over every element of every tensor of g^2)^(1/2),
 *   out_i = g_i min(1, max_norm / (norm + eps)).
 *   grads, out  host arrays of `tensors` device addresses; counts, dtypes their
 *               numbers of elements and types (host; NM_F16, NM_BF16 or NM_F32, a
 *               list may mix them; out_i has the type of g_i).  Read before the call
 *               returns.  Tensors are contiguous and aligned to their element; an
 *               empty one (count 0) may be NULL.
 *   out         grads itself, or single addresses equal to theirs, scale in place.
 *   norm        device fp32 [1];  workspace  device, nm_grad_workspace_size bytes,
 *               16-byte aligned.
 * Squares are summed in 64 bits, so that neither large nor small gradients leave the
 * range, and the norm rounded to fp32.  Of an out_i three things are rounded: the
 * factor, taken in 64 bits, to fp32, its product with g_i to fp32, and that to the type
 * (half a step each).  A NaN anywhere makes norm and every out_i NaN; an
 * Inf makes norm Inf, itself NaN and everything else 0 (with max_norm Inf nothing is
 * scaled).  A norm + eps of 0 scales by 1.  Equal calls give equal bits.
 * tensors <= 16384, counts <= 2^36; max_norm >= 0 (Inf: no limit), eps >= 0
 * (NM_ERR_SHAPE).  Nothing written may overlap anything else (NM_ERR_ALIAS): a tensor
 * named twice in place among them.  Stream-ordered; nothing is allocated or synchronised.
 */
nm_status nm_grad_workspace_size(int64_t tensors, size_t* bytes);
nm_status nm_grad_norm(const void* const* grads, const int64_t* counts, const int* dtypes, int64_t tensors, float* norm,
                       void* workspace, size_t workspace_bytes, void* stream);
nm_status nm_grad_clip(const void* const* grads, const int64_t* counts, const int* dtypes, int64_t tensors,
                       double max_norm, double eps, void* const* out, float* norm, void* workspace,
                       size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NMSPARSE_H */
