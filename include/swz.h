/*
 * swz.h -- swizzled on-chip tile movement for AMD gfx950 (MI355X).
 *
 * C ABI of libswz.so.  Plain pointers and sizes only.  Every call that moves
 * data is asynchronous on the caller's HIP stream (a hipStream_t passed as
 * void*; NULL is the default stream), except swz_tune_tile_order, which
 * times conversions on it and waits for them.  Device buffers belong to the caller;
 * the library allocates no device memory and keeps no pointer after a call
 * returns.  Errors are negative return codes, detected on the host before
 * any launch; no call aborts or throws.  All calls are thread-safe.
 *
 * Calls: the swizzle map (swz_map, swz_map_batch); transposes and batched layout
 * conversions of 1-, 2- and 4-byte elements through swizzled, padded or
 * plain LDS tiles (swz_transpose, swz_convert_layout), with a per-shape
 * tile order (swz_set_tile_order, swz_get_tile_order, swz_tune_tile_order);
 * GEMM operand staging
 * into matrix-instruction fragments (swz_stage_operand, and both operands of
 * one GEMM at once: swz_stage_operands) and their consumer
 * (swz_gemm_frag); the GEMM that stages its own operands through swizzled
 * tiles (swz_gemm, swz_gemm_ex for a bf16 result); 8-bit floating-point
 * operands with a scale per block of 128 (swz_quant_f8) and their product
 * (swz_gemm_f8); the losses of an output layer whose logits are not kept, with
 * their gradients (swz_linear_ce, swz_linear_distill); a gated feed-forward
 * block with its gradients (swz_gated), weights of 4 bits and products of a few
 * rows with them (swz_quant_w4, swz_gemm_w4, swz_gated_w4), and the norm of
 * many tensors together (swz_grad_norm, swz_clip_grads); host-only planning, bank-conflict prediction and layout
 * algebra (swz_choose, swz_plan, swz_predict_conflicts, swz_kernel_accesses,
 * swz_bank_model_get, swz_fold); and two diagnostics (swz_copy,
 * swz_lds_probe).
 *
 * The method follows four pages on CuTe's swizzle:
 *   "NVIDIA CuTe Swizzle", "CuTe Swizzle 学习手册", "cutlass 入门",
 *   "CUDA 013 - Swizzle 的工作原理".
 */
#ifndef SWZ_H
#define SWZ_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Swizzle<B,M,S> on element offsets: the B-bit field at bit M+S is XORed
 * into the B-bit field at bit M ("CuTe Swizzle 学习手册", section on the
 * swizzle formula; "CUDA 013 - Swizzle 的工作原理", section 计算公式, where
 * the same triple is written (base, bits, shift) = (M, B, S)).  M counts
 * elements: 2^M consecutive elements stay together.  A negative S moves the
 * field the other way ("NVIDIA CuTe Swizzle", the SShift comment: a negative
 * shift moves the mask to the left): the B-bit field at bit M is XORed into
 * the field at bit M + |S|. */
typedef struct swz_params {
    int32_t B;
    int32_t M;
    int32_t S;
} swz_params;

enum swz_status {
    SWZ_OK = 0,
    SWZ_EINVAL = -1,       /* bad argument: size, pointer, alignment, overlap, parameters */
    SWZ_EUNSUPPORTED = -2, /* valid request this build does not handle */
    SWZ_EHIP = -3          /* the HIP runtime reported an error at launch */
};

/* Layout of a tile in LDS.  PAD and PLAIN are the ablations: PAD adds one
 * LDS store's width to each row: one element where the tile is staged an
 * element at a time (4-byte elements), else one vector (16 bytes for the
 * 2-byte tile kinds, 8 for the 8-bit one, 4 for the narrow-row kinds of
 * smaller elements) ("CUDA 013 - Swizzle 的工作原理", section 如何避免 Bank
 * Conflict, the 32x33 array); SWZ_EUNSUPPORTED for narrow rows under 4
 * bytes (HNARROW1, BNARROW1, BNARROW2), whose 4-byte stores span rows.
 * PLAIN is the row-major tile with no remapping.
 * SWIZZLE_DIRECT is the SWIZZLE layout filled without a trip through
 * registers: the tile moves from HBM straight into LDS (the gfx950 direct
 * load, the role cp.async plays in "NVIDIA CuTe Swizzle" and "CuTe Swizzle
 * 学习手册", usage step 2).  Such a load writes each lane's bytes at
 * consecutive LDS addresses, so the swizzle is applied on the HBM side
 * instead: the lane that fills LDS slot p fetches tile element swizzle(p),
 * which places every element exactly where SWIZZLE puts it (the swizzle is
 * its own inverse when |S| >= B).  It needs |S| >= B (or B = 0, plain rows), and
 * 16-byte aligned pointers and row pitches (SWZ_EUNSUPPORTED otherwise; for
 * the narrow-row kinds (NARROW, HNARROW, BNARROW), whose tiles are
 * contiguous stretches of the input, only the output row pitch counts). */
enum swz_layout {
    SWZ_LAYOUT_SWIZZLE = 0,
    SWZ_LAYOUT_PAD = 1,
    SWZ_LAYOUT_PLAIN = 2,
    SWZ_LAYOUT_SWIZZLE_DIRECT = 3
};

/* How a staged tile is read back from LDS.
 *  SCALAR_COL : 4-byte elements, 32x32 tile, each lane reads one element
 *               of a column (two columns per 64-lane wave).
 *  B64_4X4    : 2-byte elements, 64x64 tile, each lane reads 8-byte row
 *               pieces of 8 rows and transposes 4x4 blocks in registers.
 *  B128_8X8   : 2-byte elements, 64x128 tile, each lane reads 16-byte row
 *               pieces of 8 rows and transposes an 8x8 block in registers.
 *  MFMA_16X16X32 : operand staging; see swz_stage_operand.
 *  B64_TR16   : 2-byte elements, 64x64 tile, read with the gfx950 LDS
 *               transpose read (ds_read_b64_tr_b16, the role ldmatrix .trans
 *               plays in "NVIDIA CuTe Swizzle"): each 16-lane group
 *               addresses 8-byte row pieces and every lane receives four
 *               consecutive rows of one column, so two reads give a lane one
 *               16-byte output piece with no register shuffles.
 *  B64_TR8    : 1-byte elements, 128x128 tile, read with the gfx950 8-bit
 *               transpose read (ds_read_b64_tr_b8): each lane receives eight
 *               consecutive rows of one column per read.  The 1-byte case of
 *               "CUDA 013 - Swizzle 的工作原理", usage example 2 (char rows
 *               with the low bits kept together), here with 8-byte runs.
 *  NARROW1 .. NARROW16 : 4-byte elements in matrices of exactly 1, 2, 4, 8
 *               or 16 columns.  Each tile is 4096 bytes of whole rows
 *               (1024/cols rows), contiguous in the source, and its
 *               transpose is cols output runs of 4096/cols bytes.  A row is
 *               narrower than a bank row, so the swizzle acts on the flat
 *               offset and its source bits come from rows above the ones
 *               that form one 32-element line: it spans several rows
 *               ("CUDA 013 - Swizzle 的工作原理", usage example 4).  Reads as
 *               SCALAR_COL: each lane reads four rows of one column.
 *  HNARROW1 .. HNARROW32 : the same for 2-byte elements in matrices of 1,
 *               2, 4, 8, 16 or 32 columns, staged as 4-byte LDS writes (so
 *               M >= 1).  2 to 16 columns: 4096-byte tiles of 2048/cols
 *               rows, each lane reading eight rows of one column with 2-byte
 *               loads into 16 bytes of one output row.  1 and 32 columns:
 *               each lane reads 4-byte words (eight rows of two columns, or
 *               of the one column) and splits them in registers; tiles of
 *               2048 x 1 and 128 x 32.
 *  BNARROW1 .. BNARROW64 : the same for 1-byte elements in matrices of 1 to
 *               64 columns (powers of two), 4-byte LDS writes (M >= 2):
 *               each lane reads 4-byte words of 16 rows and up to 4 columns
 *               and transposes them in registers into up to four 16-byte
 *               output pieces; tiles of 1 KiB per column up to 4 columns,
 *               8 KiB at 8 and 16 KiB above (64, 128 and 256 lanes).
 *  ROWS       : rows of any width up to 128 columns (any element size):
 *               tiles of as many whole rows as fit in 16 KiB (up to 64
 *               columns, 256 threads) or 32 KiB (65 to 128 columns, 512
 *               threads), at least 64 lane-words' worth (256 / esz rows),
 *               copied flat into LDS, each lane gathering 4 bytes of
 *               consecutive rows of one column, each wave storing 256
 *               contiguous bytes of an output row.  Lanes of a read are cols
 *               words apart: odd widths read conflict-free as they are, even
 *               widths through a swizzle of word offsets, Swizzle<B,0,S> with
 *               B <= 10 and B <= S <= 11 (the chooser's per-width pick unless
 *               given).  Layouts SWIZZLE and PLAIN only.  Where output rows
 *               are not whole 64-byte lines and a tile's run in an output row
 *               is at most 2 KiB, the runs are shifted to start on line
 *               boundaries (the tiles then also read up to 64 / esz rows
 *               past their own).
 *  AUTO       : ROWS for the widths up to 128 that are not powers of two
 *               (4-byte elements from 96 columns on only where cols % 32 is
 *               1 to 19), and for the power-of-two widths below whose output
 *               rows or pointers are not 16-byte aligned (4-byte elements,
 *               2-byte of 8 to 32 columns, 1-byte of 64: the narrow kinds
 *               would move them element by element), in the SWIZZLE and
 *               PLAIN layouts (PAD and SWIZZLE_DIRECT keep the kinds below);
 *               otherwise 4-byte ->
 *               NARROW<cols> when cols is 1,
 *               2, 4, 8 or 16, else SCALAR_COL; 2-byte -> HNARROW<cols> when
 *               cols is a power of two up to 32, else B64_TR16 when
 *               cols <= 64, B128_8X8 when cols <= 128, B64_TR16 when
 *               cols <= 256 and B64_4X4 above (the faster of the two 64x64
 *               kinds at those widths), except B64_TR16 above 256 columns
 *               for an even number of rows whose pitches or pointers are off
 *               16 bytes or whose output rows are off the 64-byte lines;
 *               1-byte -> BNARROW<cols> when cols is
 *               a power of two up to 64, else B64_TR8. */
/* The read kind is an argument of its own (read_kind, just before
 * p_or_null, in swz_transpose, swz_convert_layout, swz_tune_tile_order and
 * the tile-order calls), and it names a kernel, not a class of read.  The
 * problem statement fixes only what moves (a row-major tile read back along
 * columns, or in the matrix-operand pattern); how a column is read back is
 * the kernel's choice, and on gfx950 there are several for one element size
 * (8-byte reads with a 4x4 register transpose, the 16-bit transpose read, a
 * 16-byte 8x8 form, whole-row tiles for narrow matrices), each with its own
 * lane map and so its own conflict-free swizzle.  A single "vector column"
 * value could not say which, so that value became these kinds, AUTO picks
 * one from the element size and width exactly as a caller without the
 * argument would get, and the operand-fragment kind moved to 3.  Callers
 * pass SWZ_READ_AUTO for the behaviour of a call without the argument. */
enum swz_read_kind {
    SWZ_READ_AUTO = -1,
    SWZ_READ_SCALAR_COL = 0,
    SWZ_READ_B64_4X4 = 1,
    SWZ_READ_B128_8X8 = 2,
    SWZ_READ_MFMA_16X16X32 = 3,
    SWZ_READ_B64_TR16 = 4,
    SWZ_READ_B64_TR8 = 5,
    SWZ_READ_NARROW1 = 6,
    SWZ_READ_NARROW2 = 7,
    SWZ_READ_NARROW4 = 8,
    SWZ_READ_NARROW8 = 9,
    SWZ_READ_NARROW16 = 10,
    SWZ_READ_HNARROW1 = 11,
    SWZ_READ_HNARROW2 = 12,
    SWZ_READ_HNARROW4 = 13,
    SWZ_READ_HNARROW8 = 14,
    SWZ_READ_HNARROW16 = 15,
    SWZ_READ_HNARROW32 = 16,
    SWZ_READ_BNARROW1 = 17,
    SWZ_READ_BNARROW2 = 18,
    SWZ_READ_BNARROW4 = 19,
    SWZ_READ_BNARROW8 = 20,
    SWZ_READ_BNARROW16 = 21,
    SWZ_READ_BNARROW32 = 22,
    SWZ_READ_BNARROW64 = 23,
    SWZ_READ_ROWS = 24
};

enum swz_frag_kind { SWZ_FRAG_MFMA_F32_16X16X32_BF16 = 0 };

/* What a call will do: tile shape, read kind, LDS layout and parameters. */
typedef struct swz_plan_info {
    int32_t read_kind;   /* resolved read kind */
    int32_t tile_rows;   /* source rows per tile */
    int32_t tile_cols;   /* source columns per tile */
    int32_t layout;      /* as requested */
    swz_params params;   /* swizzle actually used (B = 0 for PAD / PLAIN) */
    int32_t pad_elems;   /* extra elements per LDS row (PAD only) */
    int32_t lds_bytes;   /* LDS bytes one tile occupies */
    int32_t vec_bytes;   /* width of the LDS stores of the staging pass (the
                            direct fill: bytes each lane's load writes) */
    int32_t aligned;     /* 1 if the 16-byte vector path is used */
    int32_t threads;     /* threads per tile */
    int32_t interior_tiles; /* whole tiles per workgroup of the whole-tile
                            launch (threads x interior_tiles threads); a
                            tile on a ragged edge takes a workgroup alone */
} swz_plan_info;

/* out[i] = Swizzle<B,M,S>(in[i]) for i < n, on the 32-bit bit patterns
 * ("CuTe Swizzle 学习手册", swizzle formula; "CUDA 013 - Swizzle 的工作原理",
 * section 计算公式).
 *   d_in, d_out : device int32 arrays of n elements; may be the same
 *                 pointer (in place) but must not otherwise overlap.
 *   p           : B, M >= 0, any S, and B + M + |S| <= 32; B = 0 is the
 *                 identity (S = 0 with B > 0 clears the field, computed as
 *                 written).
 * Errors: SWZ_EINVAL for n < 0, NULL with n > 0, partial overlap, or
 * parameters out of range. */
int swz_map(const int32_t* d_in, int32_t* d_out, int64_t n, swz_params p, void* stream);

/* out[j][i] = Swizzle<B_j,M_j,S_j>(in[i]) for j < n_params, i < n: one
 * offset range under many triples, one launch per 128 triples (the same
 * formula as swz_map, whose single-triple calls are launch-bound at small
 * n).
 *   d_in     : device int32 array of n elements.
 *   d_out    : device int32 array [n_params][n]; must not overlap d_in.
 *   h_params : host array of n_params triples, each in swz_map's range;
 *              read during the call only.
 * Errors: SWZ_EINVAL for n < 0, n_params < 0, NULL with work to do,
 * misalignment, overlap or any triple out of range (then nothing is
 * launched); SWZ_EHIP if a launch fails (earlier chunks may have run). */
int swz_map_batch(const int32_t* d_in, int32_t* d_out, int64_t n, const swz_params* h_params, int32_t n_params,
                  void* stream);

/* dst = transpose of src: src is [rows][cols] row-major, dst is
 * [cols][rows] row-major (the column-major image of src), bit-exact.  Tiles
 * are loaded with coalesced row reads into LDS in the requested layout, read
 * back along columns, and written out with coalesced row writes
 * ("CuTe Swizzle 学习手册", typical scenario: column access of a row-major
 * tile; "CUDA 013 - Swizzle 的工作原理", sections 如何避免 Bank Conflict and
 * Swizzle 技术).  Exactly swz_convert_layout with batch = 1.
 *   elem_bytes : 1, 2 or 4.
 *   layout     : enum swz_layout.
 *   read_kind  : enum swz_read_kind (AUTO picks by element size and width).
 *   p_or_null  : swizzle to use with SWZ_LAYOUT_SWIZZLE(_DIRECT), or NULL to
 *                let swz_choose pick; ignored for PAD and PLAIN.
 * Any rows, cols >= 0 are accepted (partial edge tiles are handled); 0 is a
 * no-op.  src and dst must not overlap; they must be aligned to elem_bytes.
 * Errors: SWZ_EINVAL (sizes, NULL, overlap, misalignment, a read kind that
 * does not fit elem_bytes, parameters that split a vector or move bits
 * outside the tile, S = 0 with B > 0 (not one-to-one), |S| < B with
 * SWZ_LAYOUT_SWIZZLE_DIRECT, a narrow-row kind whose width differs from
 * cols); negative S is accepted; SWZ_EUNSUPPORTED for
 * SWZ_LAYOUT_SWIZZLE_DIRECT when a pointer or a row pitch (cols * elem_bytes
 * or rows * elem_bytes; only the latter for the narrow-row kinds) is not a
 * multiple of 16 bytes, and for SWZ_LAYOUT_PAD with a narrow-row kind whose
 * rows are narrower than 4 bytes (a padded row needs whole 4-byte writes). */
int swz_transpose(const void* d_src, void* d_dst, int64_t rows, int64_t cols, int32_t elem_bytes,
                  int32_t layout, int32_t read_kind, const swz_params* p_or_null, void* stream);

/* Batched layout conversion src[batch][rows][cols] -> dst[batch][cols][rows],
 * each batch entry transposed as in swz_transpose; same arguments and errors. */
int swz_convert_layout(const void* d_src, void* d_dst, int64_t batch, int64_t rows, int64_t cols,
                       int32_t elem_bytes, int32_t layout, int32_t read_kind,
                       const swz_params* p_or_null, void* stream);

/* Order in which the workgroups of a transpose / conversion visit the tiles
 * (of the stacked blocks of tiles where a launch stacks them): workgroups
 * with consecutive numbers q take consecutive tile rows tr, each with the
 * tile column below.  Which order the HBM system serves fastest depends on
 * the matrix shape, by up to 25% at some shapes; no order is best at all of
 * them.  All orders give the same bits.
 *
 * Shapes with no pinned order (swz_set_tile_order) take a default.  With
 * at least 2,000 rows whose output rows (rows * elem_bytes) are not whole
 * 64-byte pieces: SWZ_ORDER_COLUMNS for matrices at least 16 tiles wide,
 * SWZ_ORDER_SLOPE_32 for narrower ones.  Otherwise it is set by the source
 * row pitch (cols * elem_bytes): SWZ_ORDER_SLOPE_32 when the pitch is not
 * within 1% of a multiple of 4 KiB; otherwise the diagonal, or
 * SWZ_ORDER_SLOPE_8 for fp32 matrices with at most 10,240 rows and a side
 * that is not a power of two.  The whole-row (narrow) kinds take the
 * diagonal.  (Measured over 1,273 fp32, 1,009 16-bit and 597 byte shapes
 * of 32 to 512 MiB against a copy of the same bytes; swz_get_tile_order
 * reads a shape's order.) */
enum swz_tile_order {
    SWZ_ORDER_DIAGONAL = 0,       /* tile row tr, tile column (q + tr) mod tiles */
    SWZ_ORDER_HALF_DIAGONAL = 1,  /* tile column (q + tr / 2) mod tiles */
    SWZ_ORDER_COLUMNS = 2,        /* tile column q: every tile row of one tile column in turn */
    SWZ_ORDER_STEEP_DIAGONAL = 3, /* tile column (q + 3 tr) mod tiles */
    SWZ_ORDER_SLOPE_8 = 4,        /* tile column (q + tr / 8) mod tiles */
    SWZ_ORDER_SLOPE_16 = 5,       /* tile column (q + tr / 16) mod tiles */
    SWZ_ORDER_SLOPE_32 = 6        /* tile column (q + tr / 32) mod tiles */
};

/* Pin the tile order of later swz_transpose / swz_convert_layout calls of
 * this shape (batch, rows, cols, elem_bytes, read kind after AUTO is
 * resolved), in every layout; order = -1 removes the entry (back to the
 * shape's default order).  AUTO is resolved here as swz_plan does, for
 * 16-byte aligned pointers; a call whose pointers are not resolves AUTO
 * with them and may land on another kind, whose own entry then applies
 * (swz_tune_tile_order resolves with its buffers' pointers).  Host only;
 * the table is shared by all threads and devices of the process.
 * Errors: SWZ_EINVAL for negative sizes, an order outside -1..6, or an
 * element size / read kind that swz_convert_layout would refuse. */
int swz_set_tile_order(int64_t batch, int64_t rows, int64_t cols, int32_t elem_bytes, int32_t read_kind,
                       int32_t order);

/* The tile order later conversions of this shape will use (the pinned one,
 * or the shape's default), in *order.  Host only.
 * Errors: SWZ_EINVAL for NULL order or negative sizes; as
 * swz_set_tile_order for the element size and read kind. */
int swz_get_tile_order(int64_t batch, int64_t rows, int64_t cols, int32_t elem_bytes, int32_t read_kind,
                       int32_t* order);

/* Time every tile order on this conversion and pin the fastest: three
 * interleaved rounds over the orders, each one untimed and `reps` timed
 * swz_convert_layout calls with these arguments on the caller's buffers and
 * stream, timed with HIP events; an order counts its best round, and
 * replaces the shape's default order only when at least 3% faster (the
 * calls reuse one buffer pair, which the caches partly hold).  Synchronizes the stream;
 * allocates no device memory.  d_dst ends up holding the conversion of
 * d_src (every order writes the same bits).
 *   reps   : 1..1000.
 *   chosen : receives the pinned order (enum swz_tile_order).
 * Errors: those of swz_convert_layout (then no order is pinned for the
 * shape); SWZ_EINVAL for NULL chosen or reps out of range; SWZ_EHIP if an
 * event call fails. */
int swz_tune_tile_order(const void* d_src, void* d_dst, int64_t batch, int64_t rows, int64_t cols,
                        int32_t elem_bytes, int32_t layout, int32_t read_kind, const swz_params* p_or_null,
                        int32_t reps, int32_t* chosen, void* stream);

/* GEMM operand staging without compute.  d_src is a K-contiguous operand
 * [mn][k] (A row-major, or B column-major, which is B^T row-major), 16-bit
 * elements.  Tiles of 64 x 64 are loaded coalesced into LDS in the requested
 * layout and read back in the operand-register pattern of the 16x16x32
 * 16-bit matrix instruction: lane l holds row l%16 of a 16-row block and
 * k = 8*(l/16) .. +7 of a 32-wide k step.  Each 64-lane fragment is written
 * in lane order:
 *   d_frag[i][j][l][e] = src[16*i + l%16][32*j + 8*(l/16) + e],
 *   i < mn/16, j < k/32, l < 64, e < 8  (same byte count as src).
 * The pages' version of this step is the ldmatrix / WGMMA read of a swizzled
 * tile ("NVIDIA CuTe Swizzle", on cp.async and ldmatrix; "CuTe Swizzle
 * 学习手册", usage steps 3 and 5).
 *   elem_bytes must be 2; frag_kind must be SWZ_FRAG_MFMA_F32_16X16X32_BF16.
 *   mn must be a multiple of 16 and k of 32 (partial 64x64 tiles are fine).
 *   d_src and d_frag must be 16-byte aligned and must not overlap.
 * Errors: SWZ_EINVAL otherwise. */
int swz_stage_operand(const void* d_src, void* d_frag, int64_t mn, int64_t k, int32_t elem_bytes,
                      int32_t frag_kind, int32_t layout, const swz_params* p_or_null, void* stream);

/* Both operands of one GEMM C = A * B^T staged by one launch: A [m][k]
 * row-major into d_fa ([m/16][k/32][64][8]) and B^T [n][k] (B column-major)
 * into d_fb ([n/16][k/32][64][8]), each exactly as swz_stage_operand stages
 * it (the same tiles, layout, parameters and fragments).  One launch instead
 * of two saves one launch's start-up and drain, about 5% of two 64 MiB
 * stagings.  The same operand-read step of the pages as swz_stage_operand.
 *   m and n multiples of 16, k of 32 (m or n may be 0: the other operand
 *   alone); elem_bytes 2; frag_kind SWZ_FRAG_MFMA_F32_16X16X32_BF16.
 *   The four pointers 16-byte aligned; each fragment buffer disjoint from
 *   both sources and from the other fragment buffer (the sources are only
 *   read and may overlap each other).
 * Errors: SWZ_EINVAL otherwise, and as swz_stage_operand for the layout and
 * parameters. */
int swz_stage_operands(const void* d_a, void* d_fa, int64_t m, const void* d_bt, void* d_fb, int64_t n, int64_t k,
                       int32_t elem_bytes, int32_t frag_kind, int32_t layout, const swz_params* p_or_null,
                       void* stream);

/* Consumer of staged fragments: d_c = A * B^T in fp32, where d_fa and d_fb
 * are what swz_stage_operand wrote for A [m][k] and for B^T [n][k] (B
 * column-major), on the 16x16x32 bf16 matrix instruction with fp32
 * accumulation.  The operand read that feeds the matrix unit is the step
 * the pages put after the swizzled staging ("NVIDIA CuTe Swizzle", ldmatrix
 * and WGMMA; "CuTe Swizzle 学习手册", usage step 5); since the fragments are
 * already in lane order, each is one contiguous KiB, loaded straight into
 * LDS and read back lane-linearly (every bank once).
 *   d_c : [m][n] row-major fp32, written (not accumulated into); must not
 *         overlap the inputs.
 *   m, n multiples of 16, k a multiple of 32 (the fragment format); k = 0
 *   writes zeros.  All pointers 16-byte aligned.  frag_kind must be
 *   SWZ_FRAG_MFMA_F32_16X16X32_BF16.
 * The sum over k is taken 32 at a time by the instruction and accumulated
 * in fp32 in increasing k order.
 * Errors: SWZ_EINVAL (sizes, alignment, NULL, overlap, fragment kind). */
int swz_gemm_frag(const void* d_fa, const void* d_fb, float* d_c, int64_t m, int64_t n, int64_t k,
                  int32_t frag_kind, void* stream);

/* GEMM with the staging inside: d_c = A * B^T in fp32 from bf16 operands in
 * their natural layouts, A [m][k] row-major (d_a) and B^T [n][k] row-major
 * (d_bt; B column-major).  This is the use the pages build the swizzle for:
 * each k stage copies a 256 x 64 tile of A and one of B^T from HBM straight
 * into a swizzled LDS tile (the cp.async step), and the operand reads take
 * the 16x16x32 instruction's fragments out of it (the ldmatrix step) --
 * "NVIDIA CuTe Swizzle", cp.async, ldmatrix and the MMA; "CuTe Swizzle
 * 学习手册", usage steps 2, 3 and 5.  The tile is the one swz_stage_operand
 * stages, read in the same pattern.
 *   layout    : SWZ_LAYOUT_SWIZZLE or SWZ_LAYOUT_SWIZZLE_DIRECT (the same
 *               here: the fill is always direct), or SWZ_LAYOUT_PLAIN (the
 *               ablation: row-major tiles, whose fragment reads conflict).
 *               SWZ_LAYOUT_PAD returns SWZ_EUNSUPPORTED (a direct load
 *               writes whole unpadded rows).
 *   p_or_null : the swizzle for the SWIZZLE layouts (|S| >= B, as for
 *               SWZ_LAYOUT_SWIZZLE_DIRECT), or NULL for the chooser's.
 *   d_c       : [m][n] row-major fp32, written (not accumulated into); must
 *               not overlap the inputs.
 *   m, n multiples of 16, k a multiple of 32; k = 0 writes zeros.  All
 *   pointers 16-byte aligned.
 * The products are exact in fp32 and the sum over k is accumulated in fp32,
 * 32 at a time by the instruction, in increasing k order -- the same result
 * as swz_gemm_frag on the staged operands.
 * Errors: SWZ_EINVAL (sizes, alignment, NULL, overlap, parameters),
 * SWZ_EUNSUPPORTED (PAD). */
int swz_gemm(const void* d_a, const void* d_bt, float* d_c, int64_t m, int64_t n, int64_t k, int32_t layout,
             const swz_params* p_or_null, void* stream);

/* Element type of the GEMM result. */
enum swz_c_type { SWZ_C_F32 = 0, SWZ_C_BF16 = 1 };

/* swz_gemm with a choice of result type: c_type SWZ_C_F32 is swz_gemm
 * (d_c float [m][n]); SWZ_C_BF16 writes d_c as bf16 [m][n] (uint16 bit
 * patterns), each element the fp32 result of swz_gemm rounded to nearest
 * with ties to even (NaN stays NaN), half the bytes of C to write.
 * Errors: those of swz_gemm; SWZ_EINVAL for another c_type. */
int swz_gemm_ex(const void* d_a, const void* d_bt, void* d_c, int64_t m, int64_t n, int64_t k, int32_t layout,
                const swz_params* p_or_null, int32_t c_type, void* stream);

/* Element types of the operators below. */
enum swz_x_type { SWZ_X_BF16 = 0, SWZ_X_F16 = 1, SWZ_X_F32 = 2 };
/* 8-bit floating point: e4m3 (largest value 448, no infinities) and e5m2
 * (57344, with infinities). */
enum swz_f8_type { SWZ_F8_E4M3 = 0, SWZ_F8_E5M2 = 1 };
/* What shares a scale: 128 consecutive elements of a row (the last block of
 * a row may be shorter), or a square of 128 x 128. */
enum swz_f8_block { SWZ_BLOCK_1X128 = 0, SWZ_BLOCK_128X128 = 1 };
/* How scales are stored: fp32, or one byte e + 127 for 2^e (byte 255: NaN). */
enum swz_scale_type { SWZ_SCALE_F32 = 0, SWZ_SCALE_E8M0 = 1 };

/* A matrix to 8-bit floating point with a power-of-two scale per block, and
 * on request its transpose, which the gradient products contract over.
 *   d_x       : x_type [rows][ld_x], ld_x >= cols elements; the last row ends
 *               behind its cols, here and below (columns of a wider matrix).
 *   d_q       : 8-bit [rows][ld_q]; columns cols .. ld_q - 1 stay as they were.
 *   d_scale   : SWZ_BLOCK_1X128   [rows][ceil(cols / 128)],
 *               SWZ_BLOCK_128X128 [ceil(rows / 128)][ceil(cols / 128)].
 *   d_qt, d_scale_t : the same of the transposed matrix, [cols][ld_qt] and
 *               [cols or ceil(cols / 128)][ceil(rows / 128)].  With row blocks
 *               the transpose is rounded from x with scales of its own.
 *   Either output pair may be NULL (not both).  ld_q, ld_qt: bytes, multiples
 *   of 16, as swz_gemm_f8 takes them; d_q and d_qt 16-byte aligned, d_x
 *   aligned to its element.  Rows of x whose pitch and start are multiples of
 *   16 bytes, with cols a multiple of 8, move in 16-byte pieces.
 * With a the largest finite magnitude of a block and F the format's largest
 * value, the scale is 2^e, e >= -127 the smallest integer with a <= F 2^e
 * (e = 0 for a block without a finite nonzero element); each element is
 * x 2^-e rounded to nearest, ties to even.  NaN becomes NaN; infinities stay
 * infinities in e5m2 and become NaN in e4m3.
 * Errors: SWZ_EINVAL (sizes, pitches, alignment, NULL, overlap, enum values),
 * SWZ_EUNSUPPORTED (more than 2^23 tiles of 128 x 128 with a transpose or
 * square blocks). */
int swz_quant_f8(const void* d_x, int32_t x_type, int64_t rows, int64_t cols, int64_t ld_x, int32_t f8_type,
                 int32_t block, int32_t scale_type, void* d_q, void* d_scale, int64_t ld_q, void* d_qt,
                 void* d_scale_t, int64_t ld_qt, void* stream);

/* C = A B^T of 8-bit operands with a scale per block of 128 along k:
 *   C[i][j] = sum over blocks b of sA[i][b] sB[j][b] sum over k in b of A[i][k] B[j][k].
 *   d_a       : a_type [m][lda]; d_b : b_type [n][ldb]; lda, ldb >= k bytes,
 *               multiples of 16 and below 2^23; bytes behind column k are not
 *               used, whatever they hold, and the last row ends behind k rounded
 *               up to 16 (a part of k of a wider operand is one too).
 *   d_scale_a : scale_type, laid out as swz_quant_f8 writes it for a_block;
 *   d_scale_b : the same for b_block.
 *   d_c       : float or bf16 (c_type, enum swz_c_type) [m][n], written
 *               whatever it held (k = 0 writes zeros); must not overlap the
 *               inputs.
 * A forward product takes activations in rows (1x128) and weights in squares
 * (128x128); the data gradient the weight's transpose; the weight gradient
 * both transposes in rows.  Any m, n, k >= 0; calls with up to 16 rows of A go
 * to a kernel that streams B once.  d_a, d_b 16-byte aligned, fp32 scales
 * 4-byte, d_c aligned to its element; rows of C whose pitch and start are
 * multiples of 16 bytes are written in 16-byte pieces.
 * A float C is summed in fp32 from exact products (the operands widened to
 * bf16, at the bf16 rate); with SWZ_SCALE_E8M0 a value times its scale has to
 * be a normal bf16 number for that.  So is a bf16 C of at most 16 rows; any other takes the 8-bit matrix
 * instruction, which adds the products of each eight consecutive k after
 * dropping what lies more than 13 bits below the largest of them (1.5e-5 of
 * the norm of a product of normal operands, a hundredth of the rounding to
 * bf16), sums those in fp32 and is rounded once, to nearest even.  fp32 scales
 * multiply fp32 sums within their block, by the product of a block's two
 * scales, which has to be a normal fp32 number.
 * NaN and infinities in the used elements and scales propagate.
 * Errors: SWZ_EINVAL (sizes, pitches, alignment, NULL, overlap, enum values),
 * SWZ_EUNSUPPORTED (lda or ldb of 2^23 and more; n of 2^26 and more; over 2^22
 * tiles of 256 x 256 of C). */
int swz_gemm_f8(const void* d_a, const void* d_scale_a, const void* d_b, const void* d_scale_b, void* d_c, int64_t m,
                int64_t n, int64_t k, int64_t lda, int64_t ldb, int32_t a_type, int32_t b_type, int32_t a_block,
                int32_t b_block, int32_t scale_type, int32_t c_type, void* stream);

/* Host only.  Bytes of workspace that the losses below need for n rows, v
 * words, k features and `top` entries a row (1 for cross entropy): grad 0,
 * the forward calls; 1, enough for the forward and the gradient calls.  A
 * workspace is 256-byte aligned device memory that carries nothing from one
 * call to the next; calls that may run at the same time (on two streams, in
 * two graphs) need one each.  The forward calls take 8 bytes a row and 256
 * words, a 64th of bf16 logits.  The gradient calls hold dz of a piece of up
 * to 32768 words twice, that piece of W once and H once (2 bytes each), and
 * dH's sums (4 bytes, up to 32 times where there are few rows): less than bf16
 * logits where the vocabulary is many pieces long (4096 x 262144 x 4096: 906 MB,
 * logits 2147), more where it is not or the rows are few (4096 x 65536 x 4096:
 * 906 and 537; 64 x 128256 x 4096: 290 and 16).
 * Errors: SWZ_EINVAL, SWZ_EUNSUPPORTED (sizes, as the calls). */
int swz_linear_loss_workspace(int64_t n, int64_t v, int64_t k, int32_t top, int32_t grad, int64_t* bytes);

/* Softmax cross entropy of the logits z = H W^T, in pieces of the vocabulary
 * and without keeping them:
 *   lse[i] = log sum over v of exp(z[i][v]),  loss[i] = lse[i] - z[i][target[i]].
 *   d_h      : x_type (SWZ_X_BF16 or SWZ_X_F16) [n][k]; d_w : the same type
 *              [v][k]; k a multiple of 8, both 16-byte aligned.
 *   d_target : int64 [n].  A target outside 0 .. v - 1 marks a row that does
 *              not count: its loss is 0 and it adds nothing to the gradients.
 *   d_loss, d_lse, d_zt : float [n]; zt is the logit at the target (0 for rows
 *              that do not count).  lse and zt are what the gradient call takes.
 * Products are exact in fp32 and summed in fp32; lse is never below zt, so a
 * loss is never negative.  A row with a logit that is NaN or +infinity has a
 * NaN lse.
 * Nothing written may overlap anything else.  n = 0 does nothing.
 * Errors: SWZ_EINVAL (sizes, alignment, NULL, overlap, x_type, a workspace
 * below swz_linear_loss_workspace), SWZ_EUNSUPPORTED (n or k of 2^22 and more,
 * v of 2^31 and more, over 2^22 tiles of 256 x 256 logits). */
int swz_linear_ce(const void* d_h, const void* d_w, int32_t x_type, const int64_t* d_target, float* d_loss,
                  float* d_lse, float* d_zt, int64_t n, int64_t v, int64_t k, void* d_ws, int64_t ws_bytes,
                  void* stream);

/* Its gradients, for upstream[i] = d(total) / d(loss[i]) (float [n]):
 *   dz[i][v] = upstream[i] (exp(z[i][v] - lse[i]) - [v = target[i]]),
 *   dh = dz W ([n][k]), dw = dz^T H ([v][k]), both x_type, overwritten; either
 * may be NULL.  The logits are computed again, a piece of the vocabulary at a
 * time.  Sums are fp32 and rounded to x_type at the end; their operands are
 * held in fp16 (half a step 2^-11): dz with its row's upstream taken out but
 * for a factor between 1/2 and 1, so that a row of dh keeps its digits however
 * small its upstream is beside the others' (absolutely, dz / upstream is good
 * to 2^-38); W, and H's rows times their upstream's power of two, with a power
 * of two that keeps values down to 2^-28 of the largest exact.  With fp16
 * results that rounding of dz is as large as the result's own.  Rows that do
 * not count may hold any numbers or NaN.  n = 0 writes a zero dw.  Results do
 * not depend on the order of anything: the same call gives the same bits.
 * Errors: as swz_linear_ce. */
int swz_linear_ce_grad(const void* d_h, const void* d_w, int32_t x_type, const int64_t* d_target, const float* d_lse,
                       const float* d_zt, const float* d_upstream, void* d_dh, void* d_dw, int64_t n, int64_t v,
                       int64_t k, void* d_ws, int64_t ws_bytes, void* stream);

/* Distillation from a teacher's top logits, without keeping the student's:
 *   p[i] = softmax over the row's entries of teacher[i][j] / tau,
 *   lse[i] = log sum over v of exp(z[i][v] / tau),
 *   loss[i] = tau^2 sum over j of p[i][j] (log p[i][j] - (z[i][index[i][j]] / tau - lse[i])).
 *   d_index   : int64 [n][top]; d_teacher : float [n][top]; 1 <= top <= 256.
 *               Entries whose index is outside 0 .. v - 1 or whose logit is
 *               -infinity are absent; a row without entries has loss 0 and adds
 *               nothing to the gradients.  Equal indices add up.
 *   d_zt      : float [n][top], the student's logits (before tau) at the entries.
 *   tau       : > 0, finite and a normal number.  The loss is tau^2 times a
 *               difference of fp32 numbers of the size of lse, and z / tau has
 *               to stay within fp32.
 * The rest, and the errors, as swz_linear_ce (SWZ_EUNSUPPORTED also for top
 * above 256). */
int swz_linear_distill(const void* d_h, const void* d_w, int32_t x_type, const int64_t* d_index,
                       const float* d_teacher, int32_t top, float tau, float* d_loss, float* d_lse, float* d_zt,
                       int64_t n, int64_t v, int64_t k, void* d_ws, int64_t ws_bytes, void* stream);

/* Its gradients with respect to H and W, as swz_linear_ce_grad:
 *   dz[i][v] = upstream[i] tau (exp(z[i][v] / tau - lse[i]) - sum over j with index[i][j] = v of p[i][j]). */
int swz_linear_distill_grad(const void* d_h, const void* d_w, int32_t x_type, const int64_t* d_index,
                            const float* d_teacher, int32_t top, float tau, const float* d_lse, const float* d_zt,
                            const float* d_upstream, void* d_dh, void* d_dw, int64_t n, int64_t v, int64_t k,
                            void* d_ws, int64_t ws_bytes, void* stream);

/* Activations of the gated calls: z / (1 + e^-z); z Phi(z) with the normal
 * distribution's Phi; and z (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))) / 2. */
enum swz_act { SWZ_ACT_SILU = 0, SWZ_ACT_GELU = 1, SWZ_ACT_GELU_TANH = 2 };

/* A gated feed-forward block's two projections, its activation and the
 * product:
 *   g = x Wg^T,  u = x Wu^T,  y = act(g) u.
 *   d_x      : x_type (SWZ_X_BF16 or SWZ_X_F16) [n][k]; d_wg, d_wu : the same
 *              type [f][k]; k a multiple of 8, all 16-byte aligned.
 *   d_y      : x_type [n][f], aligned to its element.
 *   d_pre    : NULL, or float [2][n][f]: g, then u, for the gradient call.
 * g and u are exact products summed in fp32; y is rounded once.  Calls of up to
 * 16 rows, and of up to 32 where f k is at most 2^22, go to a kernel that streams
 * both weights once.  Nothing written may overlap anything else.  n = 0 does nothing.
 * Errors: SWZ_EINVAL (sizes, alignment, NULL, overlap, enum values),
 * SWZ_EUNSUPPORTED (n, f or k of 2^22 - 8 and more, over 2^21 tiles of
 * 256 x 128 of y, 256 x 256 of a gradient). */
int swz_gated(const void* d_x, const void* d_wg, const void* d_wu, int32_t x_type, int32_t act, void* d_y, float* d_pre,
              int64_t n, int64_t f, int64_t k, void* stream);

/* Host only.  Bytes of workspace of the gradient call: 256-byte aligned device
 * memory that carries nothing from one call to the next; calls that may run at
 * the same time (on two streams, in two graphs) need one each.  It holds dg and
 * du (2 bytes each a place of y; 4 where n f k is up to 2^23), 16,640 bytes, and,
 * where a gradient has few tiles, fp32 sums of its parts.
 * Errors: as swz_gated. */
int swz_gated_workspace(int64_t n, int64_t f, int64_t k, int64_t* bytes);

/* Its gradients, for dy = d(total) / dy (x_type [n][f]):
 *   dg = dy u act'(g),  du = dy act(g),
 *   dx = dg Wg + du Wu ([n][k]),  dwg = dg^T x,  dwu = du^T x ([f][k]),
 * all x_type, overwritten, 16-byte aligned; each may be NULL (not all).
 *   d_pre    : what swz_gated wrote there, or NULL: g and u are made again, for
 *              4 n f k operations more.
 * dg and du are rounded to x_type once (as they are where a program holds
 * them), and for n f k up to 2^23, where few values would leave the
 * results up to 1.8 times the error of their own rounding, what that rounding
 * left is held too.  With fp16 both are held times a power of two of their own
 * where the call's largest finite value of one is beyond the type's range or
 * below 2^-4: a value of 2^-10 of the largest and more keeps all its digits, and a
 * smaller one is off by at most 2^-21 of the largest.
 * Sums are fp32 and rounded to x_type at the end.  n = 0 writes zero dwg and
 * dwu.  Results do not depend on the order of anything:
 * the same call gives the same bits.
 * Errors: as swz_gated, and SWZ_EINVAL for a workspace below
 * swz_gated_workspace. */
int swz_gated_grad(const void* d_x, const void* d_wg, const void* d_wu, int32_t x_type, int32_t act, const void* d_dy,
                   const float* d_pre, void* d_dx, void* d_dwg, void* d_dwu, int64_t n, int64_t f, int64_t k, void* d_ws,
                   int64_t ws_bytes, void* stream);

/* Weights of 4 bits: w = (code - zero) scale, with a scale, and on request a
 * zero point, per `group` consecutive values of a row (32, 64 or 128; a row's
 * last group may be shorter).
 *   d_w     : w_type (enum swz_x_type) [n][k], k a multiple of 32.
 *   d_q     : [n][k / 2] bytes: the even column's code in the low half.
 *   d_scale : x_type (SWZ_X_BF16 or SWZ_X_F16) [n][ceil(k / group)].
 *   d_zero  : NULL (every zero point is 8), or one byte per group, the same
 *             shape.
 * Without zero points scale is the group's largest magnitude times 1/7, with them
 * its range, widened to hold zero, times 1/15 (as fp32 numbers), in fp32 and
 * rounded to x_type; zero = -lowest / scale and code = w / scale + zero, quotients
 * in fp32 rounded to the nearest whole number, ties to even, and both cut to
 * 0 .. 15.  A group
 * whose scale comes out 0 is zero; one with a NaN or an infinity, or whose scale
 * leaves x_type, has a NaN scale.
 *   d_w and d_q 16-byte aligned, d_scale to its element.
 * Nothing written may overlap anything else.
 * Errors: SWZ_EINVAL (sizes, alignment, NULL, overlap, enum values, group),
 * SWZ_EUNSUPPORTED (n k of 2^34 and more). */
int swz_quant_w4(const void* d_w, int32_t w_type, int64_t n, int64_t k, int32_t group, int32_t x_type, void* d_q,
                 void* d_scale, uint8_t* d_zero, void* stream);

/* And back: d_w x_type [n][k] = (code - zero) scale, rounded once; any scales
 * and zero points (0 .. 255).  Buffers and errors as swz_quant_w4.  For many rows of x
 * the product of this is the faster one: swz_gated, or swz_gemm_ex where it takes
 * the operands (bf16, and rows and columns in sixteens). */
int swz_dequant_w4(const void* d_q, const void* d_scale, const uint8_t* d_zero, int64_t n, int64_t k, int32_t group,
                   int32_t x_type, void* d_w, void* stream);

/* C = X W^T of such weights, for few rows of X:
 *   d_x : x_type [m][k]; d_c : x_type [m][n], written whatever it held, aligned
 *   to its element; d_x and d_q 16-byte aligned.
 * Products are exact in fp32 (x times 16 + code) and summed in fp32, a group's
 * sum less (16 + zero) times the group's sum of x, and that times its scale in
 * fp32; the result is rounded once.  A group's sum of |x| (32 + zero) has to stay
 * within fp32 (any fp16 x does); a row of X that holds an infinity or NaN comes
 * out NaN, and the other rows as they would without it.
 * Meant for few rows: each 64 read the weights once.  swz_dequant_w4 with a
 * product of that, where swz_gemm_ex takes it, is the faster one from some 500
 * rows on (512 rows with 8192 x 4096: 101 us here, 113 so), for the gated block from
 * some 200 on.
 * m = 0 does nothing; any n.
 * Errors: SWZ_EINVAL (sizes, alignment, NULL, overlap, enum values, group),
 * SWZ_EUNSUPPORTED (m or k of 2^22 and more, n of 2^26 and more, n k of 2^34
 * and more). */
int swz_gemm_w4(const void* d_x, int32_t x_type, const void* d_q, const void* d_scale, const uint8_t* d_zero, int32_t group,
                void* d_c, int64_t m, int64_t n, int64_t k, void* stream);

/* The gated block of two such weights, C = act(X Wg^T) (X Wu^T): both with zero
 * points or both without.  The rest, and the errors, as swz_gemm_w4. */
int swz_gated_w4(const void* d_x, int32_t x_type, int32_t act, const void* d_qg, const void* d_scale_g,
                 const uint8_t* d_zero_g, const void* d_qu, const void* d_scale_u, const uint8_t* d_zero_u, int32_t group,
                 void* d_c, int64_t m, int64_t n, int64_t k, void* stream);

/* Host only.  Bytes of workspace (8-byte aligned device memory) of the two
 * calls below for `count` tensors: 16 KiB for each 64 of them.  It carries
 * nothing from one call to the next, and calls that may run at the same time
 * need one each.
 * Errors: SWZ_EINVAL (count < 0, NULL), SWZ_EUNSUPPORTED (over 2^20 tensors). */
int swz_grad_norm_workspace(int32_t count, int64_t* bytes);

/* d_norm[0] = sqrt(sum over all tensors of the sum of their squares), squares
 * and sums in fp64; the same call gives the same bits.
 *   d_t, numel, type : host arrays of `count` device addresses, sizes in
 *                      elements (0 allowed, then with any address) and types
 *                      (enum swz_x_type), read during the call only.
 * Tensors aligned to their element.
 * Errors: SWZ_EINVAL (NULL, sizes, types, alignment, overlap of what is written
 * with anything, a workspace below swz_grad_norm_workspace), SWZ_EUNSUPPORTED
 * (over 2^20 tensors, or one of 2^38 elements and more). */
int swz_grad_norm(const void* const* d_t, const int64_t* numel, const int32_t* type, int32_t count, float* d_norm,
                  void* d_ws, int64_t ws_bytes, void* stream);

/* The tensors scaled so that their norm together is at most max_norm (>= 0; may
 * be infinite): out = x factor, in fp32 and rounded once, with factor =
 * max_norm / norm where the norm is over max_norm and finite, else 1 (tensors as
 * they were: what to do about infinities and NaN is the caller's to say, from
 * the norm).  d_norm[0] is the norm before, d_norm[1] the factor.  Finite tensors
 * whose norm is beyond fp32 are scaled too: d_norm[0] then reads infinite, with a
 * factor below 1 beside it.
 *   d_out : NULL, in place (then a factor of 1 writes nothing); or a host array
 *           of `count` device addresses, each its tensor's own or apart from
 *           everything.
 * The same memory may not stand in the list twice.
 * Errors: as swz_grad_norm; SWZ_EINVAL for a max_norm that is negative or NaN. */
int swz_clip_grads(const void* const* d_t, void* const* d_out, const int64_t* numel, const int32_t* type, int32_t count,
                   float max_norm, float* d_norm, void* d_ws, int64_t ws_bytes, void* stream);

/* Host only.  The swizzle the library uses for a tile of tile_rows x
 * tile_cols elements of elem_bytes, staged by vec_bytes-wide stores and read
 * back by read_kind, under the built-in gfx950 LDS bank model:
 * M = log2(vec_bytes / elem_bytes), B = log2(vectors per bank row) (bounded
 * by the tile), S the smallest shift >= B with the fewest predicted
 * bank-conflict cycles over the kernel's write and read lane patterns
 * ("NVIDIA CuTe Swizzle", derivation of the three parameters; "CUDA 013 -
 * Swizzle 的工作原理", section CuTe 通用 swizzle 映射规则解析).  Only the
 * (elem_bytes, vec_bytes, tile, read_kind) combinations the kernels use are
 * accepted; others return SWZ_EUNSUPPORTED. */
int swz_choose(int32_t elem_bytes, int32_t vec_bytes, int32_t tile_rows, int32_t tile_cols,
               int32_t read_kind, swz_params* out);

/* Host only.  Folding a swizzle into a plain layout over a slice ("cutlass
 * 入门", section swizzle 融入 layout 优化).  A slice is the set of offsets
 * base | x with x ranging over the subsets of the bit mask `active` (the bits
 * a slice's coordinates can change; base has none of them).  The page's test:
 * collision = active & ~swizzle(active) marks every target bit whose source
 * bit is also active; when it is zero the swizzle restricted to the slice is
 * a plain (strided) layout:
 *   swizzle(base | x) = swizzle(base) + sum over set bits b of x of strides[b].
 *   p          : the swizzle (S of either sign; B + M + |S| <= 32).
 *   *collision : the collision bits (always written).
 *   *folded_base, strides[32] : swizzle(base) and the signed per-bit strides
 *                (strides[b] = 0 for bits outside `active`), written only
 *                when the slice folds; either may be NULL.
 * Returns SWZ_OK when the slice folds, SWZ_EUNSUPPORTED when it does not
 * (collision != 0), SWZ_EINVAL for bad parameters, base & active != 0 or a
 * NULL collision pointer. */
int swz_fold(const swz_params* p, uint32_t base, uint32_t active, uint32_t* collision, uint32_t* folded_base,
             int64_t* strides);

/* Host only.  Predicted conflict cycles (write + read, summed over one
 * tile) of the kernel pattern for read_kind under the built-in bank model,
 * for the given layout and parameters (params ignored for PAD and PLAIN;
 * with SWIZZLE_DIRECT the writes are the direct fill's lane-linear ones). */
int swz_predict_conflicts(int32_t read_kind, int32_t layout, const swz_params* p_or_null,
                          int64_t* write_cycles, int64_t* read_cycles);

/* Host only.  The LDS accesses one tile of the kernel for read_kind issues,
 * as byte addresses per lane: the staging stores (is_write = 1) or the reads
 * (is_write = 0), one 64-lane access after another (all waves, all steps),
 * in the given layout.  Writes min(count, max_accesses) x 64 addresses to
 * addrs (int32, -1 = lane idle), the total count to *n_accesses and the
 * bytes per lane to *width.  Lets tests and the bank microbenchmark check
 * the exact patterns the kernels use. */
int swz_kernel_accesses(int32_t read_kind, int32_t layout, const swz_params* p_or_null, int32_t is_write,
                        int32_t* addrs, int32_t max_accesses, int32_t* n_accesses, int32_t* width);

/* The LDS bank model the chooser uses, per access direction d (0 = read,
 * 1 = write) and width w (4 << w bytes per lane): n_banks banks of
 * bank_bytes, byte a in bank (a / bank_bytes) % n_banks ("CuTe Swizzle
 * 学习手册", bank structure, gives one geometry, 32 x 4 bytes, for NVIDIA;
 * gfx950's depends on the access and is measured with swz_lds_probe), and
 * phase[d][w][l], the group of lanes served together. */
typedef struct swz_bank_model {
    int32_t n_banks[2][3];
    int32_t bank_bytes[2][3];
    uint8_t phase[2][3][64];
} swz_bank_model;

/* Host only.  Copy the built-in gfx950 model to *out.  SWZ_EINVAL on NULL. */
int swz_bank_model_get(swz_bank_model* out);

/* Host only.  Fill *out with what swz_convert_layout (op = 0) or
 * swz_stage_operand (op = 1) would do for these arguments, without
 * launching anything; pointers are not inspected (they are taken to be
 * 16-byte aligned, so aligned reflects the row pitches).  Same validation and
 * errors as the call. */
int swz_plan(int32_t op, int64_t rows, int64_t cols, int32_t elem_bytes, int32_t layout,
             int32_t read_kind, const swz_params* p_or_null, swz_plan_info* out);

/* Host only.  Static text for a status code. */
const char* swz_strerror(int status);

/* Reference copy (diagnostic): d_dst[0..bytes) = d_src[0..bytes) with plain
 * 16-byte vector loads and stores and the same launch policy as the tile
 * kernels.  It is the read-once / write-once ceiling the tile kernels are
 * compared with, and the kernel of known size HBM byte counters are scaled
 * by.  bytes must be a multiple of 16, pointers 16-byte aligned, buffers
 * disjoint.  Errors: SWZ_EINVAL otherwise. */
int swz_copy(const void* d_src, void* d_dst, int64_t bytes, void* stream);

/* LDS bank microbenchmark (diagnostic; used to measure the bank model the
 * chooser relies on).  Launches n_patterns workgroups of `waves` 64-lane
 * waves.  Workgroup g runs pattern g: lane l of every wave accesses LDS byte
 * d_addrs[64*g + l] (taken modulo the probe's 96 KiB LDS window and aligned
 * down to width_bytes) if bit l of d_masks[g] is set, with ds_read_u8/u16/
 * b32/b64/b128 (is_write = 0) or ds_write_b8/b16/b32/b64/b128
 * (is_write = 1), 8 accesses per iteration for `iters` iterations, and
 * writes the wave's elapsed shader-clock cycles to d_cycles[g * waves + w].
 *   width_bytes: 1, 2, 4, 8 or 16; waves: 1..16; iters: 1..1<<20.
 * Errors: SWZ_EINVAL on any other value or NULL pointer. */
int swz_lds_probe(const uint32_t* d_addrs, const uint64_t* d_masks, int32_t n_patterns,
                  int32_t width_bytes, int32_t is_write, int32_t iters, int32_t waves,
                  uint64_t* d_cycles, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SWZ_H */
